// Prompt attention (causal, packed sequences, grouped heads): what its kernels share.
#pragma once

#include "kv4.cuh"

namespace spt {

struct PromptProblem {
  spatten_prompt_args a;   // sm_scale > 0 and cu_kv set
  // with weights only (else NULL).  CUDA cores: [H][total_q] score maximum (log2 units) and exponential
  // sum of each row.  Tensor cores: the negated maximum and the reciprocal of the sum (0 where a row
  // sees nothing) in two planes [H][total_q], and the heads' column sums [H][total_kv] (grouped heads).
  float2* stats;
  float* stat_m;
  float* stat_l;
  float* part;
  uint32_t wait_limit;     // polls of one pipeline wait (tensor-core kernels)
};

// The sequence and tile of block t, for tiles of `rows` packed rows that start anew at each sequence:
// tiles are counted from the last sequence's last tile backwards, so that a sequence's late rows, which
// see the most keys, are started first (FRONT: from the first sequence's first tile).  Every warp calls
// it whole; b = -1 past the last tile.
struct SeqTile {
  int b, tile;
};
template <bool FRONT = false>
__device__ __forceinline__ SeqTile find_seq_tile(const int32_t* cu, int B, int total, int rows, int t) {
  const int lane = threadIdx.x & 31;
  int all = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    int c = b0 + lane < B ? (packed_rows(cu, b0 + lane, total).n + rows - 1) / rows : 0;
    all += warp_sum_int(c);
  }
  int want = FRONT ? t : all - 1 - t;
  if (want < 0 || want >= all) return {-1, 0};
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int c = b0 + lane < B ? (packed_rows(cu, b0 + lane, total).n + rows - 1) / rows : 0;
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const int sum = __shfl_sync(0xffffffffu, inc, 31);
    if (want < sum) {
      const uint32_t past = __ballot_sync(0xffffffffu, want < inc);
      const int l = __ffs(past) - 1;
      const int before = __shfl_sync(0xffffffffu, inc - c, l);
      return {b0 + l, want - before};
    }
    want -= sum;
  }
  return {-1, 0};
}

// Reports offsets that decrease or leave their block (one block of a call does it).
__device__ __forceinline__ void report_bad_offsets(const spatten_prompt_args& a) {
  for (int b = threadIdx.x; b < a.B; b += blockDim.x)
    if (packed_rows(a.cu_q, b, a.total_q).bad || packed_rows(a.cu_kv, b, a.total_kv).bad)
      report(a.dev_status, SPATTEN_E_INDEX);
}

int32_t prompt_simt_launch(const PromptProblem& p, cudaStream_t st);
int32_t prompt_tc_launch(const PromptProblem& p, cudaStream_t st);
bool prompt_tc_supported(const spatten_prompt_args& a);

}  // namespace spt
