// Prompt attention (causal, packed sequences, grouped heads): what its kernels share.
#pragma once

#include "kv4.cuh"

namespace spt {

struct PromptProblem {
  spatten_prompt_args a;   // sm_scale > 0 and cu_kv set
  // with weights only (else NULL)
  // [H][total_q] CUDA cores: score maximum (log2 units) and reciprocal of the exponential sum of each row
  // (0, 0 where a row sees nothing); tensor cores: what each row's scores need added (before the softmax
  // scale) for their exponentials to be P
  float2* stats;
  float* offset;
  uint16_t* planes[3];     // float32 on tensor cores: q, k, v as [3][rows][heads][d_h] bfloat16 terms
  float* part;             // [H][total_kv] the heads' column sums (grouped heads)
  // few rows against long sequences: the key tiles of a row tile are dealt to `splits` CTAs (else 1), which leave
  int32_t splits;
  float2* split_ml;        // [splits][H][total_q] maximum (log2 units) and sum of each row
  float* split_o;          // [splits][H][total_q][d_h] and its output, relative to that maximum
  uint32_t wait_limit;     // polls of one pipeline wait (tensor-core kernels)
};

// Block number t's tile: KEYS = false, a tile of `rows` query rows, else of `rows` key rows (rows a multiple of
// 128), with the sequence's rows.  Tiles with the most work come first -- for up to 32 sequences over all of
// them (work in units of 128 rows against 128 keys), else within a sequence -- since the last blocks to start
// decide when the kernel ends (16 sequences of up to 1024 rows, 16 heads of 64: 70 us, in the plain order 79; 32 of
// them 111 and 123).  A lane holds a sequence, so that more of them take the plain order (33: 128 us).  Every warp
// calls it whole; b = -1 past the last tile.
struct PromptTile {
  int b, tile;
  PackedRows q, k;
};
template <bool KEYS>
__device__ __forceinline__ PromptTile find_prompt_tile(const spatten_prompt_args& a, int rows, int t) {
  PromptTile r;
  if (a.B > 32) {
    const SeqTile st = find_seq_tile<KEYS>(KEYS ? a.cu_kv : a.cu_q, a.B, KEYS ? a.total_kv : a.total_q, rows, t);
    r.b = st.b;
    r.tile = st.tile;
    if (st.b >= 0) {
      r.q = packed_rows(a.cu_q, st.b, a.total_q);
      r.k = packed_rows(a.cu_kv, st.b, a.total_kv);
    }
    return r;
  }
  // lane b holds sequence b; its tiles in the order of their work, that of the p-th being
  //   query tiles: top - p (the last tile first);  key tiles: top - max(0, p - early) (the first tile first)
  const int lane = threadIdx.x & 31;
  PackedRows q{0, 0, false}, k{0, 0, false};
  if (lane < a.B) {
    q = packed_rows(a.cu_q, lane, a.total_q);
    k = packed_rows(a.cu_kv, lane, a.total_kv);
  }
  const int unit = rows / 128, shift = k.n - q.n;
  const int tiles = ((KEYS ? k.n : q.n) + rows - 1) / rows;
  const int early = KEYS ? max(0, shift) / rows : 0;   // key tiles that (nearly) every row sees
  const int top = KEYS ? (q.n + 127) / 128 : max(0, tiles - 1 + (shift + rows - 1) / rows);
  auto at_least = [&](int level) {   // how many of the lane's tiles have that much work
    const int n = KEYS ? (level <= top ? early + 1 + (top - level) / unit : 0) : top - level + 1;
    return max(0, min(tiles, level <= 0 ? tiles : n));
  };
  int level = 0;
  if (t >= __reduce_add_sync(0xffffffffu, tiles)) {
    r.b = -1;
    r.tile = 0;
    return r;
  }
  for (int bit = 1 << (31 - __clz(__reduce_max_sync(0xffffffffu, top) | 1)); bit; bit >>= 1)
    if (__reduce_add_sync(0xffffffffu, at_least(level + bit)) > t) level += bit;
  // the rank among the tiles of this level, sequence by sequence
  const int more = at_least(level + 1), here = at_least(level) - more;
  const int rank = t - __reduce_add_sync(0xffffffffu, more);
  int inc = here;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  r.b = __ffs(__ballot_sync(0xffffffffu, rank < inc)) - 1;
  const int p = __shfl_sync(0xffffffffu, more + rank - (inc - here), r.b);
  r.tile = KEYS ? p : __shfl_sync(0xffffffffu, tiles, r.b) - 1 - p;
  r.q = {__shfl_sync(0xffffffffu, q.first, r.b), __shfl_sync(0xffffffffu, q.n, r.b), false};
  r.k = {__shfl_sync(0xffffffffu, k.first, r.b), __shfl_sync(0xffffffffu, k.n, r.b), false};
  return r;
}

// Whether the n_kv keys of sequence b are the rows that its weights count.
__device__ __forceinline__ bool counts_rows(const spatten_prompt_args& a, int b, int n_kv) {
  return !a.weight_len || a.weight_len[b] == min(n_kv, a.weight_cap);
}

// Reports offsets that decrease or leave their block, and keys that are not the weights' rows (one block of a
// call does it).
__device__ __forceinline__ void report_bad_offsets(const spatten_prompt_args& a) {
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    const PackedRows q = packed_rows(a.cu_q, b, a.total_q), k = packed_rows(a.cu_kv, b, a.total_kv);
    if (q.bad || k.bad || (a.weight && q.n > 0 && !counts_rows(a, b, k.n))) report(a.dev_status, SPATTEN_E_INDEX);
  }
}

int32_t prompt_simt_launch(const PromptProblem& p, cudaStream_t st);
int32_t prompt_reduce_launch(const PromptProblem& p, cudaStream_t st);   // weight += the heads' column sums
int32_t prompt_tc_launch(const PromptProblem& p, cudaStream_t st);
bool prompt_tc_supported(const spatten_prompt_args& a);
int prompt_tc_splits(const spatten_prompt_args& a);

}  // namespace spt
