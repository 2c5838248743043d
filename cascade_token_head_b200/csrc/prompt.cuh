// Prompt attention (causal, packed sequences, grouped heads): what its kernels share.
#pragma once

#include "kv4.cuh"

namespace spt {

struct PromptProblem {
  spatten_prompt_args a;   // sm_scale > 0 and cu_kv set
  // with weights only (else NULL).  CUDA cores: [H][total_q] score maximum (log2 units) and exponential
  // sum of each row.  Tensor cores: [H][total_q] what each row's scores need added (before the softmax
  // scale) for their exponentials to be P, and [H][total_kv] the heads' column sums (grouped heads).
  float2* stats;
  float* offset;
  float* part;
  uint32_t wait_limit;     // polls of one pipeline wait (tensor-core kernels)
};

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
