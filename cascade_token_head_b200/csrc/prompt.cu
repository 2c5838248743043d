// spatten_prompt_attention: argument checks, workspace and kernel choice.
#include <algorithm>
#include <cmath>

#include "attention.cuh"
#include "prompt.cuh"

namespace spt {
namespace {

// A poll may block for some microseconds, so this many are a few seconds.
constexpr uint32_t kPromptWaitLimit = 1u << 20;

int32_t validate(const spatten_prompt_args& a) {
  if (a.B < 1 || a.B > 65535 || a.H < 1 || a.H > 1024 || a.H_kv < 1) return SPATTEN_E_ARG;
  if (a.total_q < 0 || a.total_kv < 0) return SPATTEN_E_ARG;
  if (a.dtype != SPATTEN_F32 && a.dtype != SPATTEN_BF16) return SPATTEN_E_ARG;
  if (a.kernel != SPATTEN_ATTN_AUTO && a.kernel != SPATTEN_ATTN_CUDA_CORE && a.kernel != SPATTEN_ATTN_TENSOR_CORE)
    return SPATTEN_E_ARG;
  if (a.d_h != 64 && a.d_h != 128) return SPATTEN_E_UNSUPPORTED;
  if (a.H % a.H_kv != 0) return SPATTEN_E_SHAPE;
  if (!a.cu_q || (a.total_q > 0 && (!a.q || !a.o)) || (a.total_kv > 0 && (!a.k || !a.v))) return SPATTEN_E_ARG;
  if (!a.cu_kv && a.total_q != a.total_kv) return SPATTEN_E_SHAPE;
  const int64_t hd = static_cast<int64_t>(a.H) * a.d_h, hkd = static_cast<int64_t>(a.H_kv) * a.d_h;
  if (a.q_ld_tok < hd || a.o_ld_tok < hd || a.kv_ld_tok < hkd) return SPATTEN_E_SHAPE;
  if (a.weight && (a.weight_cap < 1 || a.weight_ld_head < a.weight_cap || a.weight_ld_seq < a.weight_cap))
    return SPATTEN_E_SHAPE;
  const int esz = a.dtype == SPATTEN_BF16 ? 2 : 4;
  if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.o) || (a.q_ld_tok * esz) % 16 != 0 ||
      (a.kv_ld_tok * esz) % 16 != 0 || (a.o_ld_tok * esz) % 16 != 0)
    return SPATTEN_E_ALIGN;
  if (a.kernel == SPATTEN_ATTN_TENSOR_CORE && a.dtype != SPATTEN_BF16) return SPATTEN_E_UNSUPPORTED;
  return SPATTEN_OK;
}

// Tensor cores wherever they can run, down to single rows (float32: 16 prompts of 512, 16 heads of 64, 163 against
// 570 us; 77 to 512 rows of 128 behind 1000 others, 145 against 603).
bool use_tc(const spatten_prompt_args& a) { return a.kernel != SPATTEN_ATTN_CUDA_CORE && prompt_tc_supported(a); }

size_t layout(const spatten_prompt_args& a, void* ws, size_t ws_bytes, PromptProblem* p) {
  const bool tc = use_tc(a);
  const bool split = tc && a.dtype == SPATTEN_F32 && a.total_q > 0;
  const int splits = tc && a.total_q > 0 ? prompt_tc_splits(a) : 1;
  if (!a.weight && !split && splits == 1) return 0;
  WsCursor c(ws, ws_bytes);
  uint16_t* planes[3] = {};
  if (split)
    for (int t = 0; t < 3; ++t)
      planes[t] = c.take<uint16_t>(3 * static_cast<size_t>(t == 0 ? a.total_q : a.total_kv) * (t == 0 ? a.H : a.H_kv) * a.d_h);
  const size_t rows = a.weight ? static_cast<size_t>(a.H) * a.total_q : 0;
  float* offset = a.weight && tc ? c.take<float>(rows) : nullptr;
  float2* stats = a.weight && !tc ? c.take<float2>(rows) : nullptr;
  float* part = a.weight && a.H > a.H_kv ? c.take<float>(static_cast<size_t>(a.H) * a.total_kv) : nullptr;
  const size_t parts = splits > 1 ? static_cast<size_t>(splits) * a.H * a.total_q : 0;
  float2* split_ml = parts ? c.take<float2>(parts) : nullptr;
  float* split_o = parts ? c.take<float>(parts * a.d_h) : nullptr;
  if (p) {
    for (int t = 0; t < 3; ++t) p->planes[t] = planes[t];
    p->splits = splits, p->split_ml = split_ml, p->split_o = split_o;
    p->offset = offset, p->stats = stats, p->part = part;
  }
  return align_up(c.used, 256);
}

// weight += the sums of a group's heads, in head order; blockIdx.y = key/value head
__global__ void __launch_bounds__(256) prompt_weight_reduce_kernel(PromptProblem p) {
  grid_dep_trigger();
  grid_dep_wait();
  const spatten_prompt_args& a = p.a;
  const int r = blockIdx.x * 256 + threadIdx.x, hk = blockIdx.y, G = a.H / a.H_kv;
  const int b = owner_of_lanes_row(a.cu_kv, a.B, a.total_kv, r);
  if (b < 0) return;
  const int first = a.cu_kv[b], j = r - first;
  if (!counts_rows(a, b, a.cu_kv[b + 1] - first)) return;
  if (j >= a.weight_cap) {
    report(a.dev_status, SPATTEN_E_INDEX);
    return;
  }
  const float* part = p.part + static_cast<int64_t>(hk) * G * a.total_kv + r;
  float sum = 0.0f;
  for (int g = 0; g < G; ++g) sum += part[static_cast<int64_t>(g) * a.total_kv];
  a.weight[static_cast<int64_t>(b) * a.weight_ld_seq + static_cast<int64_t>(hk) * a.weight_ld_head + j] += sum;
}

}  // namespace

int32_t prompt_reduce_launch(const PromptProblem& p, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(ceil_div(p.a.total_kv, 256)), p.a.H_kv);
  return launch_chained(prompt_weight_reduce_kernel, grid, dim3(256), 0, st, 1, p);
}

}  // namespace spt

extern "C" size_t spatten_prompt_workspace_size(const spatten_prompt_args* a) {
  if (!a || a->H < 1 || a->H_kv < 1 || a->d_h < 1 || a->total_q < 0 || a->total_kv < 0) return 0;
  return spt::layout(*a, nullptr, 0, nullptr);
}

extern "C" int32_t spatten_prompt_attention(const spatten_prompt_args* a, void* ws, size_t ws_bytes, void* stream) {
  spt::AbiRange nvtx_range("spatten_prompt_attention");
  using namespace spt;
  if (!a) return SPATTEN_E_ARG;
  SPT_TRY(validate(*a));
  PromptProblem p{};
  p.a = *a;
  p.wait_limit = std::min(wait_limit_setting(), kPromptWaitLimit);
  p.splits = 1;
  const size_t need = layout(*a, ws, ws_bytes, &p);
  if (need && (!ws || ws_bytes < need)) return SPATTEN_E_WORKSPACE;
  if (need && !aligned16(ws)) return SPATTEN_E_ALIGN;
  if (a->total_q == 0) return SPATTEN_OK;
  if (!p.a.cu_kv) p.a.cu_kv = p.a.cu_q;
  if (!(p.a.sm_scale > 0.0f)) p.a.sm_scale = 1.0f / std::sqrt(static_cast<float>(a->d_h));
  if (use_tc(*a)) return prompt_tc_launch(p, as_stream(stream));
  return prompt_simt_launch(p, as_stream(stream));
}
