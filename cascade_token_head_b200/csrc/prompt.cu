// spatten_prompt_attention: argument checks, workspace and kernel choice.
#include <cmath>

#include "attention.cuh"
#include "prompt.cuh"

namespace spt {
namespace {

int32_t validate(const spatten_prompt_args& a) {
  if (a.B < 1 || a.B > 65535 || a.H < 1 || a.H > 1024 || a.H_kv < 1) return SPATTEN_E_ARG;
  if (a.total_q < 0 || a.total_kv < 0) return SPATTEN_E_ARG;
  if (a.dtype != SPATTEN_F32 && a.dtype != SPATTEN_BF16) return SPATTEN_E_ARG;
  if (a.kernel != SPATTEN_ATTN_AUTO && a.kernel != SPATTEN_ATTN_CUDA_CORE && a.kernel != SPATTEN_ATTN_TENSOR_CORE)
    return SPATTEN_E_ARG;
  if (a.d_h != 64 && a.d_h != 128) return SPATTEN_E_UNSUPPORTED;
  if (a.H % a.H_kv != 0) return SPATTEN_E_SHAPE;
  if (!a.cu_q || !a.q || !a.k || !a.v || !a.o) return SPATTEN_E_ARG;
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

// Tensor cores wherever they can run, down to single rows.
bool use_tc(const spatten_prompt_args& a) { return a.kernel != SPATTEN_ATTN_CUDA_CORE && prompt_tc_supported(a); }

size_t layout(const spatten_prompt_args& a, void* ws, size_t ws_bytes, PromptProblem* p) {
  if (!a.weight) return 0;
  WsCursor c(ws, ws_bytes);
  const size_t rows = static_cast<size_t>(a.H) * a.total_q;
  if (use_tc(a)) {
    float* offset = c.take<float>(rows);
    float* part = a.H > a.H_kv ? c.take<float>(static_cast<size_t>(a.H) * a.total_kv) : nullptr;
    if (p) p->offset = offset, p->part = part;
  } else {
    float2* stats = c.take<float2>(rows);
    if (p) p->stats = stats;
  }
  return align_up(c.used, 256);
}

}  // namespace
}  // namespace spt

extern "C" size_t spatten_prompt_workspace_size(const spatten_prompt_args* a) {
  if (!a || a->H < 1 || a->total_q < 0 || a->total_kv < 0) return 0;
  return spt::layout(*a, nullptr, 0, nullptr);
}

extern "C" int32_t spatten_prompt_attention(const spatten_prompt_args* a, void* ws, size_t ws_bytes, void* stream) {
  spt::AbiRange nvtx_range("spatten_prompt_attention");
  using namespace spt;
  if (!a) return SPATTEN_E_ARG;
  SPT_TRY(validate(*a));
  PromptProblem p{};
  p.a = *a;
  p.wait_limit = wait_limit_setting();
  const size_t need = layout(*a, ws, ws_bytes, &p);
  if (need && (!ws || ws_bytes < need)) return SPATTEN_E_WORKSPACE;
  if (need && !aligned16(ws)) return SPATTEN_E_ALIGN;
  if (a->total_q == 0) return SPATTEN_OK;
  if (!p.a.cu_kv) p.a.cu_kv = p.a.cu_q;
  if (!(p.a.sm_scale > 0.0f)) p.a.sm_scale = 1.0f / std::sqrt(static_cast<float>(a->d_h));
  if (use_tc(*a)) return prompt_tc_launch(p, as_stream(stream));
  return prompt_simt_launch(p, as_stream(stream));
}
