// spatten_kv4_attention: one query row per sequence over the 4-bit cache, grouped heads.
#include <cmath>

#include "kv4.cuh"

namespace spt {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
  spatten_kv4_attn_args a;
  float* p;   // [B][H][n_max] scores, then probabilities
};

__device__ __forceinline__ float block_reduce(float v, bool is_max, float* sh) {
  v = is_max ? warp_max(v) : warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = sh[0];
  for (int w = 1; w < kThreads / 32; ++w) r = is_max ? fmaxf(r, sh[w]) : r + sh[w];
  return r;
}

// One block per (sequence, key/value head): scores with one thread per key, then the softmax, then
// the product with V with one thread per (channel, slice of the keys).
template <int DH, typename T>
__global__ void __launch_bounds__(kThreads) kv4_attn_kernel(AttnArgs x) {
  constexpr int G32 = DH / kKv4Group, kSlices = kThreads / DH;
  __shared__ float q[DH], sh[kThreads / 32], part[kThreads];
  const spatten_kv4_attn_args& a = x.a;
  const spatten_kv4_cache& c = a.cache;
  const int hk = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, group = a.H / c.H_kv;
  const int64_t base = (static_cast<int64_t>(b) * c.H_kv + hk) * c.cap;
  const int n = clamp_len(a.len[b], a.n_max, a.dev_status);
  for (int g = 0; g < group; ++g) {
    const int h = hk * group + g;
    float* p = x.p + (static_cast<int64_t>(b) * a.H + h) * a.n_max;
    __syncthreads();
    if (tid < DH) q[tid] = ld_as_float(static_cast<const T*>(a.q) + b * a.q_ld + static_cast<int64_t>(h) * DH + tid);
    __syncthreads();
    float mx = -INFINITY;
    for (int j = tid; j < n; j += kThreads) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(c.k_codes) + (base + j) * (DH / 8);
      float s = 0.0f;
      for (int gr = 0; gr < G32; ++gr) {
        float t = 0.0f;
        for (int o = 0; o < 4; ++o)
          for (int i = 0; i < 8; ++i)
            t = fmaf(static_cast<float>(static_cast<int>((w[o * G32 + gr] >> (4 * i)) & 15u) - 8), q[32 * gr + 8 * o + i], t);
        s = fmaf(t, bf16_bits_to_float(c.k_scale[(base + j) * G32 + gr]), s);
      }
      s *= a.sm_scale * kLog2e;
      p[j] = s;
      mx = fmaxf(mx, s);
    }
    mx = block_reduce(mx, true, sh);
    float l = 0.0f;
    for (int j = tid; j < n; j += kThreads) {
      p[j] = exp2f(p[j] - mx);
      l += p[j];
    }
    l = block_reduce(l, false, sh);
    for (int j = tid; j < n; j += kThreads) p[j] /= l;
    __syncthreads();
    const int d = tid % DH, slice = tid / DH, gr = d / 32, e = d % 32;
    float o = 0.0f;
    for (int j = slice; j < n; j += kSlices) {
      const uint16_t w = reinterpret_cast<const uint16_t*>(c.v_codes)[(base + j) * (DH / 4) + (e / 4) * G32 + gr];
      o = fmaf(p[j] * bf16_bits_to_float(c.v_scale[(base + j) * G32 + gr]),
               static_cast<float>(((w >> (4 * (e % 4))) & 15) - 8), o);
    }
    part[tid] = o;
    __syncthreads();
    if (tid < DH) {
      for (int s = 1; s < kSlices; ++s) o += part[s * DH + tid];
      st_from_float(static_cast<T*>(a.o) + b * a.o_ld + static_cast<int64_t>(h) * DH + tid, o);
    }
  }
  if (!a.update_weight) return;
  __syncthreads();
  const float* p = x.p + (static_cast<int64_t>(b) * a.H + static_cast<int64_t>(hk) * group) * a.n_max;
  for (int j = tid; j < n; j += kThreads) {
    float t = 0.0f;
    for (int g = 0; g < group; ++g) t += p[static_cast<int64_t>(g) * a.n_max + j];
    c.weight[base + j] += t;
  }
}

int32_t validate(const spatten_kv4_attn_args& a) {
  SPT_TRY(kv4_validate(a.cache));
  if (a.H < 1 || a.H > 1024) return SPATTEN_E_ARG;
  if (a.H % a.cache.H_kv != 0) return SPATTEN_E_SHAPE;
  if (!a.q || !a.o || !a.len) return SPATTEN_E_ARG;
  if (a.dtype != SPATTEN_F32 && a.dtype != SPATTEN_BF16) return SPATTEN_E_ARG;
  if (a.n_max < 1) return SPATTEN_E_ARG;
  if (a.n_max > a.cache.cap) return SPATTEN_E_SHAPE;
  if (a.update_weight && !a.cache.weight) return SPATTEN_E_ARG;
  const int64_t hd = static_cast<int64_t>(a.H) * a.cache.d_h;
  if (a.q_ld < hd || a.o_ld < hd) return SPATTEN_E_SHAPE;
  const int esz = a.dtype == SPATTEN_BF16 ? 2 : 4;
  if (!aligned16(a.q) || !aligned16(a.o) || (a.q_ld * esz) % 16 != 0 || (a.o_ld * esz) % 16 != 0)
    return SPATTEN_E_ALIGN;
  return SPATTEN_OK;
}

size_t layout(const spatten_kv4_attn_args& a, void* ws, size_t ws_bytes, AttnArgs* x) {
  WsCursor c(ws, ws_bytes);
  float* p = c.take<float>(static_cast<size_t>(a.cache.B) * a.H * a.n_max);
  if (x) x->p = p;
  return align_up(c.used, 256);
}

}  // namespace
}  // namespace spt

extern "C" size_t spatten_kv4_attention_workspace_size(const spatten_kv4_attn_args* a) {
  if (!a || spt::validate(*a) != SPATTEN_OK) return 0;
  return spt::layout(*a, nullptr, 0, nullptr);
}

extern "C" int32_t spatten_kv4_attention(const spatten_kv4_attn_args* a, void* ws, size_t ws_bytes, void* stream) {
  spt::AbiRange nvtx_range("spatten_kv4_attention");
  using namespace spt;
  if (!a) return SPATTEN_E_ARG;
  SPT_TRY(validate(*a));
  AttnArgs x{*a, nullptr};
  const size_t need = layout(*a, ws, ws_bytes, &x);
  if (!ws || ws_bytes < need) return SPATTEN_E_WORKSPACE;
  if (!aligned16(ws)) return SPATTEN_E_ALIGN;
  if (!(x.a.sm_scale > 0.0f)) x.a.sm_scale = 1.0f / std::sqrt(static_cast<float>(a->cache.d_h));
  cudaStream_t st = as_stream(stream);
  const dim3 grid(a->cache.H_kv, a->cache.B);
  const bool bf = a->dtype == SPATTEN_BF16;
  if (a->cache.d_h == 64) {
    if (bf) kv4_attn_kernel<64, __nv_bfloat16><<<grid, kThreads, 0, st>>>(x);
    else kv4_attn_kernel<64, float><<<grid, kThreads, 0, st>>>(x);
  } else {
    if (bf) kv4_attn_kernel<128, __nv_bfloat16><<<grid, kThreads, 0, st>>>(x);
    else kv4_attn_kernel<128, float><<<grid, kThreads, 0, st>>>(x);
  }
  return launch_status();
}
