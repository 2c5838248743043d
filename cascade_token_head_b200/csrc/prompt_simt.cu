// Prompt attention on CUDA cores in float32 arithmetic: the float32 configuration, and the on-device
// cross-check of the tensor-core kernel.
//
// Output kernel: a block owns 32 query rows of one head (4 per warp) and walks the visible keys in
// tiles of 32, one key per lane, with the running maximum and sum of the softmax; P goes through
// shared memory to the product with V, where lanes own channels.  Weight kernel: a block owns 32 keys
// of one key/value head and walks the rows that see them, with the statistics of the first kernel;
// lanes own keys, so the column sums need no exchange but a fixed-order sum over the 8 warps.
#include "prompt.cuh"

namespace spt {
namespace {

constexpr int kThreads = 256, kWarps = 8, kRows = 32, kKeys = 32, kRowsPerWarp = 4;
constexpr float kLog2e = 1.4426950408889634f;

template <int DH>
struct PromptSmem {
  float q[kRows][DH];
  float k[kKeys][DH + 1];
  float v[kKeys][DH + 1];
  float4 p[kWarps][kKeys];   // the warp's four rows of P for each key; column sums at the end
};

// rows r0 .. r0+31 of a packed block, head h, into shared memory; rows from `end` on are zero
template <int DH, int LD, typename T>
__device__ __forceinline__ void load_rows(float (*dst)[LD], const void* base, int64_t ld_tok, int h, int64_t r0, int n) {
  for (int e = threadIdx.x; e < kRows * (DH / 8); e += kThreads) {
    const int r = e / (DH / 8), c = e % (DH / 8);
    float f[8] = {};
    if (r < n) load8(static_cast<const T*>(base) + (r0 + r) * ld_tok + static_cast<int64_t>(h) * DH + c * 8, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[r][c * 8 + i] = f[i];
  }
}

// scores of the warp's four rows with the lane's key
template <int DH>
__device__ __forceinline__ void scores4(const PromptSmem<DH>& sm, int warp, int lane, float* s) {
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) s[r] = 0.0f;
#pragma unroll 4
  for (int d = 0; d < DH; d += 4) {
    float kk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) kk[i] = sm.k[lane][d + i];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
      const float4 q = *reinterpret_cast<const float4*>(&sm.q[warp * kRowsPerWarp + r][d]);
      s[r] = fmaf(q.x, kk[0], s[r]);
      s[r] = fmaf(q.y, kk[1], s[r]);
      s[r] = fmaf(q.z, kk[2], s[r]);
      s[r] = fmaf(q.w, kk[3], s[r]);
    }
  }
}

template <int DH, typename T>
__global__ void __launch_bounds__(kThreads) prompt_simt_kernel(PromptProblem p) {
  grid_dep_trigger();
  grid_dep_wait();
  extern __shared__ __align__(16) char smem_raw[];
  PromptSmem<DH>& sm = *reinterpret_cast<PromptSmem<DH>*>(smem_raw);
  constexpr int kC = DH / 32;   // channels per lane
  const spatten_prompt_args& a = p.a;
  const int h = blockIdx.x % a.H, hk = h / (a.H / a.H_kv), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0) report_bad_offsets(a);
  const SeqTile st = find_seq_tile(a.cu_q, a.B, a.total_q, kRows, blockIdx.x / a.H);
  if (st.b < 0) return;
  const PackedRows qr = packed_rows(a.cu_q, st.b, a.total_q), kr = packed_rows(a.cu_kv, st.b, a.total_kv);
  const int i0 = st.tile * kRows, rows = min(kRows, qr.n - i0), shift = kr.n - qr.n;
  load_rows<DH, DH, T>(sm.q, a.q, a.q_ld_tok, h, qr.first + i0, rows);
  const float scale = a.sm_scale * kLog2e;
  float m[kRowsPerWarp], l[kRowsPerWarp], o[kRowsPerWarp][kC];
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.0f;
#pragma unroll
    for (int c = 0; c < kC; ++c) o[r][c] = 0.0f;
  }
  const int n_vis = min(kr.n, i0 + rows + shift);   // keys that the last row sees
  for (int j0 = 0; j0 < n_vis; j0 += kKeys) {
    __syncthreads();
    load_rows<DH, DH + 1, T>(sm.k, a.k, a.kv_ld_tok, hk, static_cast<int64_t>(kr.first) + j0, min(kKeys, kr.n - j0));
    load_rows<DH, DH + 1, T>(sm.v, a.v, a.kv_ld_tok, hk, static_cast<int64_t>(kr.first) + j0, min(kKeys, kr.n - j0));
    __syncthreads();
    float s[kRowsPerWarp];
    scores4<DH>(sm, warp, lane, s);
    float pr[kRowsPerWarp];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
      const int i = i0 + warp * kRowsPerWarp + r, j = j0 + lane;
      const bool seen = j <= i + shift && j < kr.n;
      const float x = seen ? s[r] * scale : -INFINITY;
      const float mx = fmaxf(m[r], warp_max(x));
      const float base = mx == -INFINITY ? 0.0f : mx;
      const float f = exp2f(m[r] - base);
      pr[r] = exp2f(x - base);
      l[r] = l[r] * f + warp_sum(pr[r]);
      m[r] = mx;
#pragma unroll
      for (int c = 0; c < kC; ++c) o[r][c] *= f;
    }
    sm.p[warp][lane] = make_float4(pr[0], pr[1], pr[2], pr[3]);
    __syncwarp();
#pragma unroll 4
    for (int j = 0; j < kKeys; ++j) {
      const float4 w = sm.p[warp][j];
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const float v = sm.v[j][lane + 32 * c];
        o[0][c] = fmaf(w.x, v, o[0][c]);
        o[1][c] = fmaf(w.y, v, o[1][c]);
        o[2][c] = fmaf(w.z, v, o[2][c]);
        o[3][c] = fmaf(w.w, v, o[3][c]);
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) {
    const int i = warp * kRowsPerWarp + r;
    if (i >= rows) break;
    const int64_t row = qr.first + i0 + i;
    const float inv = l[r] > 0.0f ? 1.0f / l[r] : (l[r] == 0.0f ? 0.0f : l[r]);   // NaN stays NaN
    T* dst = static_cast<T*>(a.o) + row * a.o_ld_tok + static_cast<int64_t>(h) * DH;
#pragma unroll
    for (int c = 0; c < kC; ++c) st_from_float(dst + lane + 32 * c, o[r][c] * inv);
    if (p.stats && lane == 0) p.stats[static_cast<int64_t>(h) * a.total_q + row] = make_float2(m[r], l[r]);
  }
}

template <int DH, typename T>
__global__ void __launch_bounds__(kThreads) prompt_weight_simt_kernel(PromptProblem p) {
  grid_dep_trigger();
  grid_dep_wait();
  extern __shared__ __align__(16) char smem_raw[];
  PromptSmem<DH>& sm = *reinterpret_cast<PromptSmem<DH>*>(smem_raw);
  const spatten_prompt_args& a = p.a;
  const int hk = blockIdx.x % a.H_kv, G = a.H / a.H_kv, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeqTile st = find_seq_tile(a.cu_kv, a.B, a.total_kv, kKeys, blockIdx.x / a.H_kv);
  if (st.b < 0) return;
  const PackedRows qr = packed_rows(a.cu_q, st.b, a.total_q), kr = packed_rows(a.cu_kv, st.b, a.total_kv);
  const int j0 = st.tile * kKeys, j = j0 + lane, shift = kr.n - qr.n;
  load_rows<DH, DH + 1, T>(sm.k, a.k, a.kv_ld_tok, hk, static_cast<int64_t>(kr.first) + j0, min(kKeys, kr.n - j0));
  const float scale = a.sm_scale * kLog2e;
  float sum = 0.0f;
  // the first tile of rows that sees the tile's first key
  const int i_first = max(0, j0 - shift) / kRows * kRows;
  for (int g = 0; g < G; ++g) {
    const int h = hk * G + g;
    const float2* stats = p.stats + static_cast<int64_t>(h) * a.total_q + qr.first;
    for (int i0 = i_first; i0 < qr.n; i0 += kRows) {
      __syncthreads();
      load_rows<DH, DH, T>(sm.q, a.q, a.q_ld_tok, h, static_cast<int64_t>(qr.first) + i0, min(kRows, qr.n - i0));
      __syncthreads();
      float s[kRowsPerWarp];
      scores4<DH>(sm, warp, lane, s);
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; ++r) {
        const int i = i0 + warp * kRowsPerWarp + r;
        if (i < qr.n && j <= i + shift) {
          const float2 ml = stats[i];
          sum += exp2f(s[r] * scale - ml.x) / ml.y;
        }
      }
    }
  }
  float* part = reinterpret_cast<float*>(sm.p);
  part[warp * kKeys + lane] = sum;
  __syncthreads();
  if (warp == 0 && j < kr.n) {
    float t = 0.0f;
    for (int w = 0; w < kWarps; ++w) t += part[w * kKeys + lane];
    if (j < a.weight_cap)
      a.weight[static_cast<int64_t>(st.b) * a.weight_ld_seq + static_cast<int64_t>(hk) * a.weight_ld_head + j] += t;
    else
      report(a.dev_status, SPATTEN_E_INDEX);
  }
}

template <int DH, typename T>
int32_t launch(const PromptProblem& p, cudaStream_t st) {
  static DeviceOnce once;
  int dev;
  const int bytes = static_cast<int>(sizeof(PromptSmem<DH>));
  SPT_TRY(once_per_device(once, &dev, [&](int) -> int32_t {
    SPT_CUDA(cudaFuncSetAttribute(prompt_simt_kernel<DH, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    SPT_CUDA(cudaFuncSetAttribute(prompt_weight_simt_kernel<DH, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    return SPATTEN_OK;
  }));
  const spatten_prompt_args& a = p.a;
  // a sequence's rows end in at most one partial tile, so this many tiles cover any offsets
  const int64_t q_tiles = a.total_q / kRows + a.B, k_tiles = a.total_kv / kKeys + a.B;
  if (q_tiles * a.H > INT32_MAX || k_tiles * a.H_kv > INT32_MAX) return SPATTEN_E_UNSUPPORTED;
  SPT_TRY(launch_chained(prompt_simt_kernel<DH, T>, dim3(static_cast<unsigned>(q_tiles * a.H)), dim3(kThreads), bytes, st, 1, p));
  if (!a.weight || a.total_kv == 0) return SPATTEN_OK;
  return launch_chained(prompt_weight_simt_kernel<DH, T>, dim3(static_cast<unsigned>(k_tiles * a.H_kv)), dim3(kThreads), bytes, st, 1, p);
}

}  // namespace

int32_t prompt_simt_launch(const PromptProblem& p, cudaStream_t st) {
  if (p.a.d_h == 64)
    return p.a.dtype == SPATTEN_BF16 ? launch<64, __nv_bfloat16>(p, st) : launch<64, float>(p, st);
  return p.a.dtype == SPATTEN_BF16 ? launch<128, __nv_bfloat16>(p, st) : launch<128, float>(p, st);
}

}  // namespace spt
