// Prompt attention on CUDA cores in float32 arithmetic: the float32 configuration, and the on-device
// cross-check of the tensor-core kernel.
//
// Output kernel: a block owns 64 query rows of one head and walks the visible keys in tiles of 64 with the
// running maximum and sum of the softmax.  Thread (ty, tx) of 16 x 16 computes the scores of rows
// 4 ty .. + 3 with keys 4 tx .. + 3 from channel-major tiles (two 16-byte reads of shared memory for 16
// multiply-adds), passes its P through shared memory, and owns the rows' channels 4 tx .. + 3 (and, of 128,
// 64 more on) of the product with V.  Weight kernel: a block owns 64 keys of one query head and walks the
// tiles of rows that see them, with the statistics of the first kernel; a thread sums its keys over its
// rows, the block over its threads in a fixed order.  Bound by the multiply-adds and their operands' reads
// when long, by the chain of tiles when short.
#include "prompt.cuh"

namespace spt {
namespace {

constexpr int kThreads = 256, kTile = 64, kLd = kTile + 4;   // rows and keys of a tile; row length of transposed tiles
constexpr float kLog2e = 1.4426950408889634f;

template <int DH>
struct PromptSmem {
  float q[DH][kLd];      // channel-major
  float k[DH][kLd];
  float v[kTile][DH];
  float p[kTile][kLd];   // key-major
};

// Rows of a packed block into shared memory, channel-major; rows from n on are zero.  Lanes take different
// rows, so that their stores fall into different banks.
template <int DH, typename T>
__device__ __forceinline__ void load_channels(float (*dst)[kLd], const void* base, int64_t ld_tok, int h, int64_t r0, int n) {
#pragma unroll 4
  for (int e = threadIdx.x; e < kTile * (DH / 8); e += kThreads) {
    const int r = e % kTile, c = e / kTile;
    float f[8] = {};
    if (r < n) load8(static_cast<const T*>(base) + (r0 + r) * ld_tok + static_cast<int64_t>(h) * DH + c * 8, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[c * 8 + i][r] = f[i];
  }
}
template <int DH, typename T>
__device__ __forceinline__ void load_rows(float (*dst)[DH], const void* base, int64_t ld_tok, int h, int64_t r0, int n) {
#pragma unroll 4
  for (int e = threadIdx.x; e < kTile * (DH / 8); e += kThreads) {
    const int r = e / (DH / 8), c = e % (DH / 8);
    float f[8] = {};
    if (r < n) load8(static_cast<const T*>(base) + (r0 + r) * ld_tok + static_cast<int64_t>(h) * DH + c * 8, f);
    *reinterpret_cast<float4*>(&dst[r][c * 8]) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(&dst[r][c * 8 + 4]) = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// s[i][j]: scores of row 4 ty + i with key 4 tx + j
template <int DH>
__device__ __forceinline__ void scores(const PromptSmem<DH>& sm, int ty, int tx, float (*s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
#pragma unroll 8
  for (int d = 0; d < DH; ++d) {
    const float4 a = *reinterpret_cast<const float4*>(&sm.q[d][4 * ty]), b = *reinterpret_cast<const float4*>(&sm.k[d][4 * tx]);
    const float q[4] = {a.x, a.y, a.z, a.w}, k[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = fmaf(q[i], k[j], s[i][j]);
  }
}

// over the 16 threads of a row
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int DH, typename T>
__global__ void __launch_bounds__(kThreads) prompt_simt_kernel(PromptProblem p) {
  grid_dep_trigger();
  grid_dep_wait();
  extern __shared__ __align__(16) char smem_raw[];
  PromptSmem<DH>& sm = *reinterpret_cast<PromptSmem<DH>*>(smem_raw);
  constexpr int kC = DH / 64;   // groups of four channels per thread
  const spatten_prompt_args& a = p.a;
  const int h = blockIdx.x % a.H, hk = h / (a.H / a.H_kv), ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  if (blockIdx.x == 0) report_bad_offsets(a);
  const SeqTile st = find_seq_tile(a.cu_q, a.B, a.total_q, kTile, blockIdx.x / a.H);
  if (st.b < 0) return;
  const PackedRows qr = packed_rows(a.cu_q, st.b, a.total_q), kr = packed_rows(a.cu_kv, st.b, a.total_kv);
  const int i0 = st.tile * kTile, rows = min(kTile, qr.n - i0), shift = kr.n - qr.n;
  load_channels<DH, T>(sm.q, a.q, a.q_ld_tok, h, static_cast<int64_t>(qr.first) + i0, rows);
  const float scale = a.sm_scale * kLog2e;
  float m[4], l[4], o[4][kC][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.0f;
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][c][k] = 0.0f;
  }
  const int n_vis = min(kr.n, i0 + rows + shift);   // keys that the last row sees
  for (int j0 = 0; j0 < n_vis; j0 += kTile) {
    __syncthreads();
    load_channels<DH, T>(sm.k, a.k, a.kv_ld_tok, hk, static_cast<int64_t>(kr.first) + j0, min(kTile, kr.n - j0));
    load_rows<DH, T>(sm.v, a.v, a.kv_ld_tok, hk, static_cast<int64_t>(kr.first) + j0, min(kTile, kr.n - j0));
    __syncthreads();
    float s[4][4];
    scores<DH>(sm, ty, tx, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int last = min(i0 + 4 * ty + i + shift, kr.n - 1) - j0;   // the last key of the tile that the row sees
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = 4 * tx + j <= last ? s[i][j] * scale : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      mx = fmaxf(m[i], row_max(mx));
      const float base = mx == -INFINITY ? 0.0f : mx;
      const float f = exp2f(m[i] - base);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = exp2f(s[i][j] - base);
        sum += s[i][j];
      }
      l[i] = l[i] * f + row_sum(sum);
      m[i] = mx;
#pragma unroll
      for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][c][k] *= f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4*>(&sm.p[4 * tx + j][4 * ty]) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
    __syncwarp();   // a row's 16 threads are lanes of one warp
    const int keys = min(kTile, n_vis - j0);
#pragma unroll 4
    for (int j = 0; j < keys; ++j) {
      const float4 w = *reinterpret_cast<const float4*>(&sm.p[j][4 * ty]);
      const float pw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const float4 u = *reinterpret_cast<const float4*>(&sm.v[j][64 * c + 4 * tx]);
        const float v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i][c][k] = fmaf(pw[i], v[k], o[i][c][k]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (4 * ty + i >= rows) break;
    const int64_t row = static_cast<int64_t>(qr.first) + i0 + 4 * ty + i;
    const float inv = l[i] > 0.0f ? 1.0f / l[i] : (l[i] == 0.0f ? 0.0f : l[i]);   // NaN stays NaN
    T* dst = static_cast<T*>(a.o) + row * a.o_ld_tok + static_cast<int64_t>(h) * DH + 4 * tx;
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) st_from_float(dst + 64 * c + k, o[i][c][k] * inv);
    if (p.stats && tx == 0) p.stats[static_cast<int64_t>(h) * a.total_q + row] = make_float2(m[i] == -INFINITY ? 0.0f : m[i], inv);
  }
}

template <int DH, typename T>
__global__ void __launch_bounds__(kThreads) prompt_weight_simt_kernel(PromptProblem p) {
  grid_dep_trigger();
  grid_dep_wait();
  extern __shared__ __align__(16) char smem_raw[];
  PromptSmem<DH>& sm = *reinterpret_cast<PromptSmem<DH>*>(smem_raw);
  const spatten_prompt_args& a = p.a;
  const int h = blockIdx.x % a.H, G = a.H / a.H_kv, hk = h / G, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const SeqTile st = find_seq_tile<true>(a.cu_kv, a.B, a.total_kv, kTile, blockIdx.x / a.H);
  if (st.b < 0) return;
  const PackedRows qr = packed_rows(a.cu_q, st.b, a.total_q), kr = packed_rows(a.cu_kv, st.b, a.total_kv);
  const int j0 = st.tile * kTile, shift = kr.n - qr.n;
  const bool counted = counts_rows(a, st.b, kr.n);
  load_channels<DH, T>(sm.k, a.k, a.kv_ld_tok, hk, static_cast<int64_t>(kr.first) + j0, min(kTile, kr.n - j0));
  const float scale = a.sm_scale * kLog2e;
  const float2* stats = p.stats + static_cast<int64_t>(h) * a.total_q + qr.first;
  float sum[4] = {};
  // from the first tile of rows that sees the tile's first key
  for (int i0 = max(0, j0 - shift) / kTile * kTile; i0 < qr.n; i0 += kTile) {
    float2 ml[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ml[i] = i0 + 4 * ty + i < qr.n ? stats[i0 + 4 * ty + i] : make_float2(0.0f, 0.0f);
    __syncthreads();
    load_channels<DH, T>(sm.q, a.q, a.q_ld_tok, h, static_cast<int64_t>(qr.first) + i0, min(kTile, qr.n - i0));
    __syncthreads();
    float s[4][4];
    scores<DH>(sm, ty, tx, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i0 + 4 * ty + i, last = row < qr.n ? row + shift - j0 : -1;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * tx + j <= last) sum[j] = fmaf(exp2f(fmaf(s[i][j], scale, -ml[i].x)), ml[i].y, sum[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) sm.p[4 * tx + j][ty] = sum[j];
  __syncthreads();
  const int j = threadIdx.x;
  if (j >= kTile || j0 + j >= kr.n) return;
  float t = 0.0f;
#pragma unroll
  for (int y = 0; y < 16; ++y) t += sm.p[j][y];
  if (G > 1)
    p.part[static_cast<int64_t>(h) * a.total_kv + kr.first + j0 + j] = t;
  else if (!counted)
    return;
  else if (j0 + j < a.weight_cap)
    a.weight[static_cast<int64_t>(st.b) * a.weight_ld_seq + static_cast<int64_t>(hk) * a.weight_ld_head + j0 + j] += t;
  else
    report(a.dev_status, SPATTEN_E_INDEX);
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
  const int64_t q_blocks = (static_cast<int64_t>(a.total_q) / kTile + a.B) * a.H;
  const int64_t k_blocks = (static_cast<int64_t>(a.total_kv) / kTile + a.B) * a.H;
  if (q_blocks > INT32_MAX || k_blocks > INT32_MAX) return SPATTEN_E_UNSUPPORTED;
  SPT_TRY(launch_chained(prompt_simt_kernel<DH, T>, dim3(static_cast<unsigned>(q_blocks)), dim3(kThreads), bytes, st, 1, p));
  if (!a.weight || a.total_kv == 0) return SPATTEN_OK;
  SPT_TRY(launch_chained(prompt_weight_simt_kernel<DH, T>, dim3(static_cast<unsigned>(k_blocks)), dim3(kThreads), bytes, st, 1, p));
  return a.H == a.H_kv ? SPATTEN_OK : prompt_reduce_launch(p, st);
}

}  // namespace

int32_t prompt_simt_launch(const PromptProblem& p, cudaStream_t st) {
  if (p.a.d_h == 64)
    return p.a.dtype == SPATTEN_BF16 ? launch<64, __nv_bfloat16>(p, st) : launch<64, float>(p, st);
  return p.a.dtype == SPATTEN_BF16 ? launch<128, __nv_bfloat16>(p, st) : launch<128, float>(p, st);
}

}  // namespace spt
