// spatten_kv4_attention: one query row per sequence over the 4-bit cache, grouped heads.
//
// A cluster of C CTAs owns one (sequence, key/value head); each CTA takes a run of its keys, each warp
// tiles of TK keys, copied asynchronously into a ring of its own (no barriers in the loop).  The products
// run on mma.sync m16n8k16 with the codes as the 16-row operand and up to 8 heads as the 8 columns:
//   scores   S^T[16 keys][8 heads] = codes . q, one accumulator per group of 32 channels, which the
//            group's scale then multiplies (so the codes enter exactly).  A nibble u = code + 8 in the
//            low bits of a half is the subnormal u 2^-24, one place higher 16 u 2^-24: no conversion
//            beyond the masks; the 16 is taken out of q, and the 8 enters as the accumulator's start,
//            -8 sum(q).  q is scaled by a power of two to a maximum in [2^13, 2^14) and rounded to fp16
//            (bfloat16 queries: exact down to 2^-27 of the maximum), float32 queries as the sum of two.
//   output   O^T[16 channels][8 heads] += codes . P', P' = exp(S - m) times the key's scale of the
//            group, rounded to bfloat16 (its range is that of the scales) for bfloat16 queries and
//            held as the sum of three bfloat16 (24 bits) for float32 ones; movmatrix turns P' from the
//            score layout into the operand's.  Codes become bfloat16 as 128 + u - 136, exact.
// The tensor path is the register one since its operands are made in registers: a tcgen05 operand would
// have to go through shared memory first, and the kernel is bound by memory and by the unpacking, not
// by the products.
// Scores stay in shared memory (in the workspace when they do not fit), so that the weights need only
// one more exponential per score once the cluster has exchanged its maxima and sums.  Sums are float32
// in a fixed order.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "kv4.cuh"

namespace cg = cooperative_groups;

namespace spt {
namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kStages = 4;             // tiles in a warp's ring
constexpr int kStageBytes = 2304;      // 1024 + 1024 bytes of codes, 128 + 128 of scales
constexpr int kMaxHeads = 16;          // heads of a group per pass over the keys
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.0f;       // growth of a maximum (log2) that makes the sums be rescaled
constexpr int kRing = kWarps * kStages * kStageBytes;

// shared memory left for scores: with two CTAs on an SM, and with one (an SM has 228 KB, 1 KB of it per
// CTA reserved; the CTA's other arrays take up to 10 KB)
constexpr size_t kSharedTwo = 227 * 1024 / 2 - kRing - 11 * 1024, kSharedOne = 227 * 1024 - kRing - 11 * 1024;

template <int DH> constexpr int kTileKeys = 2048 / DH;

struct AttnArgs {
  spatten_kv4_attn_args a;
  float* x;         // ws [B][H_kv][C][heads][x_ld] scores, or NULL: in shared memory
  int32_t x_ld;     // floats between the heads' scores of one CTA's keys
  int32_t heads;    // min(H / H_kv, kMaxHeads)
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? BYTES : 0;   // 0 bytes read: the destination is zero-filled
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 half_pair(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two nibbles (bits 0-3 and 16-19 of w) as the bfloat16 pair of their codes
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  const uint32_t u = (w & 0x000f000fu) | 0x43004300u;   // 128 + u: exact in bfloat16's 8 bits
  const __nv_bfloat162 off = __halves2bfloat162(__float2bfloat16_rn(-136.0f), __float2bfloat16_rn(-136.0f));
  const __nv_bfloat162 r = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&u), off);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Where row r of a tile of V codes lies in its stage: with the rows of a quad's four lanes (2t, or
// 2t + 1) in neighbouring slots, and at 128 channels 32 bytes apart in every other pair of slots, a warp's
// reads of V take every bank once.
__device__ __forceinline__ int v_slot(int r) { return (r & ~7) | ((r & 1) << 2) | ((r >> 1) & 3); }
template <int DH>
__device__ __forceinline__ int v_offset(int r, int byte) {
  const int s = v_slot(r);
  return s * (DH / 2) + (DH == 128 ? byte ^ ((s & 2) << 4) : byte);
}

// NH: columns of 8 heads per pass; T: type of q and o
template <int DH, int NH, typename T>
struct Warp {
  static constexpr int TK = kTileKeys<DH>, G32 = DH / kKv4Group;
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int kQ = kF32 ? 2 : 1;   // terms of a query
  static constexpr int kP = kF32 ? 3 : 1;   // terms of a P'
  uint32_t q[NH][kQ][G32][2][2];            // B operand of the scores
  float start[NH][G32][2], scale[NH][2];    // accumulators' start, factor to log2 units (heads 2t, 2t + 1)
  float o[NH][DH / 16][4];
  float m[NH][2], nb[NH][2], l[NH][2];      // maximum, what the exponents add (-m, or 0), sum of this lane's keys

  // heads h0 .. of query row qrow (heads past `heads` are zeros)
  __device__ __forceinline__ void init(const T* qrow, int heads, float sm_scale, int lane) {
    const int gid = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      const int h = nh * 8 + gid;
      float f[G32][8], amax = 0.0f;
#pragma unroll
      for (int j = 0; j < G32; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[j][i] = 0.0f;
        if (h < heads) load8(qrow + static_cast<int64_t>(h) * DH + 32 * j + 8 * t, f[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[j][i]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^E q has its maximum in [2^13, 2^14); E stays where 2^E and 2^(12 - E) are normal numbers
      const int E = max(-114, min(126, 13 + 127 - static_cast<int>(__float_as_uint(amax) >> 23)));
      const float up = __uint_as_float(static_cast<uint32_t>(E + 127) << 23);
      const float sc = sm_scale * kLog2e * __uint_as_float(static_cast<uint32_t>(12 - E + 127) << 23);
#pragma unroll
      for (int j = 0; j < G32; ++j) {
        float sum = 0.0f;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int k = 0; k < 2; ++k) {   // channels c, c + 4 of the word; the odd ones against 16 u
            const int c = 2 * s + k;
            const float w = k ? 0.0625f : 1.0f;
            float a = f[j][c] * up * w, b = f[j][c + 4] * up * w;
#pragma unroll
            for (int e = 0; e < kQ; ++e) {
              const uint32_t u = pack_half(a, b);
              const float2 r = half_pair(u);
              q[nh][e][j][s][k] = u;
              sum += (r.x + r.y) * (k ? 16.0f : 1.0f);
              a -= r.x;
              b -= r.y;
            }
          }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= -8.0f * 5.9604644775390625e-08f;   // -8 2^-24
#pragma unroll
        for (int c = 0; c < 2; ++c) start[nh][j][c] = __shfl_sync(0xffffffffu, sum, (2 * t + c) * 4);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        scale[nh][c] = __shfl_sync(0xffffffffu, sc, (2 * t + c) * 4);
        m[nh][c] = -INFINITY;
        nb[nh][c] = l[nh][c] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < DH / 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nh][i][k] = 0.0f;
    }
  }

  // keys 16 sub .. + 15 of the staged tile, key0 the first one's index in the CTA's run, n its keys
  __device__ __forceinline__ void tile16(const uint8_t* st, int sub, int key0, int n, float* x, int x_ld, int heads, int lane) {
    const int gid = lane >> 2, t = lane & 3;
    const uint8_t *sk = st, *sv = st + 1024, *sks = st + 2048, *svs = st + 2176;
    const int r0 = sub * 16 + gid, r1 = r0 + 8;
    // scores
    uint32_t kw[2][G32], ks[2][G32 / 2], vs[2][G32 / 2];
    if constexpr (DH == 128) {
      const uint4 a = *reinterpret_cast<const uint4*>(sk + r0 * 64 + t * 16), b = *reinterpret_cast<const uint4*>(sk + r1 * 64 + t * 16);
      kw[0][0] = a.x, kw[0][1] = a.y, kw[0][2] = a.z, kw[0][3] = a.w;
      kw[1][0] = b.x, kw[1][1] = b.y, kw[1][2] = b.z, kw[1][3] = b.w;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint2 c = *reinterpret_cast<const uint2*>(sks + (r ? r1 : r0) * 8), d = *reinterpret_cast<const uint2*>(svs + (r ? r1 : r0) * 8);
        ks[r][0] = c.x, ks[r][1] = c.y, vs[r][0] = d.x, vs[r][1] = d.y;
      }
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(sk + r0 * 32 + t * 8), b = *reinterpret_cast<const uint2*>(sk + r1 * 32 + t * 8);
      kw[0][0] = a.x, kw[0][1] = a.y, kw[1][0] = b.x, kw[1][1] = b.y;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        ks[r][0] = *reinterpret_cast<const uint32_t*>(sks + (r ? r1 : r0) * 4);
        vs[r][0] = *reinterpret_cast<const uint32_t*>(svs + (r ? r1 : r0) * 4);
      }
    }
    float s[NH][4];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[nh][k] = 0.0f;
#pragma unroll
    for (int j = 0; j < G32; ++j) {
      const uint32_t w0 = kw[0][j], w1 = kw[1][j], v0 = w0 >> 8, v1 = w1 >> 8;
      const uint32_t a0[4] = {w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u};
      const uint32_t a1[4] = {v0 & 0x000f000fu, v1 & 0x000f000fu, v0 & 0x00f000f0u, v1 & 0x00f000f0u};
      const float f0 = (j & 1) ? bf_hi(ks[0][j >> 1]) : bf_lo(ks[0][j >> 1]);
      const float f1 = (j & 1) ? bf_hi(ks[1][j >> 1]) : bf_lo(ks[1][j >> 1]);
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        float c[4] = {start[nh][j][0], start[nh][j][1], start[nh][j][0], start[nh][j][1]};
#pragma unroll
        for (int e = 0; e < kQ; ++e) {
          mma_f16(c, a0, q[nh][e][j][0][0], q[nh][e][j][0][1]);
          mma_f16(c, a1, q[nh][e][j][1][0], q[nh][e][j][1][1]);
        }
        s[nh][0] = fmaf(f0, c[0], s[nh][0]);
        s[nh][1] = fmaf(f0, c[1], s[nh][1]);
        s[nh][2] = fmaf(f1, c[2], s[nh][2]);
        s[nh][3] = fmaf(f1, c[3], s[nh][3]);
      }
    }
    const int i0 = key0 + r0, i1 = key0 + r1;
    bool grown = false;
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float y = (s[nh][k] * 4096.0f) * scale[nh][k & 1];   // 2^24 in two factors that stay in range
        s[nh][k] = (k < 2 ? i0 : i1) < n ? y : -INFINITY;
        grown |= s[nh][k] > m[nh][k & 1] + kRescale;
      }
      if (x) {
        const int h = nh * 8 + 2 * t;
        if (h < heads) {
          if (i0 < n) x[h * x_ld + i0] = s[nh][0];
          if (i1 < n) x[h * x_ld + i1] = s[nh][2];
        }
        if (h + 1 < heads) {
          if (i0 < n) x[(h + 1) * x_ld + i0] = s[nh][1];
          if (i1 < n) x[(h + 1) * x_ld + i1] = s[nh][3];
        }
      }
    }
    if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(s[nh][c], s[nh][c + 2]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
          mx = fmaxf(mx, m[nh][c]);
          nb[nh][c] = mx == -INFINITY ? 0.0f : -mx;
          const float f = ex2(m[nh][c] + nb[nh][c]);
          m[nh][c] = mx;
          l[nh][c] *= f;
#pragma unroll
          for (int i = 0; i < DH / 16; ++i) {
            o[nh][i][c] *= f;
            o[nh][i][c + 2] *= f;
          }
        }
    }
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s[nh][k] = ex2(s[nh][k] + nb[nh][k & 1]);
        l[nh][k & 1] += s[nh][k];
      }
    // output: keys 2t, 2t + 1 (and + 8) of four channels of every group
    uint32_t vw[2][G32];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int ra = sub * 16 + half * 8 + 2 * t;
      if constexpr (DH == 128) {
        const uint2 a = *reinterpret_cast<const uint2*>(sv + v_offset<DH>(ra, gid * 8));
        const uint2 b = *reinterpret_cast<const uint2*>(sv + v_offset<DH>(ra + 1, gid * 8));
        vw[half][0] = __byte_perm(a.x, b.x, 0x5410), vw[half][1] = __byte_perm(a.x, b.x, 0x7632);
        vw[half][2] = __byte_perm(a.y, b.y, 0x5410), vw[half][3] = __byte_perm(a.y, b.y, 0x7632);
      } else {
        const uint32_t a = *reinterpret_cast<const uint32_t*>(sv + v_offset<DH>(ra, gid * 4));
        const uint32_t b = *reinterpret_cast<const uint32_t*>(sv + v_offset<DH>(ra + 1, gid * 4));
        vw[half][0] = __byte_perm(a, b, 0x5410), vw[half][1] = __byte_perm(a, b, 0x7632);
      }
    }
#pragma unroll
    for (int j = 0; j < G32; ++j) {
      const float f0 = (j & 1) ? bf_hi(vs[0][j >> 1]) : bf_lo(vs[0][j >> 1]);
      const float f1 = (j & 1) ? bf_hi(vs[1][j >> 1]) : bf_lo(vs[1][j >> 1]);
      uint32_t av[2][4];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        av[c][0] = code_pair(vw[0][j] >> (8 * c));
        av[c][1] = code_pair(vw[0][j] >> (8 * c + 4));
        av[c][2] = code_pair(vw[1][j] >> (8 * c));
        av[c][3] = code_pair(vw[1][j] >> (8 * c + 4));
      }
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        float p[4] = {s[nh][0] * f0, s[nh][1] * f0, s[nh][2] * f1, s[nh][3] * f1};
#pragma unroll
        for (int e = 0; e < kP; ++e) {
          const uint32_t u0 = pack_bf16(p[0], p[1]), u1 = pack_bf16(p[2], p[3]);
          if (e + 1 < kP) {
            p[0] -= bf_lo(u0);
            p[1] -= bf_hi(u0);
            p[2] -= bf_lo(u1);
            p[3] -= bf_hi(u1);
          }
          const uint32_t b0 = transpose8x8(u0), b1 = transpose8x8(u1);
          mma_bf16(o[nh][2 * j], av[0], b0, b1);
          mma_bf16(o[nh][2 * j + 1], av[1], b0, b1);
        }
      }
    }
  }
};

template <int DH, int NH, typename T>
__global__ void __launch_bounds__(kThreads, NH == 2 && sizeof(T) == 4 ? 1 : 2) kv4_attn_kernel(AttnArgs args) {
  using W = Warp<DH, NH, T>;
  constexpr int TK = W::TK, G32 = W::G32, kHeads = NH * 8;
  extern __shared__ __align__(128) uint8_t smem[];   // the warps' rings (later their sums), then the scores
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  __shared__ float c_m[kHeads], c_l[kHeads], f_m[kHeads], f_l[kHeads];   // the CTA's, the cluster's (sum inverted)
  __shared__ float c_o[kHeads][DH];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = gridDim.x, rank = blockIdx.x;
  const spatten_kv4_attn_args& a = args.a;
  const spatten_kv4_cache& c = a.cache;
  const int hk = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.H / c.H_kv;
  const int n_all = clamp_len(a.len[b], a.n_max, a.dev_status);
  const int run = (((n_all + C - 1) / C) + TK - 1) / TK * TK;   // keys per CTA
  const int first = min(n_all, rank * run), n = min(run, n_all - first);
  const int64_t row0 = (static_cast<int64_t>(b) * c.H_kv + hk) * c.cap + first;
  const int tiles = (n + TK - 1) / TK;
  uint8_t* ring = smem + warp * kStages * kStageBytes;
  float* x = args.x ? args.x + ((static_cast<int64_t>(b) * c.H_kv + hk) * C + rank) * args.heads * static_cast<int64_t>(args.x_ld)
                    : reinterpret_cast<float*>(smem + kRing);
  if (!a.update_weight) x = nullptr;

  auto load = [&](int tile, int stage) {
    const uint32_t dst = smem_addr(ring + stage * kStageBytes);
    const int key0 = tile * TK;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = lane + 32 * i, r = e / (DH / 32), ch = e % (DH / 32);
      const bool ok = key0 + r < n;
      const int64_t at = (row0 + (ok ? key0 + r : 0)) * (DH / 2) + ch * 16;
      cp_async<16>(dst + r * (DH / 2) + ch * 16, c.k_codes + at, ok);
      cp_async<16>(dst + 1024 + v_offset<DH>(r, ch * 16), c.v_codes + at, ok);
    }
    if constexpr (DH == 128) {
      const int r = lane & 15;
      const bool ok = key0 + r < n;
      cp_async<8>(dst + 2048 + lane * 8, (lane < 16 ? c.k_scale : c.v_scale) + (row0 + (ok ? key0 + r : 0)) * G32, ok);
    } else {
      const bool ok = key0 + lane < n;
      const int64_t at = (row0 + (ok ? key0 + lane : 0)) * G32;
      cp_async<4>(dst + 2048 + lane * 4, c.k_scale + at, ok);
      cp_async<4>(dst + 2176 + lane * 4, c.v_scale + at, ok);
    }
  };

  for (int h0 = 0; h0 < group; h0 += kHeads) {
    const int heads = min(kHeads, group - h0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (warp + kWarps * i < tiles) load(warp + kWarps * i, i);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    W w;
    w.init(static_cast<const T*>(a.q) + b * a.q_ld + (static_cast<int64_t>(hk) * group + h0) * DH, heads, a.sm_scale, lane);
    for (int tile = warp, i = 0; tile < tiles; tile += kWarps, ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();   // every lane's copies have landed, and every lane is done with the previous tile
      if (tile + kWarps * (kStages - 1) < tiles) load(tile + kWarps * (kStages - 1), (i + kStages - 1) % kStages);
      asm volatile("cp.async.commit_group;" ::: "memory");
      const uint8_t* st = ring + (i % kStages) * kStageBytes;
#pragma unroll
      for (int sub = 0; sub < TK / 16; ++sub) w.tile16(st, sub, tile * TK, n, x, args.x_ld, heads, lane);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");

    // the warps' sums, over their common maximum, in warp order
    const int gid = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float l = w.l[nh][k];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (gid == 0) {
          s_m[warp][nh * 8 + 2 * t + k] = w.m[nh][k];
          s_l[warp][nh * 8 + 2 * t + k] = l;
        }
      }
    __syncthreads();   // also: every ring is free
    float* part = reinterpret_cast<float*>(smem);   // [warp][head][channel]
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int h = nh * 8 + 2 * t + k;
        float mx = s_m[0][h];
#pragma unroll
        for (int v = 1; v < kWarps; ++v) mx = fmaxf(mx, s_m[v][h]);
        const float f = ex2(w.m[nh][k] - (mx == -INFINITY ? 0.0f : mx));
        float* dst = part + (warp * kHeads + h) * DH;
#pragma unroll
        for (int j = 0; j < G32; ++j) {   // channels 32 j + 4 gid .. + 3
          const float4 v = make_float4(w.o[nh][2 * j][k] * f, w.o[nh][2 * j][k + 2] * f, w.o[nh][2 * j + 1][k] * f,
                                       w.o[nh][2 * j + 1][k + 2] * f);
          if (h < heads) *reinterpret_cast<float4*>(dst + 32 * j + 4 * gid) = v;
        }
      }
    if (tid < heads) {
      float mx = s_m[0][tid], l = 0.0f;
      for (int v = 1; v < kWarps; ++v) mx = fmaxf(mx, s_m[v][tid]);
      const float base = mx == -INFINITY ? 0.0f : mx;
      for (int v = 0; v < kWarps; ++v) l = fmaf(s_l[v][tid], ex2(s_m[v][tid] - base), l);
      c_m[tid] = mx;
      c_l[tid] = l;
    }
    __syncthreads();
    for (int e = tid; e < heads * DH; e += kThreads) {
      float v = 0.0f;
#pragma unroll
      for (int u = 0; u < kWarps; ++u) v += part[u * kHeads * DH + e];
      c_o[e / DH][e % DH] = v;
    }
    // the cluster's sums, in rank order
    if (C > 1) cluster.sync();
    else __syncthreads();
    if (tid < heads) {
      float mx = -INFINITY, l = 0.0f;
      for (int r = 0; r < C; ++r) mx = fmaxf(mx, *cluster.map_shared_rank(&c_m[tid], r));
      const float base = mx == -INFINITY ? 0.0f : mx;
      for (int r = 0; r < C; ++r) l = fmaf(*cluster.map_shared_rank(&c_l[tid], r), ex2(*cluster.map_shared_rank(&c_m[tid], r) - base), l);
      f_m[tid] = base;
      f_l[tid] = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // an empty sequence gives 0, NaN stays
    }
    __syncthreads();
    for (int e = rank * kThreads + tid; e < heads * DH; e += C * kThreads) {
      const int h = e / DH, ch = e % DH;
      float v = 0.0f;
      for (int r = 0; r < C; ++r)
        v = fmaf(*cluster.map_shared_rank(&c_o[h][ch], r), ex2(*cluster.map_shared_rank(&c_m[h], r) - f_m[h]), v);
      st_from_float(static_cast<T*>(a.o) + b * a.o_ld + (static_cast<int64_t>(hk) * group + h0 + h) * DH + ch, v * f_l[h]);
    }
    if (x)
      for (int i = tid; i < n; i += kThreads) {
        float v = 0.0f;
        for (int h = 0; h < heads; ++h) v = fmaf(ex2(x[h * args.x_ld + i] - f_m[h]), f_l[h], v);
        c.weight[row0 + i] += v;
      }
    if (C > 1) cluster.sync();   // peers have read this CTA's sums
    else __syncthreads();
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

struct Shape {
  int C;           // CTAs per (sequence, key/value head)
  int x_ld, heads;
  size_t x_smem;   // bytes of scores in shared memory (0: none, or in the workspace)
  bool x_ws;
};

// Enough CTAs to fill the SMs, none with less than a tile per warp, and scores that let two CTAs share
// an SM where more CTAs achieve that; scores that fit no SM go to the workspace.
Shape shape(const spatten_kv4_attn_args& a) {
  Shape s{};
  const int tk = 2048 / a.cache.d_h;
  s.heads = std::min(a.H / a.cache.H_kv, kMaxHeads);
  const int64_t pairs = static_cast<int64_t>(a.cache.B) * a.cache.H_kv;
  auto ld = [&](int C) { return static_cast<int>(align_up(static_cast<size_t>(ceil_div(a.n_max, C)), 32) + 4); };
  auto bytes = [&](int C) { return a.update_weight ? static_cast<size_t>(s.heads) * ld(C) * sizeof(float) : 0; };
  s.C = 1;
  while (s.C < 8 && a.n_max > s.C * kWarps * tk && (pairs * s.C < sm_count() || bytes(s.C) > kSharedTwo)) s.C *= 2;
  s.x_ld = ld(s.C);
  s.x_ws = bytes(s.C) > kSharedOne;
  s.x_smem = s.x_ws ? 0 : bytes(s.C);
  return s;
}

size_t layout(const spatten_kv4_attn_args& a, void* ws, size_t ws_bytes, AttnArgs* x) {
  const Shape s = shape(a);
  WsCursor c(ws, ws_bytes);
  float* p = s.x_ws ? c.take<float>(static_cast<size_t>(a.cache.B) * a.cache.H_kv * s.C * s.heads * s.x_ld) : nullptr;
  if (x) x->x = p, x->x_ld = s.x_ld, x->heads = s.heads;
  return align_up(std::max<size_t>(c.used, 1), 256);   // never 0: callers allocate it as it comes
}

template <int DH, int NH, typename T>
int32_t launch(const AttnArgs& x, const Shape& s, cudaStream_t st) {
  static DeviceOnce once;
  int dev;
  SPT_TRY(once_per_device(once, &dev, [](int) -> int32_t {
    SPT_CUDA(cudaFuncSetAttribute(kv4_attn_kernel<DH, NH, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(kRing + kSharedOne)));
    return SPATTEN_OK;
  }));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(s.C);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(s.C), static_cast<unsigned>(x.a.cache.H_kv), static_cast<unsigned>(x.a.cache.B));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kRing + s.x_smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  SPT_CUDA(cudaLaunchKernelEx(&cfg, kv4_attn_kernel<DH, NH, T>, x));
  return launch_status();
}

template <int DH, typename T>
int32_t launch_heads(const AttnArgs& x, const Shape& s, cudaStream_t st) {
  return s.heads <= 8 ? launch<DH, 1, T>(x, s, st) : launch<DH, 2, T>(x, s, st);
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
  AttnArgs x{};
  x.a = *a;
  const size_t need = layout(*a, ws, ws_bytes, &x);
  if (!ws || ws_bytes < need) return SPATTEN_E_WORKSPACE;
  if (!aligned16(ws)) return SPATTEN_E_ALIGN;
  if (!(x.a.sm_scale > 0.0f)) x.a.sm_scale = 1.0f / std::sqrt(static_cast<float>(a->cache.d_h));
  const Shape s = shape(*a);
  cudaStream_t st = as_stream(stream);
  const bool bf = a->dtype == SPATTEN_BF16;
  if (a->cache.d_h == 64)
    return bf ? launch_heads<64, __nv_bfloat16>(x, s, st) : launch_heads<64, float>(x, s, st);
  return bf ? launch_heads<128, __nv_bfloat16>(x, s, st) : launch_heads<128, float>(x, s, st);
}
