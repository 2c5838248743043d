// spatten_kv4_attention: one query row per sequence over the 4-bit cache, grouped heads.
//
// Up to a wave of CTAs, a cluster of C CTAs owns one (sequence, key/value head) and each CTA a run of its keys
// (the cluster form); beyond it, all tiles of the call are dealt out evenly to two CTAs per SM, which leave
// their parts and scores in the workspace for a second kernel that joins them (the split form: shape() has the
// rule, both sides measured).  In both, each warp takes tiles of TK keys, copied asynchronously into a ring of
// its own (no barriers in the loop).  The products
// run on mma.sync m16n8k16 with the codes as the 16-row operand and up to 8 heads as the 8 columns:
//   scores   S^T[16 keys][8 heads] = codes . q, one accumulator per group of 32 channels, which the
//            group's scale then multiplies (so the codes enter exactly).  A nibble u = code + 8 in the
//            low bits of a half is the subnormal u 2^-24, one place higher 16 u 2^-24: no conversion
//            beyond the masks; the 16 is taken out of q, and the 8 enters as the accumulator's start,
//            -8 sum(q).  q is scaled by a power of two to a maximum in [2^13, 2^14) and rounded to fp16
//            (bfloat16 queries: exact down to 2^-27 of the maximum).  Float32 queries are the sum of two
//            fp16, and against them the nibbles become codes, 1024 + u - 1032: the sums with u in place of
//            the code are larger and cost two bits.
//   output   O^T[16 channels][8 heads] += codes . P', P' = exp(S - m) times the key's scale of the
//            group, rounded to bfloat16 (its range is that of the scales) for bfloat16 queries and
//            held as the sum of three bfloat16 (24 bits) for float32 ones, whose products leave the tensor cores
//            every 16 keys; movmatrix turns P' from the
//            score layout into the operand's.  Codes become bfloat16 as 128 + u - 136, exact.
// The tensor path is the register one since its operands are made in registers: a tcgen05 operand would
// have to go through shared memory first, and the kernel is bound by memory and by the unpacking, not
// by the products.
// In the cluster form scores stay in shared memory (in the workspace when they do not fit), so that the
// weights need only one more exponential per score once the cluster has exchanged its maxima and sums.  Sums
// are float32 in a fixed order.
// Groups of nine to sixteen heads take two columns in one pass, larger ones several passes: 4 x 8192 rows of 4 heads
// of 128 with 16 queries each 42 us (float32 45).  In bfloat16 at 128 channels two columns need more registers than
// two CTAs an SM have (588 bytes spill); one CTA an SM took 31 us there, but 29 for 16 x 1152 rows against 22, and
// passes of eight heads 34 and 20.
// What bounds them: 16 x 1152 rows of 16 heads of 64, 11.6 us a call, the chain of one CTA (query, tiles, joining,
// weights: 13,500 cycles); 32 x 16,384 rows of 8 heads of 128 with 4 queries each (478 MB), 142 us, of which the
// split kernel takes 119 (no unit is full: 2.6 of 4 instructions a clock, ALU pipe 58 %, DRAM 51 %; a warp's chain
// scores, vote, exponentials, product is what is left of the latency) and reading the scores back for the weights 22.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "kv4.cuh"

namespace cg = cooperative_groups;

namespace spt {
namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kStages = 3;             // tiles in a warp's ring (4 leave room for less scores)
constexpr int kStageBytes = 2304;      // 1024 + 1024 bytes of codes, 128 + 128 of scales
constexpr int kMaxHeads = 16;          // heads of a group per pass over the keys
constexpr int kMaxC = 8;               // CTAs per cluster
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.0f;       // growth of a maximum (log2) that makes the sums be rescaled
// the warps' rings, which later hold their output sums
__host__ __device__ constexpr int ring_bytes(int dh, int nh) {
  return kWarps * (kStages * kStageBytes > nh * 8 * dh * 4 ? kStages * kStageBytes : nh * 8 * dh * 4);
}

template <int DH> constexpr int kTileKeys = 2048 / DH;

struct AttnArgs {
  spatten_kv4_attn_args a;
  float* x;         // ws scores: [B][H_kv][C][heads][x_ld] of clusters (NULL: in shared memory), [B][H_kv][heads][x_ld] of
                    // the split form (NULL: no weights)
  int64_t x_ld;     // floats between the heads' scores
  int32_t heads;    // min(H / H_kv, kMaxHeads)
  // the split form: CTAs, first head of the pass, and each segment's maxima, sums and outputs
  int32_t ctas, h0;
  float2* part_ml;  // ws [ctas + B H_kv][heads]
  float* part_o;    // ws [ctas + B H_kv][heads][d_h]
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
// copies, or zero-fills; `valid` is an address that may be read in either case
template <int BYTES>
__device__ __forceinline__ void cp_async_if(uint32_t dst, const void* src, const void* valid, bool ok) {
  const void* p = ok ? src : valid;
  const int n = ok ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(p), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(p), "n"(BYTES), "r"(n) : "memory");
}
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_zero(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_bf16_zero(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
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
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0xc308c308u));   // - 136
  return r;
}

// two nibbles at bits 0-3 and 16-19 (ODD: 4-7 and 20-23) of w as the fp16 pair of their codes, exact
template <bool ODD>
__device__ __forceinline__ uint32_t code_pair_f16(uint32_t w) {
  const uint32_t u = (w & (ODD ? 0x00f000f0u : 0x000f000fu)) | 0x64006400u;   // 1024 + u, 1024 + 16 u
  uint32_t r;
  if constexpr (ODD) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(u), "r"(0x2c002c00u), "r"(0xd480d480u));   // / 16 - 72
  else asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0xe408e408u));                                   // - 1032
  return r;
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
  // what the lanes need of one column of heads, made once per CTA, a warp for each group of channels
  struct Query {
    uint4 q[kQ][G32][32];         // B operand of the scores: (step, half) of a group
    float sum[8][G32];            // -8 2^-24 sum(q) of each head's groups
    float scale[8];               // factor to log2 units
  };
  static constexpr int kPrepareWarps = NH * G32;
  uint32_t q[NH][kQ][G32][4];
  uint32_t start[NH][2];
  float scale[NH][2];
  float o[NH][DH / 16][4];
  float lim[NH][2], nb[NH][2], l[NH][2];    // maximum + kRescale, what the exponents add (-maximum, or 0), sum of this lane's keys

  // a lane's share of a head's channels: of every group eight, as they are loaded
  struct Raw {
    uint4 u[G32][sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* qrow, int nh, int heads, int lane) {   // heads past `heads` are zeros
      const int h = nh * 8 + (lane >> 2);
#pragma unroll
      for (int j = 0; j < G32; ++j)
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
          u[j][i] = h < heads ? reinterpret_cast<const uint4*>(qrow + static_cast<int64_t>(h) * DH + 32 * j + 8 * (lane & 3))[i] : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(int j, float* x) const {
      const uint32_t w[4] = {u[j][0].x, u[j][0].y, u[j][0].z, u[j][0].w};
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = bf_lo(w[i]), x[2 * i + 1] = bf_hi(w[i]);
      } else {
        const uint4 v = u[j][sizeof(T) / 2 - 1];
        const uint32_t w1[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]), x[4 + i] = __uint_as_float(w1[i]);
      }
    }
  };
  // group `own` of a column of heads; one warp
  static __device__ __forceinline__ void prepare(Query& out, const Raw& raw, int own, float sm_scale, int lane) {
    const int gid = lane >> 2, t = lane & 3;
    float g[8], amax = 0.0f;
#pragma unroll
    for (int j = 0; j < G32; ++j) {
      float x[8];
      raw.get(j, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        amax = fmaxf(amax, fabsf(x[i]));
        g[i] = j == 0 || j == own ? x[i] : g[i];
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // 2^E q has its maximum in [2^13, 2^14); E stays where 2^E and 2^(12 - E) are normal numbers
    const int E = max(-114, min(126, 13 + 127 - static_cast<int>(__float_as_uint(amax) >> 23)));
    const float up = __uint_as_float(static_cast<uint32_t>(E + 127) << 23);
    float sum = 0.0f;
    uint32_t u[kQ][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {   // channels c, c + 4 of the word; the odd ones against 16 u
      const float w = !kF32 && (c & 1) ? 0.0625f : 1.0f;
      float x = g[c] * up * w, y = g[c + 4] * up * w;
#pragma unroll
      for (int e = 0; e < kQ; ++e) {
        u[e][c] = pack_half(x, y);
        const float2 r = half_pair(u[e][c]);
        sum += (r.x + r.y) * ((c & 1) ? 16.0f : 1.0f);
        x -= r.x;
        y -= r.y;
      }
    }
#pragma unroll
    for (int e = 0; e < kQ; ++e) out.q[e][own][lane] = make_uint4(u[e][0], u[e][1], u[e][2], u[e][3]);
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (t == 0) {
      out.sum[gid][own] = sum * (-8.0f * 5.9604644775390625e-08f);   // -8 2^-24
      if (own == 0) out.scale[gid] = sm_scale * kLog2e * __uint_as_float(static_cast<uint32_t>(12 - E + 127) << 23);
    }
  }

  __device__ __forceinline__ void init(const Query* in, int lane) {
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
      for (int j = 0; j < G32; ++j) {
#pragma unroll
        for (int e = 0; e < kQ; ++e) {
          const uint4 u = in[nh].q[e][j][lane];
          q[nh][e][j][0] = u.x, q[nh][e][j][1] = u.y, q[nh][e][j][2] = u.z, q[nh][e][j][3] = u.w;
        }
      }
      // -8 sum(q) of the groups as three bfloat16 each, along the operand's 16 rows against the keys' scales:
      // rows 2t, 2t + 1 hold a term of two groups (128 channels: t = 0, 1 the first, 2, 3 the second, 0, 1 of
      // the upper eight the third; 64: t = 0, 1, 2)
      const int t = lane & 3;
      const float2 st = *reinterpret_cast<const float2*>(&in[nh].sum[lane >> 2][DH == 128 ? 2 * (t & 1) : 0]);
      const uint32_t t0 = pack_bf16(st.x, st.y);
      const float x1 = st.x - bf_lo(t0), y1 = st.y - bf_hi(t0);
      const uint32_t t1 = pack_bf16(x1, y1), t2 = pack_bf16(x1 - bf_lo(t1), y1 - bf_hi(t1));
      if constexpr (DH == 128) {
        start[nh][0] = t < 2 ? t0 : t1;
        start[nh][1] = t < 2 ? t2 : 0u;
      } else {
        start[nh][0] = t == 0 ? t0 : (t == 1 ? t1 : (t == 2 ? t2 : 0u));
        start[nh][1] = 0u;
      }
      const float2 sc = *reinterpret_cast<const float2*>(&in[nh].scale[2 * t]);
      scale[nh][0] = sc.x, scale[nh][1] = sc.y;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        lim[nh][c] = -INFINITY;
        nb[nh][c] = l[nh][c] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < DH / 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nh][i][k] = 0.0f;
    }
  }
  __device__ __forceinline__ float maximum(int nh, int c) const { return lim[nh][c] == -INFINITY ? -INFINITY : -nb[nh][c]; }

  // sixteen keys of a staged tile; sk, sv, ss: this lane's first K and V codes and K scales of them.
  // xs: where this lane's scores go (keys gid and gid + 8 of heads 2t and, x_ld behind, 2t + 1; 8 x_ld per
  // column), or NULL.  left: keys there are, counted from key gid (FULL: all).
  template <bool FULL>
  __device__ __forceinline__ void tile16(const uint8_t* sk, const uint8_t* sv, const uint8_t* ss, float* xs, int64_t x_ld, int heads,
                                         int left, int lane) {
    const int t = lane & 3;
    uint32_t kw[2][G32], ks[2][G32 / 2], vs[2][G32 / 2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {   // keys gid, gid + 8
      if constexpr (DH == 128) {
        const uint4 k = *reinterpret_cast<const uint4*>(sk + r * 512);
        kw[r][0] = k.x, kw[r][1] = k.y, kw[r][2] = k.z, kw[r][3] = k.w;
        const uint2 c = *reinterpret_cast<const uint2*>(ss + r * 64), d = *reinterpret_cast<const uint2*>(ss + 128 + r * 64);
        ks[r][0] = c.x, ks[r][1] = c.y, vs[r][0] = d.x, vs[r][1] = d.y;
      } else {
        const uint2 k = *reinterpret_cast<const uint2*>(sk + r * 256);
        kw[r][0] = k.x, kw[r][1] = k.y;
        ks[r][0] = *reinterpret_cast<const uint32_t*>(ss + r * 32);
        vs[r][0] = *reinterpret_cast<const uint32_t*>(ss + 128 + r * 32);
      }
    }
    float s[NH][4];
    if constexpr (kF32) {
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[nh][k] = 0.0f;
    } else {
      // 128 channels: scales 0, 1 on even, 2, 3 on odd lanes of a quad
      const uint8_t* sa = DH == 128 ? ss + (t & 1) * 4 : ss;
      const uint32_t k0 = *reinterpret_cast<const uint32_t*>(sa), k1 = *reinterpret_cast<const uint32_t*>(sa + (DH == 128 ? 64 : 32));
      const uint32_t ak[4] = {k0, k1, k0, k1};
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) mma_bf16_zero(s[nh], ak, start[nh][0], start[nh][1]);
    }
#pragma unroll
    for (int j = 0; j < G32; ++j) {
      const uint32_t w0 = kw[0][j], w1 = kw[1][j], v0 = w0 >> 8, v1 = w1 >> 8;
      uint32_t a0[4] = {w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u};
      uint32_t a1[4] = {v0 & 0x000f000fu, v1 & 0x000f000fu, v0 & 0x00f000f0u, v1 & 0x00f000f0u};
      if constexpr (kF32) {
        a0[0] = code_pair_f16<false>(w0), a0[1] = code_pair_f16<false>(w1), a0[2] = code_pair_f16<true>(w0), a0[3] = code_pair_f16<true>(w1);
        a1[0] = code_pair_f16<false>(v0), a1[1] = code_pair_f16<false>(v1), a1[2] = code_pair_f16<true>(v0), a1[3] = code_pair_f16<true>(v1);
      }
      const float f0 = (j & 1) ? bf_hi(ks[0][j >> 1]) : bf_lo(ks[0][j >> 1]);
      const float f1 = (j & 1) ? bf_hi(ks[1][j >> 1]) : bf_lo(ks[1][j >> 1]);
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        float c[4];
#pragma unroll
        for (int e = 0; e < kQ; ++e) {
          if (e == 0) mma_f16_zero(c, a0, q[nh][e][j][0], q[nh][e][j][1]);
          else mma_f16(c, a0, q[nh][e][j][0], q[nh][e][j][1]);
          mma_f16(c, a1, q[nh][e][j][2], q[nh][e][j][3]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) s[nh][k] = fmaf(k < 2 ? f0 : f1, c[k], s[nh][k]);
      }
    }
    bool grown = false;
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // 2^24 (of nibbles), 1 (of codes) 2^-E in two factors that stay in range
        s[nh][k] = (s[nh][k] * (kF32 ? 1.0f / 4096.0f : 4096.0f)) * scale[nh][k & 1];
        if (!FULL && left <= (k < 2 ? 0 : 8)) s[nh][k] = -INFINITY;
        grown |= s[nh][k] > lim[nh][k & 1];
      }
      if (xs) {
        float* p = xs + nh * 8 * x_ld;
        const int h = nh * 8 + 2 * t;
        if (h < heads) {
          if (FULL || left > 0) p[0] = s[nh][0];
          if (FULL || left > 8) p[8] = s[nh][2];
        }
        if (h + 1 < heads) {
          if (FULL || left > 0) p[x_ld] = s[nh][1];
          if (FULL || left > 8) p[x_ld + 8] = s[nh][3];
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
          const float old = maximum(nh, c);
          mx = fmaxf(mx, old);
          lim[nh][c] = mx + kRescale;
          nb[nh][c] = mx == -INFINITY ? 0.0f : -mx;
          const float f = ex2(old + nb[nh][c]);
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
      if constexpr (DH == 128) {
        const uint2 a = *reinterpret_cast<const uint2*>(sv + half * 512), b = *reinterpret_cast<const uint2*>(sv + half * 512 + 256);
        vw[half][0] = __byte_perm(a.x, b.x, 0x5410), vw[half][1] = __byte_perm(a.x, b.x, 0x7632);
        vw[half][2] = __byte_perm(a.y, b.y, 0x5410), vw[half][3] = __byte_perm(a.y, b.y, 0x7632);
      } else {
        const uint32_t a = *reinterpret_cast<const uint32_t*>(sv + half * 256), b = *reinterpret_cast<const uint32_t*>(sv + half * 256 + 128);
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
        if constexpr (kP == 1) {
          const uint32_t b0 = transpose8x8(pack_bf16(p[0], p[1])), b1 = transpose8x8(pack_bf16(p[2], p[3]));
          mma_bf16(o[nh][2 * j], av[0], b0, b1);
          mma_bf16(o[nh][2 * j + 1], av[1], b0, b1);
        } else {
          // The tensor cores cut their sums off: over a long run these would drift towards 0.  Sixteen keys start from
          // 0, small terms first, and are added here, rounded to nearest.
          uint32_t b[kP][2];
#pragma unroll
          for (int e = 0; e < kP; ++e) {
            const uint32_t u0 = pack_bf16(p[0], p[1]), u1 = pack_bf16(p[2], p[3]);
            p[0] -= bf_lo(u0), p[1] -= bf_hi(u0), p[2] -= bf_lo(u1), p[3] -= bf_hi(u1);
            b[e][0] = transpose8x8(u0), b[e][1] = transpose8x8(u1);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float t16[4];
            mma_bf16_zero(t16, av[c], b[kP - 1][0], b[kP - 1][1]);
#pragma unroll
            for (int e = kP - 2; e >= 0; --e) mma_bf16(t16, av[c], b[e][0], b[e][1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[nh][2 * j + c][k] += t16[k];
          }
        }
      }
    }
  }
};

// A warp's way through a run of n rows of the cache from row0 on: the CTA's kWarps warps take its tiles in turn.
template <int DH>
struct Run {
  static constexpr int TK = kTileKeys<DH>, G32 = DH / kKv4Group;
  static constexpr int kPieces = DH / 32;   // 16-byte pieces of a row's codes
  static constexpr int kRingBytes = kStages * kStageBytes;
  const spatten_kv4_cache& c;
  uint8_t* ring;
  int warp, lane;
  // this lane's pieces of the tile to copy next: where they come from, where they go, and the run's rows from that
  // tile on.  (Addresses made anew for every tile were an eighth of the kernel's instructions.)
  const uint8_t *pk, *pv, *ps, *pt;
  uint32_t d_code, d_v0, d_v1, d_scale, d_stage;
  int to_copy, rows;
  int lk, lv, ls;   // its first codes and scales of a staged tile

  __device__ __forceinline__ Run(const spatten_kv4_cache& cache, uint8_t* rings, int warp_, int lane_)
      : c(cache), ring(rings + warp_ * kRingBytes), warp(warp_), lane(lane_) {
    const int r = lane / kPieces, ch = lane % kPieces, gid = lane >> 2, t = lane & 3;
    d_code = smem_addr(ring) + lane * 16;
    d_v0 = smem_addr(ring) + 1024 + v_offset<DH>(r, ch * 16);
    d_v1 = smem_addr(ring) + 1024 + v_offset<DH>(r + 32 / kPieces, ch * 16);
    d_scale = smem_addr(ring) + 2048 + lane * (DH / 16);
    lk = gid * (DH / 2) + t * (DH / 8);
    lv = 1024 + v_offset<DH>(2 * t, gid * (DH / 16));   // slot t holds V's row 2t, slot 4 + t row 2t + 1
    ls = 2048 + gid * (DH / 16);
  }
  __device__ __forceinline__ void load() {   // copies the warp's next tile, if there is one
    const uint32_t d = d_stage;
    if (to_copy >= TK) {
      cp_async<16>(d_code + d, pk);
      cp_async<16>(d_code + d + 512, pk + 512);
      cp_async<16>(d_v0 + d, pv);
      cp_async<16>(d_v1 + d, pv + 512);
      if constexpr (DH == 128) {
        cp_async<8>(d_scale + d, ps);
      } else {
        cp_async<4>(d_scale + d, ps);
        cp_async<4>(d_scale + d + 128, pt);
      }
    } else if (to_copy > 0) {   // rows past the keys are zero-filled, not read
      const int r = lane / kPieces;
      const bool ok0 = r < to_copy, ok1 = r + 32 / kPieces < to_copy, oks = (DH == 128 ? lane & 15 : lane) < to_copy;
      cp_async_if<16>(d_code + d, pk, c.k_codes, ok0);
      cp_async_if<16>(d_code + d + 512, pk + 512, c.k_codes, ok1);
      cp_async_if<16>(d_v0 + d, pv, c.v_codes, ok0);
      cp_async_if<16>(d_v1 + d, pv + 512, c.v_codes, ok1);
      if constexpr (DH == 128) {
        cp_async_if<8>(d_scale + d, ps, c.k_scale, oks);
      } else {
        cp_async_if<4>(d_scale + d, ps, c.k_scale, oks);
        cp_async_if<4>(d_scale + d + 128, pt, c.v_scale, oks);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    pk += kWarps * TK * (DH / 2);
    pv += kWarps * TK * (DH / 2);
    ps += kWarps * TK * G32 * 2;
    if constexpr (DH == 64) pt += kWarps * TK * G32 * 2;
    to_copy -= kWarps * TK;
    d_stage = d_stage == kRingBytes - kStageBytes ? 0 : d_stage + kStageBytes;
  }
  __device__ __forceinline__ void start(int64_t row0, int n) {
    const int64_t at = (row0 + warp * TK) * (DH / 2) + lane * 16, as = (row0 + warp * TK + (DH == 128 ? lane & 15 : lane)) * G32;
    pk = c.k_codes + at;
    pv = c.v_codes + at;
    ps = reinterpret_cast<const uint8_t*>((DH == 64 || lane < 16 ? c.k_scale : c.v_scale) + as);
    pt = reinterpret_cast<const uint8_t*>(c.v_scale + as);   // 64 channels
    rows = to_copy = n - warp * TK;
    d_stage = 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load();
  }
  // x: the scores of the run's first key, or NULL
  template <class W>
  __device__ __forceinline__ void process(W& w, float* x, int64_t x_ld, int heads) {
    float* xt = x ? x + 2 * (lane & 3) * x_ld + warp * TK + (lane >> 2) : nullptr;
    const uint8_t* st = ring;
    for (int left = rows; left > 0; left -= kWarps * TK) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();   // every lane's copies have landed, and every lane is done with the previous tile
      load();
      if (left >= TK) {
#pragma unroll
        for (int sub = 0; sub < TK / 16; ++sub)
          w.template tile16<true>(st + lk + sub * 512, st + lv + sub * 512, st + ls + sub * 64, xt ? xt + 16 * sub : nullptr, x_ld, heads, 0, lane);
      } else {
#pragma unroll 1
        for (int sub = 0; sub < TK / 16; ++sub)
          w.template tile16<false>(st + lk + sub * 512, st + lv + sub * 512, st + ls + sub * 64, xt ? xt + 16 * sub : nullptr, x_ld, heads,
                                   left - 16 * sub - (lane >> 2), lane);
      }
      if (xt) xt += kWarps * TK;
      st = st == ring + (kRingBytes - kStageBytes) ? ring : st + kStageBytes;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
};

// The warps' sums over their common maxima, in warp order: ml(h, maximum, sum) by the threads that `by` gives a
// head (-1: none), o(e, sum) for the heads' channels e; between() runs before the block meets.
template <int DH, int NH, class W, typename By, typename Between, typename Ml, typename O>
__device__ __forceinline__ void merge_warps(const W& w, uint8_t* smem, float (*s_m)[NH * 8], float (*s_l)[NH * 8], int heads, By by,
                                            Between between, Ml ml, O o) {
  constexpr int kPart = ring_bytes(DH, NH) / kWarps / 4;   // floats of a warp's share of the rings
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nh = 0; nh < NH; ++nh)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float l = w.l[nh][k];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      if (gid == 0) {
        s_m[warp][nh * 8 + 2 * t + k] = w.maximum(nh, k);
        s_l[warp][nh * 8 + 2 * t + k] = l;
      }
    }
  __syncwarp();
  float* part = reinterpret_cast<float*>(smem);   // [warp][head][channel]: over the warp's own ring (and, 16 heads, more)
  if (ring_bytes(DH, NH) > kWarps * kStages * kStageBytes) __syncthreads();   // which others may still read
#pragma unroll
  for (int nh = 0; nh < NH; ++nh)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int h = nh * 8 + 2 * t + k;
      if (h < heads) {
        float* dst = part + warp * kPart + h * DH + 4 * gid;
#pragma unroll
        for (int j = 0; j < DH / 32; ++j)   // channels 32 j + 4 gid .. + 3
          *reinterpret_cast<float4*>(dst + 32 * j) = make_float4(w.o[nh][2 * j][k], w.o[nh][2 * j][k + 2], w.o[nh][2 * j + 1][k], w.o[nh][2 * j + 1][k + 2]);
      }
    }
  between();
  __syncthreads();
  float fac[kWarps];
  auto factors = [&](int h) {   // of the warps' sums; the maximum
    float m[kWarps], mx = -INFINITY;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) mx = fmaxf(mx, m[v] = s_m[v][h]);
#pragma unroll
    for (int v = 0; v < kWarps; ++v) fac[v] = ex2(m[v] - (mx == -INFINITY ? 0.0f : mx));
    return mx;
  };
  if (const int h = by(tid); h >= 0) {
    const float mx = factors(h);
    float l = 0.0f;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) l = fmaf(s_l[v][h], fac[v], l);
    ml(h, mx, l);
  }
  for (int e = tid; e < heads * DH; e += kThreads) {
    factors(e / DH);
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v = fmaf(part[k * kPart + e], fac[k], v);
    o(e, v);
  }
}

template <int DH, int NH, typename T>
__global__ void __launch_bounds__(kThreads, NH == 2 && sizeof(T) == 4 ? 1 : 2) kv4_attn_kernel(AttnArgs args) {
  using W = Warp<DH, NH, T>;
  constexpr int TK = W::TK, G32 = W::G32, kHeads = NH * 8;
  extern __shared__ __align__(128) uint8_t smem[];   // the warps' rings (later their sums), then the scores
  __shared__ __align__(16) typename W::Query query[NH];
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  // what the CTAs of the cluster send: maxima and sums, and their share of the outputs this CTA adds up
  __shared__ float2 in_ml[kMaxC][kHeads];
  __shared__ float in_o[kHeads * DH];
  __shared__ float2 f[kHeads];                   // the cluster's maxima, and sums inverted
  __shared__ float rank_factor[kMaxC][kHeads];
  grid_dep_trigger();
  grid_dep_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int C = gridDim.x, rank = blockIdx.x;
  const spatten_kv4_attn_args& a = args.a;
  const spatten_kv4_cache& c = a.cache;
  const int hk = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.H / c.H_kv;
  // the query's loads go out first: what follows them waits for the length
  typename W::Raw raw;
  const T* qrow = static_cast<const T*>(a.q) + b * a.q_ld + static_cast<int64_t>(hk) * group * DH;
  if (warp < W::kPrepareWarps) raw.load(qrow, warp / G32, min(kHeads, group), lane);
  const int n_all = clamp_len(a.len[b], a.n_max, a.dev_status);
  const int run = (((n_all + C - 1) / C) + TK - 1) / TK * TK;   // keys per CTA
  const int first = min(n_all, rank * run), n = min(run, n_all - first);
  const int64_t row0 = (static_cast<int64_t>(b) * c.H_kv + hk) * c.cap + first;
  const int64_t x_ld = args.x_ld;
  float* x = args.x ? args.x + ((static_cast<int64_t>(b) * c.H_kv + hk) * C + rank) * args.heads * x_ld
                    : reinterpret_cast<float*>(smem + ring_bytes(DH, NH));
  if (!a.update_weight) x = nullptr;

  Run<DH> way(c, smem, warp, lane);
  if (C > 1) cluster.barrier_arrive();   // this CTA runs: its shared memory can be written
  for (int h0 = 0; h0 < group; h0 += kHeads) {
    const int heads = min(kHeads, group - h0);
    way.start(row0, n);
    if (warp < W::kPrepareWarps) {
      if (h0) raw.load(qrow + static_cast<int64_t>(h0) * DH, warp / G32, heads, lane);
      W::prepare(query[warp / G32], raw, warp % G32, a.sm_scale, lane);
    }
    __syncthreads();
    W w;
    w.init(query, lane);
    way.process(w, x, x_ld, heads);
    const int share = heads * DH / C;   // the outputs that a CTA adds up
    merge_warps<DH, NH>(
        w, smem, s_m, s_l, heads, [&](int i) { return i < heads * C ? i % heads : -1; },   // maxima and sums to every CTA
        [&]() { if (C > 1 && h0 == 0) cluster.barrier_wait(); },                           // which all run by now
        [&](int h, float mx, float l) { *cluster.map_shared_rank(&in_ml[rank][h], tid / heads) = make_float2(mx, l); },
        [&](int e, float v) {
          const int to = e / share;
          *cluster.map_shared_rank(&in_o[rank * share + (e - to * share)], to) = v;
        });
    if (C > 1) cluster.sync();
    else __syncthreads();
    // the cluster's sums, in rank order
    if (tid < heads) {
      float2 ml[kMaxC];
      float mx = -INFINITY, l = 0.0f;
#pragma unroll
      for (int r = 0; r < kMaxC; ++r) ml[r] = r < C ? in_ml[r][tid] : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int r = 0; r < kMaxC; ++r) mx = fmaxf(mx, ml[r].x);
      const float base = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
      for (int r = 0; r < kMaxC; ++r) {
        const float g = ex2(ml[r].x - base);
        l = fmaf(ml[r].y, g, l);
        rank_factor[r][tid] = g;
      }
      f[tid] = make_float2(base, l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l));   // an empty sequence gives 0, NaN stays
    }
    __syncthreads();
    for (int e = tid; e < share; e += kThreads) {
      const int h = (rank * share + e) / DH;
      float v = 0.0f;
#pragma unroll
      for (int r = 0; r < kMaxC; ++r)
        if (r < C) v = fmaf(in_o[r * share + e], rank_factor[r][h], v);
      st_from_float(static_cast<T*>(a.o) + b * a.o_ld + (static_cast<int64_t>(hk) * group + h0) * DH + rank * share + e, v * f[h].y);
    }
    if (x) {
      constexpr int kU = 4;   // rows in flight
      for (int i0 = tid; i0 < n; i0 += kU * kThreads) {
        float w0[kU], v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          w0[u] = i0 + u * kThreads < n ? c.weight[row0 + i0 + u * kThreads] : 0.0f;
          v[u] = 0.0f;
        }
#pragma unroll 2
        for (int h = 0; h < heads; ++h) {
          const float2 fh = f[h];
          const float* xh = x + h * x_ld + i0;
#pragma unroll
          for (int u = 0; u < kU; ++u)
            if (i0 + u * kThreads < n) v[u] = fmaf(ex2(xh[u * kThreads] - fh.x), fh.y, v[u]);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (i0 + u * kThreads < n) c.weight[row0 + i0 + u * kThreads] = w0[u] + v[u];
      }
    }
    if (h0 + kHeads < group) {   // the next heads' sums arrive once every CTA has read these
      if (C > 1) cluster.sync();
      else __syncthreads();
    }
  }
}

// ---- the split form: more keys than one wave of clusters holds ----------------------------------------
// All tiles of all (sequence, head) pairs, in order, are dealt to the CTAs in equal runs (two CTAs an SM; a run of
// one pair is a segment), so that no CTA waits for others and the work is even whatever the lengths are.  A CTA's
// segment of pair p leaves its maxima, sums and outputs in slot CTA + p; the scores go to the workspace.  A second
// kernel adds up and makes the weights.
struct Deal {
  int64_t total;   // tiles
  int N;
  __device__ __forceinline__ int64_t begin(int cta) const { return cta * total / N; }
};
template <int TK>
__device__ __forceinline__ int tiles_of(const spatten_kv4_attn_args& a, int b) {
  const int n = b < a.cache.B ? max(0, min(a.n_max, a.len[b])) : 0;
  return (n + TK - 1) / TK;
}
// tiles of sequences b < end, per head; whole warps
template <int TK>
__device__ __forceinline__ int64_t tiles_before(const spatten_kv4_attn_args& a, int end) {
  int64_t sum = 0;
  for (int b0 = 0; b0 < end; b0 += 32) {
    const int b = b0 + (threadIdx.x & 31);
    sum += __reduce_add_sync(0xffffffffu, b < end ? tiles_of<TK>(a, b) : 0);
  }
  return sum;
}

template <int DH, int NH, typename T>
__global__ void __launch_bounds__(kThreads, NH == 2 && sizeof(T) == 4 ? 1 : 2) kv4_attn_split_kernel(AttnArgs args) {
  using W = Warp<DH, NH, T>;
  constexpr int TK = W::TK, G32 = W::G32, kHeads = NH * 8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) typename W::Query query[NH];
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  grid_dep_trigger();
  grid_dep_wait();
  const spatten_kv4_attn_args& a = args.a;
  const spatten_kv4_cache& c = a.cache;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, group = a.H / c.H_kv, heads = min(kHeads, group - args.h0);
  if (blockIdx.x == 0 && args.h0 == 0)
    for (int b = tid; b < c.B; b += kThreads) clamp_len(a.len[b], a.n_max, a.dev_status);   // reports
  const Deal deal{tiles_before<TK>(a, c.B) * c.H_kv, static_cast<int>(gridDim.x)};
  int64_t at = deal.begin(blockIdx.x);
  const int64_t end = deal.begin(blockIdx.x + 1);
  if (at == end) return;
  // the sequence, head and tile of the first
  int b = 0, hk = 0, t0 = 0;
  {
    int64_t before = 0;
    for (int b0 = 0;; b0 += 32) {
      const int mine = tiles_of<TK>(a, b0 + lane);
      int inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, before + static_cast<int64_t>(inc) * c.H_kv > at);
      if (past) {
        const int l = __ffs(past) - 1;
        const int tiles = __shfl_sync(0xffffffffu, mine, l);
        const int64_t in = at - before - static_cast<int64_t>(__shfl_sync(0xffffffffu, inc - mine, l)) * c.H_kv;
        b = b0 + l;
        hk = static_cast<int>(in / tiles);
        t0 = static_cast<int>(in - static_cast<int64_t>(hk) * tiles);
        break;
      }
      before += static_cast<int64_t>(__shfl_sync(0xffffffffu, inc, 31)) * c.H_kv;
    }
  }
  Run<DH> way(c, smem, warp, lane);
  while (at < end) {
    const int n_all = max(0, min(a.n_max, a.len[b])), tiles = (n_all + TK - 1) / TK;
    if (t0 < tiles) {
      const int count = static_cast<int>(min(static_cast<int64_t>(tiles - t0), end - at));
      const int64_t pair = static_cast<int64_t>(b) * c.H_kv + hk;
      way.start(pair * c.cap + static_cast<int64_t>(t0) * TK, min(n_all - t0 * TK, count * TK));
      if (warp < W::kPrepareWarps) {
        typename W::Raw raw;
        raw.load(static_cast<const T*>(a.q) + b * a.q_ld + (static_cast<int64_t>(hk) * group + args.h0) * DH, warp / G32, heads, lane);
        W::prepare(query[warp / G32], raw, warp % G32, a.sm_scale, lane);
      }
      __syncthreads();
      W w;
      w.init(query, lane);
      way.process(w, args.x ? args.x + pair * args.heads * args.x_ld + static_cast<int64_t>(t0) * TK : nullptr, args.x_ld, heads);
      const int64_t slot = (blockIdx.x + pair) * args.heads;
      merge_warps<DH, NH>(
          w, smem, s_m, s_l, heads, [&](int i) { return i < heads ? i : -1; }, []() {},
          [&](int h, float mx, float l) { args.part_ml[slot + h] = make_float2(mx, l); },
          [&](int e, float v) { args.part_o[slot * DH + e] = v; });
      __syncthreads();   // the rings and the query are free again
      at += count;
    }
    t0 = 0;
    if (++hk == c.H_kv) hk = 0, ++b;
  }
}

constexpr int kFinishKeys = 4 * kThreads;
template <int DH, typename T>
__global__ void __launch_bounds__(kThreads) kv4_attn_finish_kernel(AttnArgs args) {
  constexpr int TK = kTileKeys<DH>;
  __shared__ float2 f[kMaxHeads];   // maxima, and sums inverted
  __shared__ int first_cta, ctas;
  __shared__ int64_t total;
  grid_dep_trigger();
  grid_dep_wait();
  const spatten_kv4_attn_args& a = args.a;
  const spatten_kv4_cache& c = a.cache;
  const int hk = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, group = a.H / c.H_kv, heads = min(args.heads, group - args.h0);
  const int n = max(0, min(a.n_max, a.len[b])), blocks = min(static_cast<int>(gridDim.x), max(1, (n + kFinishKeys - 1) / kFinishKeys));
  if (blockIdx.x >= blocks) return;
  const int64_t pair = static_cast<int64_t>(b) * c.H_kv + hk;
  if (tid < 32) {   // the CTAs that had tiles of this pair
    const Deal deal{tiles_before<TK>(a, c.B) * c.H_kv, args.ctas};
    const int tiles = (n + TK - 1) / TK;
    const int64_t from = tiles_before<TK>(a, b) * c.H_kv + static_cast<int64_t>(hk) * tiles;
    if (tid == 0) {
      int i = 0, k = 0;
      if (tiles) {
        i = static_cast<int>(from * args.ctas / deal.total);
        while (deal.begin(i + 1) <= from) ++i;
        while (deal.begin(i) > from) --i;
        while (i + k < args.ctas && deal.begin(i + k) < from + tiles) ++k;
      }
      first_cta = i;
      ctas = k;
      total = deal.total;
    }
  }
  __syncthreads();
  // with fewer tiles than CTAs some of these have none, and no slot: those whose runs are empty
  const int64_t slot0 = (first_cta + pair) * args.heads;
  const Deal deal{total, args.ctas};
  auto has = [&](int k) { return total >= args.ctas || deal.begin(first_cta + k + 1) > deal.begin(first_cta + k); };
  if (tid < heads) {
    float mx = -INFINITY, l = 0.0f;
    for (int k = 0; k < ctas; ++k)
      if (has(k)) mx = fmaxf(mx, args.part_ml[slot0 + k * args.heads + tid].x);
    const float base = mx == -INFINITY ? 0.0f : mx;
    for (int k = 0; k < ctas; ++k)
      if (has(k)) {
        const float2 ml = args.part_ml[slot0 + k * args.heads + tid];
        l = fmaf(ml.y, ex2(ml.x - base), l);
      }
    f[tid] = make_float2(base, l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l));   // an empty sequence gives 0, NaN stays
  }
  __syncthreads();
  for (int e = blockIdx.x * kThreads + tid; e < heads * DH; e += blocks * kThreads) {
    const int h = e / DH;
    float v = 0.0f;
    for (int k = 0; k < ctas; ++k)
      if (has(k)) v = fmaf(args.part_o[(slot0 + k * args.heads) * DH + e], ex2(args.part_ml[slot0 + k * args.heads + h].x - f[h].x), v);
    st_from_float(static_cast<T*>(a.o) + b * a.o_ld + (static_cast<int64_t>(hk) * group + args.h0) * DH + e, v * f[h].y);
  }
  if (!args.x) return;
  for (int i0 = blockIdx.x * kFinishKeys + tid; i0 < n; i0 += blocks * kFinishKeys) {
    float* weight = c.weight + pair * c.cap + i0;
    const float* x = args.x + pair * args.heads * args.x_ld + i0;
    float w0[4], v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      w0[u] = i0 + u * kThreads < n ? weight[u * kThreads] : 0.0f;
      v[u] = 0.0f;
    }
#pragma unroll 4
    for (int h = 0; h < heads; ++h) {
      const float2 fh = f[h];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + u * kThreads < n) v[u] = fmaf(ex2(x[h * args.x_ld + u * kThreads] - fh.x), fh.y, v[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * kThreads < n) weight[u * kThreads] = w0[u] + v[u];
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
  int64_t x_ld;
  int heads;
  size_t x_smem;   // bytes of scores in shared memory (0: none, or in the workspace)
  bool x_ws, split;
  int ctas;        // of the split form
};

// ring and scores (an SM has 228 KB, 1 KB of it per CTA reserved; a CTA's static arrays take up to 16 KB where two
// fit, else 20)
constexpr size_t kSharedTwo = (113 - 16) * 1024, kSharedOne = (227 - 20) * 1024;

// One launch of clusters: enough CTAs to fill the SMs, none with less than a tile per warp, and scores that let two
// CTAs share an SM where more CTAs achieve that.  What takes more than one wave of them, or has scores that fit no
// SM, is split instead (32 x 16384 rows, 8 heads of 128 with 4 queries each: 140 against 174 us; batches of
// more than 1024 sequences, through which every CTA would have to look, are not).
Shape shape(const spatten_kv4_attn_args& a) {
  Shape s{};
  const int tk = 2048 / a.cache.d_h;
  s.heads = std::min(a.H / a.cache.H_kv, kMaxHeads);
  const int64_t pairs = static_cast<int64_t>(a.cache.B) * a.cache.H_kv;
  auto ld = [&](int C) { return static_cast<int64_t>(align_up(static_cast<size_t>(ceil_div(a.n_max, C)), 32) + 4); };
  const size_t ring = ring_bytes(a.cache.d_h, s.heads > 8 ? 2 : 1);
  auto bytes = [&](int C) { return ring + (a.update_weight ? static_cast<size_t>(s.heads) * ld(C) * sizeof(float) : 0); };
  s.C = 1;
  while (s.C < kMaxC && a.n_max > s.C * kWarps * tk && (pairs * s.C < sm_count() || bytes(s.C) > kSharedTwo)) s.C *= 2;
  s.x_ws = bytes(s.C) > kSharedOne;
  const int per_sm = s.heads > 8 && a.dtype == SPATTEN_F32 ? 1 : 2;
  s.ctas = per_sm * sm_count();
  s.split = (pairs * s.C > s.ctas || s.x_ws) && a.cache.B <= 1024 && a.n_max > kWarps * tk;
  if (s.split) s.C = 1;
  s.x_ld = ld(s.C);
  s.x_smem = s.x_ws || s.split ? 0 : bytes(s.C) - ring;
  return s;
}

size_t layout(const spatten_kv4_attn_args& a, void* ws, size_t ws_bytes, AttnArgs* x) {
  const Shape s = shape(a);
  WsCursor c(ws, ws_bytes);
  const size_t pairs = static_cast<size_t>(a.cache.B) * a.cache.H_kv, slots = pairs + s.ctas;
  float* p = (s.x_ws || s.split) && a.update_weight ? c.take<float>(pairs * s.C * s.heads * s.x_ld) : nullptr;
  float2* ml = s.split ? c.take<float2>(slots * s.heads) : nullptr;
  float* o = s.split ? c.take<float>(slots * s.heads * a.cache.d_h) : nullptr;
  if (x) x->x = p, x->x_ld = s.x_ld, x->heads = s.heads, x->ctas = s.ctas, x->part_ml = ml, x->part_o = o;
  return align_up(std::max<size_t>(c.used, 1), 256);   // never 0: callers allocate it as it comes
}

template <int DH, int NH, typename T>
int32_t launch(AttnArgs x, const Shape& s, cudaStream_t st) {
  static DeviceOnce once;
  int dev;
  SPT_TRY(once_per_device(once, &dev, [](int) -> int32_t {
    SPT_CUDA(cudaFuncSetAttribute(kv4_attn_kernel<DH, NH, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSharedOne)));
    SPT_CUDA(cudaFuncSetAttribute(kv4_attn_split_kernel<DH, NH, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, ring_bytes(DH, NH)));
    return SPATTEN_OK;
  }));
  const spatten_kv4_cache& c = x.a.cache;
  if (!s.split)
    return launch_chained(kv4_attn_kernel<DH, NH, T>, dim3(s.C, c.H_kv, c.B), dim3(kThreads), ring_bytes(DH, NH) + s.x_smem, st, s.C, x);
  for (; x.h0 < x.a.H / c.H_kv; x.h0 += kMaxHeads) {
    SPT_TRY(launch_chained(kv4_attn_split_kernel<DH, NH, T>, dim3(s.ctas), dim3(kThreads), ring_bytes(DH, NH), st, 1, x));
    // about a wave of blocks: each looks its pair's CTAs up before it works through its keys
    const int64_t most = ceil_div(8 * sm_count(), static_cast<int64_t>(c.B) * c.H_kv);
    const dim3 grid(static_cast<unsigned>(std::min(ceil_div(x.a.n_max, kFinishKeys), most)), c.H_kv, c.B);
    SPT_TRY(launch_chained(kv4_attn_finish_kernel<DH, T>, grid, dim3(kThreads), 0, st, 1, x));
  }
  return SPATTEN_OK;
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
