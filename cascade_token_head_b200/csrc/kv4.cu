// The 4-bit cache: append (quantize new rows), read (rows back as values) and evict (give up the
// rows with the least attention weight).  Layout and rules: spatten.h.
#include <cooperative_groups.h>

#include <type_traits>

#include "kv4.cuh"

namespace cg = cooperative_groups;

namespace spt {

int32_t kv4_validate(const spatten_kv4_cache& c) {
  if (c.B < 1 || c.B > 65535 || c.H_kv < 1 || c.H_kv > 1024 || c.cap < 1) return SPATTEN_E_ARG;
  if (c.d_h != 64 && c.d_h != 128) return SPATTEN_E_UNSUPPORTED;
  if (!c.k_codes || !c.k_scale || !c.v_codes || !c.v_scale) return SPATTEN_E_ARG;
  if (!aligned16(c.k_codes) || !aligned16(c.k_scale) || !aligned16(c.v_codes) || !aligned16(c.v_scale) ||
      !aligned16(c.weight) || !aligned16(c.pos))
    return SPATTEN_E_ALIGN;
  return SPATTEN_OK;
}

namespace {

constexpr int kThreads = 256;

// ----------------------------------------------------------------------------------------------
// append
// ----------------------------------------------------------------------------------------------
struct AppendArgs {
  spatten_kv4_cache c;
  const void* x[2];   // K, V
  int64_t ld_tok;
  int32_t total;
  const int32_t* cu;
  const int32_t* len;
  int32_t* len_out;
  const int32_t* seen;
  int32_t* seen_out;
  int32_t* status;
};

// Eight channels as they are loaded.
struct Bf16x8 {
  static constexpr bool kEightBits = true;   // significands
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  // bits of the largest magnitude; a NaN counts as larger than infinity
  __device__ __forceinline__ uint32_t absmax() const {
    constexpr uint32_t M = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vmaxu2(u.x & M, u.y & M), __vmaxu2(u.z & M, u.w & M));
    return max(m << 16, m & 0xffff0000u);
  }
};
struct F32x8 {
  static constexpr bool kEightBits = false;
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ uint32_t absmax() const {
    float x[8];
    get(x);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    return m;
  }
};
template <typename T> struct Octet { using type = Bf16x8; };
template <> struct Octet<float> { using type = F32x8; };

// What quantize8 does, by IEEE divisions: the codes, and the scale's bits with bit 31 set where this lane
// held a value that is not finite.
template <typename X>
__device__ __noinline__ uint2 quantize8_by_division(X raw) {
  float x[8];
  raw.get(x);
  bool bad = false;
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (!isfinite(x[i])) {
      x[i] = 0.0f;
      bad = true;
    }
    amax = fmaxf(amax, fabsf(x[i]));
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(amax, 7.0f));
  if (__bfloat162float(sb) == 0.0f) sb = __float2bfloat16_rn(1.0f);
  const float s = __bfloat162float(sb);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int q = max(-7, min(7, __float2int_rn(__fdiv_rn(x[i], s))));
    w |= static_cast<uint32_t>(q + 8) << (4 * i);
  }
  return make_uint2(w, static_cast<uint32_t>(__bfloat16_as_ushort(sb)) | (bad ? 0x80000000u : 0u));
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Eight channels (one lane's share: a quarter of a 32-channel group) of one row to codes; the four
// lanes of the group share their amax; whole warps call it.  Returns the codes as nibbles (channel i at
// bits 4i) and the scale's bfloat16 bits.
// Both roundings are those of IEEE quotients.
//  float32   amax (1 / 7) is within 2 steps of the quotient, so both round to the same bfloat16 unless it
//    is that near to a border.  x / s is rounded as the quotient is by Markstein's theorem (1990): with
//    y = 1 / s rounded to nearest, q = x y and r = x - q s, which is exact, q + r y rounds to the nearest
//    x / s (s is no number of all ones: it has eight bits).
//  bfloat16  amax / 7 is never a border: that would have nine bits and its sevenfold more than eight; the
//    next quotients are 2^-12 away.  x and s have eight bits, and x is at least s / 4 near a half, so
//    |x / s - (k + 1/2)| = |2 x - (2 k + 1) s| / (2 s) is 0 or at least 1 / 1020.  x y (within 2^-19) rounded to
//    multiples of 2^-12 is therefore the half itself or on the quotient's side of it, and the second rounding,
//    to integers, is that of the quotient.
// Borders, values that are not finite and scales below 2^-100, where products underflow and the quotient may
// pass 7, are left to divisions (*divide); elsewhere the quotient is at most 7 (1 + 2^-8).  Dividing everywhere
// took 1.7 times as long (16,384 rows of 16 heads of 64).
template <typename X>
__device__ __forceinline__ uint32_t quantize8(const X& raw, uint32_t* scale_bits, bool* divide) {
  float x[8];
  raw.get(x);
  uint32_t am = raw.absmax();
  am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
  am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
  const uint32_t q7 = __float_as_uint(__uint_as_float(am) * (1.0f / 7.0f));
  uint32_t sb = (q7 + 0x7fffu + ((q7 >> 16) & 1u)) >> 16;   // to the nearest bfloat16
  const bool zero = am == 0;
  *divide = am >= 0x7f800000u || (!X::kEightBits && (q7 & 0xffffu) - 0x7ffcu <= 8u) || (sb < (27u << 7) && !zero);
  sb = zero ? 0x3f80u : sb;
  *scale_bits = sb;
  const float s = __uint_as_float(sb << 16), y = X::kEightBits ? rcp_approx(s) : __frcp_rn(s);
  const float2 y2 = make_float2(y, y), s2 = make_float2(-s, -s);
  constexpr float kCodeRound = 1.5f * 8388608.0f + 8.0f;   // 1.5 * 2^23 + 8: the sum's low bits are rint(x / s) + 8
  constexpr float kFine = 1.5f * 2048.0f;                  // sums with it are multiples of 2^-12
  const float2 up = make_float2(kCodeRound, kCodeRound), fine = make_float2(kFine, kFine);
  const float2 rest = make_float2(kCodeRound - kFine, kCodeRound - kFine);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 v = make_float2(x[i], x[i + 1]);
    float2 t;
    if constexpr (X::kEightBits) {
      t = __fadd2_rn(__ffma2_rn(v, y2, fine), rest);
    } else {
      const float2 q = __fmul2_rn(v, y2);
      t = __fadd2_rn(__ffma2_rn(__ffma2_rn(q, s2, v), y2, q), up);
    }
    // the sums' high bits are constants, which drop out at the end
    w += __float_as_uint(t.x) * (1u << (4 * i)) + __float_as_uint(t.y) * (16u << (4 * i));
  }
  constexpr uint32_t kHigh = 0x4b400000u * 0x11111111u;
  return w - kHigh;
}

// The lane's octet `oct` of a row as the row's words: K's word as it is; V's runs of four channels of two
// neighbouring groups make a word, so lanes of groups g and g ^ 1 (four lanes apart) trade halves and
// keep run 2t (even g) or 2t + 1.
template <int DH>
__device__ __forceinline__ uint32_t v_word(uint32_t w, int oct) {
  const bool odd = (oct >> 2) & 1;
  const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? w & 0xffffu : w >> 16, 4);
  return odd ? other | (w & 0xffff0000u) : (w & 0xffffu) | other << 16;
}
template <int DH>
__device__ __forceinline__ int k_word_at(int oct) {
  return (oct & 3) * (DH / 32) + (oct >> 2);
}
template <int DH>
__device__ __forceinline__ int v_word_at(int oct) {
  const int g = oct >> 2, run = 2 * (oct & 3) + (g & 1);
  return run * (DH / 64) + (g >> 1);
}

// Packed rows: a warp takes runs of kSteps * 256 / DH rows of one head, eight channels a lane and step, all
// loads before the first use: rows of a head are whole lines on both sides.  A warp waits for memory, then quantizes,
// and the warps that an SM holds hide half of that: 16,384 rows of 16 heads of 64 from bfloat16 (86 MB) take 24 us
// by themselves, 3.6 TB/s (issue slots 56 %), from float32 (153 MB) 33 us, 4.6 TB/s.  Loading V's values before K's
// are codes spilled and gave nothing.
template <int DH> constexpr int kRowLanes = DH / 8;
constexpr int kSteps = 4;
constexpr int kChunks = 2, kReadChunks = 1;   // runs a warp: blocks that look their rows up, against blocks to even out
template <int DH> constexpr int kStepRows = 32 / kRowLanes<DH>;
template <int DH> constexpr int kTaskRows = kSteps * kStepRows<DH>;
template <int DH, int CHUNKS> constexpr int kBlockRows = CHUNKS * kTaskRows<DH> * (kThreads / 32);   // of one sequence

// The rows i0 .. of sequence b (n rows from packed row `first`) that block blockIdx.x works on; b = -1: none.
// The whole block calls it, once.
struct BlockRows {
  int b, i0, first, n;
};
__device__ __forceinline__ BlockRows find_block_rows(const int32_t* cu, int B, int total, int rows) {
  __shared__ BlockRows sh;
  if (threadIdx.x < 32) {
    const SeqTile st = find_seq_tile<true>(cu, B, total, rows, blockIdx.x);
    const PackedRows p = st.b < 0 ? PackedRows{0, 0, false} : packed_rows(cu, st.b, total);
    if (threadIdx.x == 0) sh = {st.b, st.tile * rows, p.first, p.n};
  }
  __syncthreads();
  return sh;
}

// A run's rows once more by divisions (rare: out of the way of the loop's registers); x, codes and scale point
// to the lane's share of the first step.  Returns whether it held a value that is not finite; whole warps call it.
template <int DH, typename T>
__device__ __noinline__ bool append_by_division(const T* x, int64_t ld_tok, uint32_t* codes, uint16_t* scale, int fit, bool is_v) {
  const int lane = threadIdx.x & 31, oct = lane % kRowLanes<DH>, r = lane / kRowLanes<DH>;
  bool bad = false;
#pragma unroll 1
  for (int i = 0; i < kTaskRows<DH>; i += kStepRows<DH>) {
    const bool there = i + r < fit;
    typename Octet<T>::type v;
    if (there) v.load(x + i * ld_tok);
    else v.zero();
    const uint2 q = quantize8_by_division(v);
    const uint32_t w = is_v ? v_word<DH>(q.x, oct) : q.x;
    bad |= q.y >> 31;
    if (there) {
      codes[i * (DH / 8)] = w;
      if ((oct & 3) == 0) scale[i * (DH / kKv4Group)] = static_cast<uint16_t>(q.y);
    }
  }
  return bad;
}

template <int DH, typename T>
__global__ void __launch_bounds__(kThreads, 4) kv4_append_kernel(AppendArgs a, bool counts) {
  grid_dep_trigger();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, oct = lane % kRowLanes<DH>;
  // the counts, where no other block still reads them (len_out and seen_out are buffers of their own)
  if (counts && blockIdx.y == 0)
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; s < a.c.B; s += static_cast<int64_t>(gridDim.x) * kThreads) {
      const PackedRows p = packed_rows(a.cu, static_cast<int>(s), a.total);
      if (p.bad) report(a.status, SPATTEN_E_INDEX);
      const int old = clamp_len(a.len[s], a.c.cap, a.status), n = min(p.n, a.c.cap - old);
      a.len_out[s] = old + n;
      if (a.seen_out) a.seen_out[s] = a.seen[s] + n;
    }
  const int h = blockIdx.y;
  const BlockRows p = find_block_rows(a.cu, a.c.B, a.total, kBlockRows<DH, kChunks>);
  if (p.b < 0) return;
  constexpr int G = DH / kKv4Group;
  const int old = clamp_len(a.len[p.b], a.c.cap, a.status), r = lane / kRowLanes<DH>;
  const int64_t pair = (static_cast<int64_t>(p.b) * a.c.H_kv + h) * a.c.cap;
  bool bad = false;
#pragma unroll 1
  for (int c = 0; c < kChunks; ++c) {
    const int i0 = p.i0 + (c * (kThreads / 32) + static_cast<int>(threadIdx.x >> 5)) * kTaskRows<DH>;
    const int n = min(kTaskRows<DH>, p.n - i0);   // rows of the run
    const int room = a.c.cap - old - i0;          // of which these fit
    if (n > 0 && room < n && lane == 0) report(a.status, SPATTEN_E_INDEX);
    const int fit = min(n, room);
    if (fit <= 0) break;   // as for the runs behind
    const int64_t row0 = pair + old + i0, src = (static_cast<int64_t>(p.first) + i0 + r) * a.ld_tok + static_cast<int64_t>(h) * DH + oct * 8;
    auto run = [&](auto full, int t) {   // full: all rows of the run are there
      constexpr bool kFull = decltype(full)::value;
      const T* x = static_cast<const T*>(t ? a.x[1] : a.x[0]) + src;
      uint32_t* codes = reinterpret_cast<uint32_t*>(t ? a.c.v_codes : a.c.k_codes) + (row0 + r) * (DH / 8) + (t ? v_word_at<DH>(oct) : k_word_at<DH>(oct));
      uint16_t* scale = (t ? a.c.v_scale : a.c.k_scale) + (row0 + r) * G + (oct >> 2);
      typename Octet<T>::type v[kSteps];
      bool redo = false;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        if (kFull || k * kStepRows<DH> + r < fit) v[k].load(x + k * kStepRows<DH> * a.ld_tok);
        else v[k].zero();
      }
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        uint32_t sb;
        bool divide;
        uint32_t w = quantize8(v[k], &sb, &divide);
        if (t) w = v_word<DH>(w, oct);
        redo |= divide;
        if (kFull || k * kStepRows<DH> + r < fit) {
          codes[k * kStepRows<DH> * (DH / 8)] = w;
          if ((oct & 3) == 0) scale[k * kStepRows<DH> * G] = static_cast<uint16_t>(sb);
        }
      }
      if (__any_sync(0xffffffffu, redo)) bad |= append_by_division<DH>(x, a.ld_tok, codes, scale, fit, t);
    };
#pragma unroll 1   // unrolled it is too large for the instruction cache
    for (int t = 0; t < 2; ++t) {
      if (fit == kTaskRows<DH>) run(std::true_type{}, t);
      else run(std::false_type{}, t);
    }
    if (lane < fit) {
      if (a.c.weight) a.c.weight[row0 + lane] = 0.0f;
      if (a.c.pos) a.c.pos[row0 + lane] = a.seen[p.b] + i0 + lane;
    }
  }
  if (bad) report(a.status, SPATTEN_E_NONFINITE);
}

// The counts of a call whose outputs are its inputs, after the rows.
__global__ void __launch_bounds__(kThreads) kv4_counts_kernel(AppendArgs a) {
  grid_dep_trigger();
  grid_dep_wait();
  for (int s = blockIdx.x * kThreads + threadIdx.x; s < a.c.B; s += gridDim.x * kThreads) {
    const PackedRows p = packed_rows(a.cu, s, a.total);
    if (p.bad) report(a.status, SPATTEN_E_INDEX);
    const int old = clamp_len(a.len[s], a.c.cap, a.status), n = min(p.n, a.c.cap - old);
    a.len_out[s] = old + n;
    if (a.seen_out) a.seen_out[s] = a.seen[s] + n;
  }
}

// One row per sequence (a generated token): one block per sequence, which may therefore update the
// sequence's counts in place once its threads have read them.
template <int DH, typename T>
__global__ void __launch_bounds__(kThreads) kv4_append_token_kernel(AppendArgs a) {
  grid_dep_trigger();
  grid_dep_wait();
  constexpr int kLanes = DH / 8;
  const int b = blockIdx.x;
  const int row = clamp_len(a.len[b], a.c.cap, a.status);
  const int seen = a.seen ? a.seen[b] : 0;
  const bool room = row < a.c.cap;
  if (!room && threadIdx.x == 0) report(a.status, SPATTEN_E_INDEX);
  const int per_row = a.c.H_kv * kLanes, units = 2 * per_row;
  for (int u0 = 0; u0 < units; u0 += kThreads) {
    const int u = u0 + threadIdx.x;
    const int tensor = u >= per_row, rest = u - tensor * per_row, h = rest / kLanes, oct = rest % kLanes;
    const bool ok = room && u < units;
    const int64_t at = (static_cast<int64_t>(b) * a.c.H_kv + h) * a.c.cap + row;
    typename Octet<T>::type x;
    if (ok) x.load(static_cast<const T*>(a.x[tensor]) + b * a.ld_tok + static_cast<int64_t>(h) * DH + oct * 8);
    else x.zero();
    // per_row is a multiple of 8 lanes: a group's four lanes, and V's pairs of groups, have one tensor
    uint32_t sb;
    bool divide, bad = false;
    uint32_t w = quantize8(x, &sb, &divide);
    if (__any_sync(0xffffffffu, divide)) {
      const uint2 q = quantize8_by_division(x);
      w = q.x, sb = q.y & 0xffffu, bad = q.y >> 31;
    }
    const uint32_t v = v_word<DH>(w, oct);
    if (ok) {
      if (bad) report(a.status, SPATTEN_E_NONFINITE);
      uint32_t* codes = reinterpret_cast<uint32_t*>(tensor ? a.c.v_codes : a.c.k_codes) + at * (DH / 8);
      codes[tensor ? v_word_at<DH>(oct) : k_word_at<DH>(oct)] = tensor ? v : w;
      if ((oct & 3) == 0) (tensor ? a.c.v_scale : a.c.k_scale)[at * (DH / kKv4Group) + (oct >> 2)] = static_cast<uint16_t>(sb);
      if (oct == 0 && tensor == 0) {
        if (a.c.weight) a.c.weight[at] = 0.0f;
        if (a.c.pos) a.c.pos[at] = seen;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    a.len_out[b] = row + (room ? 1 : 0);
    if (a.seen_out) a.seen_out[b] = seen + (room ? 1 : 0);
  }
}

template <int DH, typename T>
int32_t append_launch(const AppendArgs& a, cudaStream_t st) {
  if (!a.cu) {
    return launch_chained(kv4_append_token_kernel<DH, T>, dim3(a.c.B), dim3(kThreads), 0, st, 1, a);
  }
  const bool apart = a.len_out != a.len && (!a.seen_out || a.seen_out != a.seen);
  if (a.total > 0) {
    // a sequence's rows end in at most one partial run, so this many cover any offsets
    const dim3 grid(a.total / kBlockRows<DH, kChunks> + a.c.B, a.c.H_kv);
    SPT_TRY(launch_chained(kv4_append_kernel<DH, T>, grid, dim3(kThreads), 0, st, 1, a, apart));
    if (apart) return SPATTEN_OK;
  }
  return launch_chained(kv4_counts_kernel, dim3(static_cast<unsigned>(ceil_div(a.c.B, kThreads))), dim3(kThreads), 0, st, 1, a);
}

// ----------------------------------------------------------------------------------------------
// read
// ----------------------------------------------------------------------------------------------
struct ReadArgs {
  spatten_kv4_cache c;
  const int32_t* cu;
  const int32_t* row0;
  int32_t total;
  void* out[2];
  int64_t ld_tok;
  int32_t* status;
};

// Stores the eight codes of a word times a scale (bfloat16 bits).
__device__ __forceinline__ void store_values(float* p, uint32_t w, uint32_t sb) {
  const float s = bf16_bits_to_float(sb);
  uint32_t x[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {   // 2^23 + u, less 2^23 + 8
    const float2 u = make_float2(__uint_as_float(((w >> (4 * i)) & 15u) | 0x4b000000u), __uint_as_float(((w >> (4 * i + 4)) & 15u) | 0x4b000000u));
    const float2 v = __fmul2_rn(__fadd2_rn(u, make_float2(-8388616.0f, -8388616.0f)), make_float2(s, s));
    x[i] = __float_as_uint(v.x), x[i + 1] = __float_as_uint(v.y);
  }
  // whole sectors where the address allows it (18 x 330 rows of 12 heads of 128, 73 MB: 14.9 us, halves 21.4)
  store32(p, x);
}
// In bfloat16 the code is exact and the product is rounded once, as the float32 product would be.
__device__ __forceinline__ void store_values(__nv_bfloat16* p, uint32_t w, uint32_t sb) {
  const uint32_t s2 = sb | sb << 16;
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // channels i, i + 4: 128 + u, less 136
    const uint32_t u = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    asm("{\n.reg .b32 t;\nadd.rn.bf16x2 t, %1, %2;\nmul.rn.bf16x2 %0, t, %3;\n}" : "=r"(v[i]) : "r"(u), "r"(0xc308c308u), "r"(s2));
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                                            __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}

// A warp takes the rows of one head as the append kernel does, all loads before the first use.  Three
// quarters of what memory copies: 16,384 rows of 16 heads of 64 to bfloat16 (86 MB) take 17 us, 5.0 TB/s, to float32
// (153 MB) 29 us, 5.2 TB/s; one run a warp, whose start and end nothing hides.
template <int DH, typename T>
__global__ void __launch_bounds__(kThreads, 6) kv4_read_kernel(ReadArgs a) {
  grid_dep_trigger();
  grid_dep_wait();
  constexpr int G = DH / kKv4Group;
  const int lane = threadIdx.x & 31, oct = lane % kRowLanes<DH>, g = oct >> 2;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int b = threadIdx.x; b < a.c.B; b += kThreads)
      if (packed_rows(a.cu, b, a.total).bad) report(a.status, SPATTEN_E_INDEX);
  const int h = blockIdx.y;
  const BlockRows p = find_block_rows(a.cu, a.c.B, a.total, kBlockRows<DH, kReadChunks>);
  if (p.b < 0) return;
  const int row0 = a.row0 ? a.row0[p.b] : 0, r = lane / kRowLanes<DH>;
  const int64_t pair = (static_cast<int64_t>(p.b) * a.c.H_kv + h) * a.c.cap;
#pragma unroll 1
  for (int c = 0; c < kReadChunks; ++c) {
    const int i0 = p.i0 + (c * (kThreads / 32) + static_cast<int>(threadIdx.x >> 5)) * kTaskRows<DH>;
    const int n = min(kTaskRows<DH>, p.n - i0);
    if (n <= 0) break;
    const int64_t first = static_cast<int64_t>(row0) + i0;   // cache row of the run's first
    const bool inside = first >= 0 && first + n <= a.c.cap;
    if (lane == 0 && !inside) report(a.status, SPATTEN_E_INDEX);
    const int64_t dst = (static_cast<int64_t>(p.first) + i0 + r) * a.ld_tok + static_cast<int64_t>(h) * DH + oct * 8;
    auto run = [&](auto full) {   // full: all rows of the run are there; else rows outside the cache read as 0
      constexpr bool kFull = decltype(full)::value;
      const int lo = first < -kTaskRows<DH> ? kTaskRows<DH> : max(0, -static_cast<int>(first));
      const int hi = first + n <= a.c.cap ? n : (first < a.c.cap ? static_cast<int>(a.c.cap - first) : 0);
      uint32_t w[2][kSteps], s[2][kSteps];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t* codes = reinterpret_cast<const uint32_t*>(t ? a.c.v_codes : a.c.k_codes) + (pair + first + r) * (DH / 8) +
                                (t ? v_word_at<DH>(oct) : k_word_at<DH>(oct));
        const uint16_t* scale = (t ? a.c.v_scale : a.c.k_scale) + (pair + first + r) * G + g;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const int i = k * kStepRows<DH> + r;
          const bool ok = kFull || (i >= lo && i < hi);
          w[t][k] = ok ? codes[k * kStepRows<DH> * (DH / 8)] : 0u;
          s[t][k] = ok ? scale[k * kStepRows<DH> * G] : 0u;
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        T* out = static_cast<T*>(a.out[t]);
        if (!out) continue;
        out += dst;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const uint32_t u = t ? v_word<DH>(w[t][k], oct) : w[t][k];
          if (kFull || k * kStepRows<DH> + r < n) store_values(out + k * kStepRows<DH> * a.ld_tok, u, s[t][k]);
        }
      }
    };
    if (inside && n == kTaskRows<DH>) run(std::true_type{});
    else run(std::false_type{});
  }
}

// ----------------------------------------------------------------------------------------------
// evict
// ----------------------------------------------------------------------------------------------
constexpr int kSelThreads = 1024;   // of the two-launch form

struct EvictArgs {
  spatten_kv4_cache s, d;
  const int32_t* len;
  int32_t* len_out;
  const int32_t* seen;
  int32_t n_max, keep, recent;
  bool in_place;
  // plan: per (b, h) the number of moves and the rows left, and the moves: dst[i] <- src[i] (in
  // place: the holes and the rows that fill them; else every kept row, dst[i] = i)
  int32_t* count;   // [B*H][2]
  int32_t* hole;    // [B*H][m]
  int32_t* tail;    // [B*H][m]
  int32_t* from;    // [B*H][keep] (not in place)
  int32_t m;        // min(keep, n_max - keep), at least 0
  int32_t* status;
};

// A row's rank as a number, larger first: rows with pos >= safe_from before all others, NaN weights last.
__device__ __forceinline__ uint32_t key_of(float w, int pos, int safe_from, bool has_safe) {
  return has_safe && pos >= safe_from ? 0xffffffffu : (isnan(w) ? 0u : float_key(w));
}
__device__ __forceinline__ uint32_t row_key(const EvictArgs& a, int64_t base, int j, int safe_from, bool has_safe) {
  return key_of(a.s.weight[base + j], has_safe ? a.s.pos[base + j] : 0, safe_from, has_safe);
}

// Inclusive prefix sum over a warp.
__device__ __forceinline__ int warp_scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}
// Sum of the counts of the warps before this one; *all: of all of them.  Every lane of a warp gives the
// warp's count.  One barrier; `sums` is not used again before the next one.
template <int THREADS>
__device__ __forceinline__ int before_warp(int count, int* sums, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) sums[warp] = count;
  __syncthreads();
  const int c = lane < THREADS / 32 ? sums[lane] : 0, inc = warp_scan(c);
  *all = __shfl_sync(0xffffffffu, inc, 31);
  return __shfl_sync(0xffffffffu, inc - c, warp);
}

struct Threshold {
  uint32_t key;   // the k-th largest key
  int ties;       // how many rows with this key stay,
  bool all;       // which are all of them
};

constexpr int kBins = 2048;   // digits of 11, 11 and 10 bits

// The k-th largest of n keys (1 <= k <= n) by three radix passes; get(j) gives the keys of rows j .. j + 3 (j a
// multiple of 4; any number past n); `hist` has kBins entries.
template <int THREADS, typename Get>
__device__ __forceinline__ Threshold radix_select(int n, int k, Get get, int* hist, int (*sums)[32]) {
  __shared__ Threshold found;
  const int tid = threadIdx.x;
  uint32_t prefix = 0;
  int want = k;
  bool all_stay = false;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bins = pass == 2 ? kBins / 2 : kBins;
    // thread t has the t-th `per` bins; bin b's count lies where the threads' i-th ones are neighbours
    const int per = bins / THREADS, log_per = 31 - __clz(per);
    auto place = [&](int b) { return (b & (per - 1)) * THREADS + (b >> log_per); };
    for (int i = tid; i < bins; i += THREADS) hist[i] = 0;
    __syncthreads();
    const uint32_t above = pass == 0 ? 0u : (pass == 1 ? ~0u << 21 : ~0u << 10);
#pragma unroll 2
    for (int j0 = 0; j0 < n; j0 += 4 * THREADS) {
      const int j = j0 + 4 * tid;
      const uint4 q = j < n ? get(j) : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t key[4] = {q.x, q.y, q.z, q.w};
      int bin[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        bin[u] = j + u < n && (key[u] & above) == prefix ? static_cast<int>((key[u] >> shift) & (bins - 1u)) : -1;
      // equal weights (a new cache's zeros) would queue up at one bin: a warp of one bin adds once
      int one;
      __match_all_sync(0xffffffffu, bin[0] == bin[1] && bin[0] == bin[2] && bin[0] == bin[3] ? bin[0] : -2 - (tid & 31), &one);
      if (one) {
        if (bin[0] >= 0 && (tid & 31) == 0) atomicAdd(&hist[place(bin[0])], 128);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (bin[u] >= 0) atomicAdd(&hist[place(bin[u])], 1);
      }
    }
    __syncthreads();
    // from the largest: thread t adds up those of thread THREADS - 1 - t
    int c[kBins / THREADS], sum = 0;
#pragma unroll
    for (int i = 0; i < kBins / THREADS; ++i) {
      c[i] = i < per ? hist[place(bins - 1 - tid * per - i)] : 0;
      sum += c[i];
    }
    const int inc = warp_scan(sum);
    int all;
    int before = before_warp<THREADS>(__shfl_sync(0xffffffffu, inc, 31), sums[pass & 1], &all) + inc - sum;
    if (before < want && want <= before + sum) {
#pragma unroll
      for (int i = 0; i < kBins / THREADS; ++i) {
        if (before < want && want <= before + c[i])
          found = {prefix | static_cast<uint32_t>(bins - 1 - tid * per - i) << shift, want - before, want == before + c[i]};
        before += c[i];
      }
    }
    __syncthreads();
    prefix = found.key;
    want = found.ties;
    all_stay = found.all;
  }
  return {prefix, want, all_stay};
}

// Of flags in row order (four rows a lane, bit u of `bits` the u-th): how many are set in the lanes before
// this one; *total: in the warp.
__device__ __forceinline__ int flags_before(uint32_t bits, int* total) {
  const uint32_t below = (1u << (threadIdx.x & 31)) - 1u;
  int before = 0;
  *total = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint32_t m = __ballot_sync(0xffffffffu, (bits >> u) & 1u);
    before += __popc(m & below);
    *total += __popc(m);
  }
  return before;
}

// Ranks the rows in their order, each warp a run of them, each lane rows j .. j + 3: low(j, holes, i) names the
// rows below k among them that go (bits of `holes`), the first of which is the i-th such row of all;
// high(j, tails, i) so the rows from k on that stay.  Returns the number of either.
template <int THREADS, typename Get, typename Low, typename High>
__device__ __forceinline__ int rank_rows(int n, int k, Threshold th, Get get, int (*sums)[32], Low low_rows, High high_rows) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int run = (n + 4 * THREADS - 1) / (4 * THREADS) * 128, j0 = min(n, warp * run), j1 = min(n, j0 + run);
  // rows j .. j + 3 of a lane: which have the threshold's key, and which a larger one
  auto compare = [&](int j, uint32_t& ties) {
    const uint4 q = j < j1 ? get(j) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t key[4] = {q.x, q.y, q.z, q.w};
    uint32_t larger = 0;
    ties = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      larger |= (j + u < j1 && key[u] > th.key ? 1u : 0u) << u;
      ties |= (j + u < j1 && key[u] == th.key ? 1u : 0u) << u;
    }
    return larger;
  };
  int t0 = 0, all;
  if (!th.all) {   // of the ties the first ones stay: they are ranked first
    int ties = 0;
    for (int jw = j0; jw < j1; jw += 128) {
      uint32_t bits;
      compare(jw + 4 * lane, bits);
      ties += __popc(bits);
    }
    t0 = before_warp<THREADS>(warp_sum_int(ties), sums[0], &all);
  }
  auto kept_rows = [&](int j, int& t) {
    uint32_t ties;
    const uint32_t larger = compare(j, ties);
    if (th.all) return larger | ties;
    int total, r = t + flags_before(ties, &total);
    t += total;
    uint32_t kept = larger;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if ((ties >> u) & 1u) kept |= (r++ < th.ties ? 1u : 0u) << u;
    return kept;
  };
  // masks of the rows below k, and of the rows there are
  auto rows_to = [&](int j, int end) { return (1u << max(0, min(4, end - j))) - 1u; };
  int holes = 0, tails = 0, t = t0;
  for (int jw = j0; jw < j1; jw += 128) {
    const int j = jw + 4 * lane;
    const uint32_t kept = kept_rows(j, t), low = rows_to(j, min(k, j1));
    holes += __popc(low & ~kept);
    tails += __popc(kept & ~rows_to(j, k));
  }
  int moved;
  int h = before_warp<THREADS>(warp_sum_int(holes), sums[1], &moved), w = before_warp<THREADS>(warp_sum_int(tails), sums[2], &all);
  t = t0;
  for (int jw = j0; jw < j1; jw += 128) {
    const int j = jw + 4 * lane;
    const uint32_t kept = kept_rows(j, t), low = rows_to(j, min(k, j1));
    const uint32_t is_hole = low & ~kept, is_tail = kept & ~rows_to(j, k);
    int n_hole, n_tail;
    if (jw < k) {
      low_rows(j, is_hole, h + flags_before(is_hole, &n_hole));
      h += n_hole;
    }
    if (jw + 128 > k) {
      high_rows(j, is_tail, w + flags_before(is_tail, &n_tail));
      w += n_tail;
    }
  }
  return moved;
}

// Moves rows i < n of a (sequence, head): rows(i, &to, &from) names them; thread `me` of `threads`.  First
// the codes, 16-byte pieces of K and V side by side, then words: the scales, the weight, the position.  Lanes
// of one kind of piece in separate branches would wait for memory once a kind; so they differ by pointers.
template <int DH, typename Rows>
__device__ __forceinline__ void move_rows(const EvictArgs& a, int64_t s_base, int64_t d_base, int n, int me, int threads, Rows rows) {
  {
    constexpr int kCode = DH / 32, kLanes = 2 * kCode, kU = 4;
    const int piece = me % kLanes, step = threads / kLanes;
    const bool v = piece >= kCode;
    const uint4* src = reinterpret_cast<const uint4*>(v ? a.s.v_codes : a.s.k_codes) + s_base * kCode + piece % kCode;
    uint4* dst = reinterpret_cast<uint4*>(v ? a.d.v_codes : a.d.k_codes) + d_base * kCode + piece % kCode;
    for (int i0 = me / kLanes; i0 < n; i0 += kU * step) {
      uint4 x[kU];
      int to[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        int from;
        to[u] = -1;
        if (i0 + u * step < n) {
          rows(i0 + u * step, to[u], from);
          x[u] = src[static_cast<int64_t>(from) * kCode];
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (to[u] >= 0) dst[static_cast<int64_t>(to[u]) * kCode] = x[u];
    }
  }
  {
    constexpr int kScale = DH / 64, kLanes = DH == 64 ? 4 : 8, kU = 8;   // words of a row's scales; 128 channels: 6 in use
    const int piece = me % kLanes, step = threads / kLanes;
    const bool v = piece >= kScale, scale = piece < 2 * kScale, weight = piece == 2 * kScale;
    const int width = scale ? kScale : 1, at = scale ? piece % kScale : 0;
    const uint32_t* src = scale ? reinterpret_cast<const uint32_t*>(v ? a.s.v_scale : a.s.k_scale)
                                : (weight ? reinterpret_cast<const uint32_t*>(a.s.weight) : reinterpret_cast<const uint32_t*>(a.s.pos));
    uint32_t* dst = scale ? reinterpret_cast<uint32_t*>(v ? a.d.v_scale : a.d.k_scale)
                          : (weight ? reinterpret_cast<uint32_t*>(a.d.weight) : reinterpret_cast<uint32_t*>(a.d.pos));
    if (piece > 2 * kScale + 1 || !src) n = 0;
    src += s_base * width + at;
    dst += d_base * width + at;
    for (int i0 = me / kLanes; i0 < n; i0 += kU * step) {
      uint32_t x[kU];
      int to[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        int from;
        to[u] = -1;
        if (i0 + u * step < n) {
          rows(i0 + u * step, to[u], from);
          x[u] = src[static_cast<int64_t>(from) * width];
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (to[u] >= 0) dst[static_cast<int64_t>(to[u]) * width] = x[u];
    }
  }
}

__device__ __forceinline__ void report_nan(const EvictArgs& a, int64_t base, int n) {
  bool bad = false;
  for (int j = threadIdx.x; j < n; j += kSelThreads) bad |= isnan(a.s.weight[base + j]);
  if (bad) report(a.status, SPATTEN_E_NONFINITE);
}

// One launch: a cluster per (sequence, head).  Each of its CTAs selects on its own, from keys in shared memory
// (so that nothing but the end of the selection has to be agreed on), and then moves its share of the rows.
// The work per row is small; latency bounds it: the passes of the radix select, the ranks and then the moves
// follow each other (16 x 16 heads of 1152 rows of 64 to 576: 16 us, 5 of them passes and ranks; 4 x 8 heads of
// 16,384 rows of 128 to 4096: 30 us).
template <int DH, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) kv4_evict_kernel(EvictArgs a) {
  grid_dep_trigger();
  grid_dep_wait();
  extern __shared__ __align__(16) uint32_t keys[];   // [n_max] keys (to a multiple of 4), then the lists
  __shared__ int hist[kBins], sums[3][32];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = gridDim.x, rank = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, k = a.keep;
  const int64_t bh = static_cast<int64_t>(b) * a.s.H_kv + h, base = bh * a.s.cap, d_base = bh * a.d.cap;
  const int n = clamp_len(a.len[b], a.n_max, a.status);
  if (a.len_out != a.len && rank == 0 && h == 0 && tid == 0) a.len_out[b] = min(n, k);
  int* tail = reinterpret_cast<int*>(keys) + (a.n_max + 3) / 4 * 4;   // [m]
  int* list = tail + (a.m + 3) / 4 * 4;   // in place [m]: the holes; else [keep]: row, or -1 - i for the i-th hole
  int moves = a.in_place ? 0 : n;
  const bool select = n > k;
  if (select) {
    const bool has_safe = a.recent > 0;
    const int safe_from = has_safe ? a.seen[b] - a.recent : 0;
    bool bad = false;
    for (int j0 = tid; j0 < n; j0 += 8 * THREADS) {
      float w[8];
      int pos[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {   // all loads before the first use
        const int j = j0 + u * THREADS;
        w[u] = j < n ? a.s.weight[base + j] : 0.0f;
        pos[u] = j < n && has_safe ? a.s.pos[base + j] : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int j = j0 + u * THREADS;
        bad |= isnan(w[u]);
        if (j < n) keys[j] = key_of(w[u], pos[u], safe_from, has_safe);
      }
    }
    if (bad && rank == 0) report(a.status, SPATTEN_E_NONFINITE);
    auto get = [&](int j) { return *reinterpret_cast<const uint4*>(keys + j); };
    const Threshold th = radix_select<THREADS>(n, k, get, hist, sums);   // its first barrier: the keys are there
    const bool in_place = a.in_place;
    moves = rank_rows<THREADS>(
        n, k, th, get, sums,
        [&](int j, uint32_t holes, int i) {
          if (in_place) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if ((holes >> u) & 1u) list[i++] = j + u;
          } else if (j < k) {   // whole words: the list is padded to a multiple of four
            int x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const bool hole = (holes >> u) & 1u;
              x[u] = hole ? -1 - i : j + u;
              i += hole;
            }
            *reinterpret_cast<int4*>(list + j) = make_int4(x[0], x[1], x[2], x[3]);
          }
        },
        [&](int j, uint32_t tails, int i) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if ((tails >> u) & 1u) tail[i++] = j + u;
        });
    if (!in_place) moves = k;
  }
  if (C > 1 && a.in_place) cluster.sync();   // every CTA has read the weights and positions
  else __syncthreads();
  move_rows<DH>(a, base, d_base, moves, rank * THREADS + tid, C * THREADS,
                [&](int i, int& to, int& from) {
                  if (a.in_place) {
                    to = list[i];
                    from = tail[i];
                  } else {
                    const int f = select ? list[i] : i;
                    to = i;
                    from = f < 0 ? tail[-1 - f] : f;
                  }
                });
}

__global__ void __launch_bounds__(kThreads) kv4_evict_counts_kernel(EvictArgs a) {
  grid_dep_trigger();
  grid_dep_wait();
  for (int b = blockIdx.x * kThreads + threadIdx.x; b < a.s.B; b += gridDim.x * kThreads)
    a.len_out[b] = min(clamp_len(a.len[b], a.n_max, nullptr), a.keep);
}

// Caches whose keys and lists do not fit shared memory: one CTA per (sequence, head) selects from the weights
// themselves and writes the moves to the workspace, a second launch moves.
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(EvictArgs a) {
  grid_dep_trigger();
  grid_dep_wait();
  __shared__ int hist[kBins], sums[3][32];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int64_t bh = static_cast<int64_t>(b) * a.s.H_kv + h, base = bh * a.s.cap;
  const int n = clamp_len(a.len[b], a.n_max, a.status), k = a.keep;
  int32_t* from = a.from + bh * a.keep;
  int moved = 0;
  if (n > k) {
    const bool has_safe = a.recent > 0;
    const int safe_from = has_safe ? a.seen[b] - a.recent : 0;
    int32_t *hole = a.hole + bh * a.m, *tail = a.tail + bh * a.m;
    report_nan(a, base, n);
    auto get = [&](int j) {
      uint32_t key[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) key[u] = row_key(a, base, min(j + u, n - 1), safe_from, has_safe);
      return make_uint4(key[0], key[1], key[2], key[3]);
    };
    const Threshold th = radix_select<kSelThreads>(n, k, get, hist, sums);
    const bool in_place = a.in_place;
    moved = rank_rows<kSelThreads>(
        n, k, th, get, sums,
        [&](int j, uint32_t holes, int i) {
          for (int u = 0; u < 4; ++u) {
            if ((holes >> u) & 1u) hole[i++] = j + u;
            else if (!in_place && j + u < k) from[j + u] = j + u;
          }
        },
        [&](int j, uint32_t tails, int i) {
          for (int u = 0; u < 4; ++u)
            if ((tails >> u) & 1u) tail[i++] = j + u;
        });
    __syncthreads();
    if (!a.in_place)
      for (int i = tid; i < moved; i += kSelThreads) from[hole[i]] = tail[i];
  } else if (!a.in_place) {
    for (int i = tid; i < n; i += kSelThreads) from[i] = i;
  }
  if (tid == 0) {
    a.count[2 * bh] = a.in_place ? moved : min(n, k);
    a.count[2 * bh + 1] = min(n, k);
  }
}

template <int DH>
__global__ void __launch_bounds__(kThreads) kv4_move_kernel(EvictArgs a) {
  grid_dep_trigger();
  grid_dep_wait();
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t bh = static_cast<int64_t>(b) * a.s.H_kv + h;
  const int n = a.count[2 * bh];
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) a.len_out[b] = a.count[2 * bh + 1];
  move_rows<DH>(a, bh * a.s.cap, bh * a.d.cap, n, blockIdx.x * kThreads + threadIdx.x, gridDim.x * kThreads, [&](int i, int& to, int& from) {
                  to = a.in_place ? a.hole[bh * a.m + i] : i;
                  from = a.in_place ? a.tail[bh * a.m + i] : a.from[bh * a.keep + i];
                });
}

bool same_cache(const spatten_kv4_cache& a, const spatten_kv4_cache& b) {
  return a.cap == b.cap && a.k_codes == b.k_codes && a.k_scale == b.k_scale && a.v_codes == b.v_codes &&
         a.v_scale == b.v_scale && a.weight == b.weight && a.pos == b.pos;
}
bool any_shared(const spatten_kv4_cache& a, const spatten_kv4_cache& b) {
  return a.k_codes == b.k_codes || a.k_scale == b.k_scale || a.v_codes == b.v_codes || a.v_scale == b.v_scale ||
         (a.weight && a.weight == b.weight) || (a.pos && a.pos == b.pos);
}

// shared memory of the one-launch kernel: keys and lists (17 KB of static arrays besides)
size_t evict_shared(int32_t n_max, int32_t keep, int32_t m) {
  return 4 * (align_up(n_max, 4) + align_up(m, 4) + align_up(keep > m ? keep : m, 4));
}
constexpr size_t kEvictShared = 208 * 1024;

size_t evict_layout(const spatten_kv4_cache& c, int32_t n_max, int32_t keep, void* ws, size_t ws_bytes, EvictArgs* out) {
  WsCursor cur(ws, ws_bytes);
  const size_t bh = static_cast<size_t>(c.B) * c.H_kv;
  const int32_t m = n_max > keep ? (n_max - keep < keep ? n_max - keep : keep) : 0;
  int32_t* count = cur.take<int32_t>(2 * bh);
  int32_t* hole = cur.take<int32_t>(bh * m);
  int32_t* tail = cur.take<int32_t>(bh * m);
  int32_t* from = cur.take<int32_t>(bh * keep);
  if (out) {
    out->count = count;
    out->hole = hole;
    out->tail = tail;
    out->from = from;
    out->m = m;
  }
  return align_up(cur.used, 256);
}

template <int DH, int THREADS>
int32_t evict_one_launch(const EvictArgs& a, int C, size_t shared, cudaStream_t st) {
  static DeviceOnce once;
  int dev;
  SPT_TRY(once_per_device(once, &dev, [](int) -> int32_t {
    SPT_CUDA(cudaFuncSetAttribute(kv4_evict_kernel<DH, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kEvictShared)));
    return SPATTEN_OK;
  }));
  SPT_TRY(launch_chained(kv4_evict_kernel<DH, THREADS>, dim3(C, a.s.H_kv, a.s.B), dim3(THREADS), shared, st, C, a));
  if (a.len_out != a.len) return SPATTEN_OK;
  return launch_chained(kv4_evict_counts_kernel, dim3(static_cast<unsigned>(ceil_div(a.s.B, kThreads))), dim3(kThreads), 0, st, 1, a);
}

template <int DH>
int32_t evict_launch(const EvictArgs& a, cudaStream_t st) {
  const int64_t rows = a.in_place ? a.m : a.keep, pairs = static_cast<int64_t>(a.s.B) * a.s.H_kv;
  const size_t shared = evict_shared(a.n_max, a.keep, a.m);
  if (shared <= kEvictShared) {
    // More CTAs while SMs are free and each has rows enough to move (half of 600 rows of 64, 64 heads: 8.2 us, with two
    // CTAs a head 9.8; half of 2500 of 128, 8 heads: 16.3, with eight 10.6).  Clusters of eight wait for SMs of one
    // part of the GPU and are taken up to 64 CTAs (16 heads, half of 10,000 rows of 128: 35.6, in fours 21.9; 8 heads
    // 18.6, in fours 21.7).  Large CTAs where one has an SM to itself and the rows or the CTAs are many (32 heads, half
    // of 10,000 rows: 22.3 against 32.6 with the middle size; 128 heads, half of 1200: 12.3 against 14.7; but 8 heads,
    // half of 600: 9.5 against 7.7); small ones, of which an SM holds four, where two an SM do not hold them all (512
    // heads, 1000 rows of 64 to 500: 33.9 against 39.5 with the middle size; 64 rows to 32: 13.5 against 19.7; but 224
    // heads, 2585 rows: 33.0 against 28.4).
    int C = 1;
    while (C < 8 && pairs * C * 2 <= (C < 4 ? sm_count() : 64) && rows >= 256 * C) C *= 2;
    if (pairs * C <= sm_count() && (a.n_max > 2048 || pairs * C > 64)) return evict_one_launch<DH, 1024>(a, C, shared, st);
    return pairs * C <= 2 * sm_count() ? evict_one_launch<DH, 512>(a, C, shared, st) : evict_one_launch<DH, 256>(a, C, shared, st);
  }
  SPT_TRY(launch_chained(kv4_select_kernel, dim3(a.s.H_kv, a.s.B), dim3(kSelThreads), 0, st, 1, a));
  // a few rows per thread group when there are many
  const int per_block = kThreads / (DH / 16);
  const int64_t want = ceil_div(rows, per_block), most = ceil_div(8 * sm_count(), pairs);
  const dim3 grid(static_cast<unsigned>(want < 1 ? 1 : (want < most ? want : most)), a.s.H_kv, a.s.B);
  return launch_chained(kv4_move_kernel<DH>, grid, dim3(kThreads), 0, st, 1, a);
}

}  // namespace
}  // namespace spt

extern "C" int32_t spatten_kv4_append(const spatten_kv4_cache* c, const void* k, const void* v, int32_t dtype,
                                      int64_t ld_tok, int32_t total, const int32_t* cu, const int32_t* len,
                                      int32_t* len_out, const int32_t* seen, int32_t* seen_out,
                                      int32_t* dev_status, void* stream) {
  spt::AbiRange nvtx_range("spatten_kv4_append");
  using namespace spt;
  if (!c || (total != 0 && (!k || !v)) || !len || !len_out) return SPATTEN_E_ARG;
  SPT_TRY(kv4_validate(*c));
  if (dtype != SPATTEN_F32 && dtype != SPATTEN_BF16) return SPATTEN_E_ARG;
  if (total < 0) return SPATTEN_E_ARG;
  if (!cu && total != c->B) return SPATTEN_E_SHAPE;
  if (c->pos && !seen) return SPATTEN_E_ARG;
  if ((seen == nullptr) != (seen_out == nullptr)) return SPATTEN_E_ARG;
  if (ld_tok < static_cast<int64_t>(c->H_kv) * c->d_h) return SPATTEN_E_SHAPE;
  const int esz = dtype == SPATTEN_BF16 ? 2 : 4;
  if (!aligned16(k) || !aligned16(v) || (ld_tok * esz) % 16 != 0) return SPATTEN_E_ALIGN;
  const AppendArgs a{*c, {k, v}, ld_tok, total, cu, len, len_out, seen, seen_out, dev_status};
  if (c->d_h == 64)
    return dtype == SPATTEN_BF16 ? append_launch<64, __nv_bfloat16>(a, as_stream(stream))
                                 : append_launch<64, float>(a, as_stream(stream));
  return dtype == SPATTEN_BF16 ? append_launch<128, __nv_bfloat16>(a, as_stream(stream))
                               : append_launch<128, float>(a, as_stream(stream));
}

extern "C" int32_t spatten_kv4_read(const spatten_kv4_cache* c, const int32_t* cu, const int32_t* row0, int32_t total,
                                    void* k_out, void* v_out, int32_t dtype, int64_t ld_tok, int32_t* dev_status,
                                    void* stream) {
  spt::AbiRange nvtx_range("spatten_kv4_read");
  using namespace spt;
  if (!c || !cu || (total != 0 && !k_out && !v_out)) return SPATTEN_E_ARG;
  SPT_TRY(kv4_validate(*c));
  if (dtype != SPATTEN_F32 && dtype != SPATTEN_BF16) return SPATTEN_E_ARG;
  if (total < 0) return SPATTEN_E_ARG;
  if (ld_tok < static_cast<int64_t>(c->H_kv) * c->d_h) return SPATTEN_E_SHAPE;
  const int esz = dtype == SPATTEN_BF16 ? 2 : 4;
  if (!aligned16(k_out) || !aligned16(v_out) || (ld_tok * esz) % 16 != 0) return SPATTEN_E_ALIGN;
  if (total == 0) return SPATTEN_OK;
  const ReadArgs a{*c, cu, row0, total, {k_out, v_out}, ld_tok, dev_status};
  const dim3 grid(total / (c->d_h == 64 ? kBlockRows<64, kReadChunks> : kBlockRows<128, kReadChunks>) + c->B, c->H_kv);
  const bool bf = dtype == SPATTEN_BF16;
  const auto kernel = c->d_h == 64 ? (bf ? kv4_read_kernel<64, __nv_bfloat16> : kv4_read_kernel<64, float>)
                                   : (bf ? kv4_read_kernel<128, __nv_bfloat16> : kv4_read_kernel<128, float>);
  return launch_chained(kernel, grid, dim3(kThreads), 0, as_stream(stream), 1, a);
}

extern "C" size_t spatten_kv4_evict_workspace_size(const spatten_kv4_cache* src, int32_t n_max, int32_t keep) {
  if (!src || src->B < 1 || src->H_kv < 1 || n_max < 1 || keep < 1) return 0;
  keep = keep < n_max ? keep : n_max;
  return spt::evict_layout(*src, n_max, keep, nullptr, 0, nullptr);
}

extern "C" int32_t spatten_kv4_evict(const spatten_kv4_cache* src, const spatten_kv4_cache* dst, const int32_t* len,
                                     int32_t* len_out, const int32_t* seen, int32_t n_max, int32_t keep,
                                     int32_t recent, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  spt::AbiRange nvtx_range("spatten_kv4_evict");
  using namespace spt;
  if (!src || !dst || !len || !len_out) return SPATTEN_E_ARG;
  SPT_TRY(kv4_validate(*src));
  SPT_TRY(kv4_validate(*dst));
  if (src->B != dst->B || src->H_kv != dst->H_kv || src->d_h != dst->d_h) return SPATTEN_E_SHAPE;
  if (n_max < 1 || keep < 1 || recent < 0 || recent > keep) return SPATTEN_E_ARG;
  if (n_max > src->cap || dst->cap < (keep < n_max ? keep : n_max)) return SPATTEN_E_SHAPE;
  if (!src->weight || !dst->weight || (src->pos && !dst->pos)) return SPATTEN_E_ARG;
  if (recent > 0 && (!src->pos || !seen)) return SPATTEN_E_ARG;
  keep = keep < n_max ? keep : n_max;   // no sequence of this call is longer
  EvictArgs a{*src, *dst, len, len_out, seen, n_max, keep, recent, same_cache(*src, *dst),
              nullptr, nullptr, nullptr, nullptr, 0, dev_status};
  if (!a.in_place && any_shared(*src, *dst)) return SPATTEN_E_ARG;
  if (!ws || ws_bytes < evict_layout(*src, n_max, keep, ws, ws_bytes, &a)) return SPATTEN_E_WORKSPACE;
  if (!aligned16(ws)) return SPATTEN_E_ALIGN;
  return src->d_h == 64 ? evict_launch<64>(a, as_stream(stream)) : evict_launch<128>(a, as_stream(stream));
}
