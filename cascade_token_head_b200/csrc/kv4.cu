// The 4-bit cache: append (quantize new rows), read (rows back as values) and evict (give up the
// rows with the least attention weight).  Layout and rules: spatten.h.
#include "kv4.cuh"

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

// Eight channels (one lane's share: a quarter of a 32-channel group) of one row to codes; the four
// lanes of the group share their amax; whole warps call it.  Returns the codes as nibbles (channel i at
// bits 4i) and the scale's bfloat16 bits.
// The code is rint(x / s) of the IEEE quotient.  The product with an approximate reciprocal is off by less
// than 2e-6 here, so its rounding is the quotient's unless it lies that near to a half; such lanes, and
// subnormal scales (where the quotient may pass 7), divide.
__device__ __forceinline__ uint32_t quantize8(float* x, uint32_t* scale_bits, bool* bad) {
  float z = 0.0f, amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) z = fmaf(x[i], 0.0f, z);   // NaN if any is not finite
  *bad = z != 0.0f;
  if (*bad)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = isfinite(x[i]) ? x[i] : 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(amax, 7.0f));
  if (__bfloat162float(sb) == 0.0f) sb = __float2bfloat16_rn(1.0f);
  const float s = __bfloat162float(sb);
  *scale_bits = __bfloat16_as_ushort(sb);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  constexpr float kRound = 12582912.0f + 8.0f;   // 1.5 * 2^23 + 8: the sum's low bits are rint(x / s) + 8
  uint32_t w = 0;
  float off = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = x[i] * inv, t = q + kRound;
    off = fmaxf(off, fabsf(q - (t - kRound)));
    w |= (__float_as_uint(t) & 15u) << (4 * i);
  }
  if (off > 0.499995f || s < 1.17549435e-38f) {
    w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = max(-7, min(7, __float2int_rn(__fdiv_rn(x[i], s))));
      w |= static_cast<uint32_t>(q + 8) << (4 * i);
    }
  }
  return w;
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

// Stores eight quantized channels of cache row `at` (over all heads and rows); whole warps call it, `ok`
// says whether this lane has a row.
template <int DH>
__device__ __forceinline__ void append8(const AppendArgs& a, int tensor, float* x, int64_t at, int oct, bool ok) {
  constexpr int G = DH / kKv4Group;
  uint32_t sb;
  bool bad;
  uint32_t w = quantize8(x, &sb, &bad);
  if (tensor) w = v_word<DH>(w, oct);
  if (!ok) return;
  if (bad) report(a.status, SPATTEN_E_NONFINITE);
  reinterpret_cast<uint32_t*>(tensor ? a.c.v_codes : a.c.k_codes)[at * (DH / 8) + (tensor ? v_word_at<DH>(oct) : k_word_at<DH>(oct))] = w;
  if ((oct & 3) == 0) (tensor ? a.c.v_scale : a.c.k_scale)[at * G + (oct >> 2)] = static_cast<uint16_t>(sb);
}

// Packed rows: a warp takes kSteps * 256 / DH rows of one head, eight channels a lane and step, all loads
// before the first use: rows of a head are whole lines on both sides.  Bound by memory and, next to it, by
// the quantization's instructions: 16,384 rows of 16 heads of 64 (bfloat16, 86 MB) take <T_APPEND>.
template <int DH> constexpr int kRowLanes = DH / 8;
constexpr int kSteps = 4;
template <int DH> constexpr int kTaskRows = kSteps * 32 / kRowLanes<DH>;

template <int DH, typename T>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(AppendArgs a, bool counts) {
  const int lane = threadIdx.x & 31, oct = lane % kRowLanes<DH>;
  // the counts, where no other block still reads them (len_out and seen_out are buffers of their own)
  if (counts)
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; s < a.c.B; s += static_cast<int64_t>(gridDim.x) * kThreads) {
      const PackedRows p = packed_rows(a.cu, static_cast<int>(s), a.total);
      if (p.bad) report(a.status, SPATTEN_E_INDEX);
      const int old = clamp_len(a.len[s], a.c.cap, a.status), n = min(p.n, a.c.cap - old);
      a.len_out[s] = old + n;
      if (a.seen_out) a.seen_out[s] = a.seen[s] + n;
    }
  const int64_t task = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int h = static_cast<int>(task % a.c.H_kv);
  const SeqTile st = find_seq_tile<true>(a.cu, a.c.B, a.total, kTaskRows<DH>, static_cast<int>(task / a.c.H_kv));
  if (st.b < 0) return;
  const PackedRows p = packed_rows(a.cu, st.b, a.total);
  const int old = clamp_len(a.len[st.b], a.c.cap, a.status);
  const int i0 = st.tile * kTaskRows<DH>, n = min(kTaskRows<DH>, p.n - i0);   // rows of the task
  const int room = a.c.cap - old - i0;                                        // of which these fit
  if (room < n && lane == 0) report(a.status, SPATTEN_E_INDEX);
  const int fit = min(n, room);
  if (fit <= 0) return;
  const int64_t src = (static_cast<int64_t>(p.first) + i0) * a.ld_tok + static_cast<int64_t>(h) * DH + oct * 8;
  const int64_t row0 = (static_cast<int64_t>(st.b) * a.c.H_kv + h) * a.c.cap + old + i0;
  float x[2][kSteps][8];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int r = k * (32 / kRowLanes<DH>) + lane / kRowLanes<DH>;
      if (r < fit) {
        load8(static_cast<const T*>(a.x[t]) + src + r * a.ld_tok, x[t][k]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[t][k][i] = 0.0f;
      }
    }
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int r = k * (32 / kRowLanes<DH>) + lane / kRowLanes<DH>;
      append8<DH>(a, t, x[t][k], row0 + r, oct, r < fit);
    }
  if (lane < fit) {
    if (a.c.weight) a.c.weight[row0 + lane] = 0.0f;
    if (a.c.pos) a.c.pos[row0 + lane] = a.seen[st.b] + i0 + lane;
  }
}

// The counts of a call whose outputs are its inputs, after the rows.
__global__ void __launch_bounds__(kThreads) kv4_counts_kernel(AppendArgs a) {
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
    float x[8] = {};
    if (ok) load8(static_cast<const T*>(a.x[tensor]) + b * a.ld_tok + static_cast<int64_t>(h) * DH + oct * 8, x);
    // per_row is a multiple of 8 lanes: a group's four lanes, and V's pairs of groups, have one tensor
    uint32_t sb;
    bool bad;
    const uint32_t w = quantize8(x, &sb, &bad), v = v_word<DH>(w, oct);
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
    kv4_append_token_kernel<DH, T><<<a.c.B, kThreads, 0, st>>>(a);
    return launch_status();
  }
  const bool apart = a.len_out != a.len && (!a.seen_out || a.seen_out != a.seen);
  if (a.total > 0) {
    // a sequence's rows end in at most one partial task, so this many cover any offsets
    const int64_t tasks = (static_cast<int64_t>(a.total) / kTaskRows<DH> + a.c.B) * a.c.H_kv, blocks = ceil_div(tasks, kThreads / 32);
    if (blocks > INT32_MAX) return SPATTEN_E_UNSUPPORTED;
    kv4_append_kernel<DH, T><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(a, apart);
    SPT_TRY(launch_status());
    if (apart) return SPATTEN_OK;
  }
  kv4_counts_kernel<<<static_cast<unsigned>(ceil_div(a.c.B, kThreads)), kThreads, 0, st>>>(a);
  return launch_status();
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

__device__ __forceinline__ void store8(float* p, const float* f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* f) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    r[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
}

// Eight codes in a word's nibbles, times s.
__device__ __forceinline__ void values8(uint32_t w, float s, float* x) {
#pragma unroll
  for (int i = 0; i < 8; ++i)   // 2^23 + u, less 2^23 + 8
    x[i] = s * (__uint_as_float(((w >> (4 * i)) & 15u) | 0x4b000000u) - 8388616.0f);
}

// A warp takes the rows of one head as the append kernel does, all loads before the first use.  Bound by
// memory: 16,384 rows of 16 heads of 64 to bfloat16 (86 MB) take <T_READ>.
template <int DH, typename T>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(ReadArgs a) {
  constexpr int G = DH / kKv4Group;
  const int lane = threadIdx.x & 31, oct = lane % kRowLanes<DH>, g = oct >> 2;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.c.B; b += kThreads)
      if (packed_rows(a.cu, b, a.total).bad) report(a.status, SPATTEN_E_INDEX);
  const int64_t task = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int h = static_cast<int>(task % a.c.H_kv);
  const SeqTile st = find_seq_tile<true>(a.cu, a.c.B, a.total, kTaskRows<DH>, static_cast<int>(task / a.c.H_kv));
  if (st.b < 0) return;
  const PackedRows p = packed_rows(a.cu, st.b, a.total);
  const int i0 = st.tile * kTaskRows<DH>, n = min(kTaskRows<DH>, p.n - i0);
  const int64_t first = static_cast<int64_t>(a.row0 ? a.row0[st.b] : 0) + i0;   // cache row of the task's first
  if (lane == 0 && (first < 0 || first + n > a.c.cap)) report(a.status, SPATTEN_E_INDEX);
  const int64_t base = (static_cast<int64_t>(st.b) * a.c.H_kv + h) * a.c.cap + first;
  const int64_t dst = (static_cast<int64_t>(p.first) + i0) * a.ld_tok + static_cast<int64_t>(h) * DH + oct * 8;
  uint32_t w[2][kSteps];
  float s[2][kSteps];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int r = k * (32 / kRowLanes<DH>) + lane / kRowLanes<DH>;
      const bool ok = r < n && first + r >= 0 && first + r < a.c.cap && a.out[t];   // else 0
      w[t][k] = ok ? reinterpret_cast<const uint32_t*>(t ? a.c.v_codes : a.c.k_codes)[(base + r) * (DH / 8) + (t ? v_word_at<DH>(oct) : k_word_at<DH>(oct))] : 0u;
      s[t][k] = ok ? bf16_bits_to_float((t ? a.c.v_scale : a.c.k_scale)[(base + r) * G + g]) : 0.0f;
    }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    T* out = static_cast<T*>(a.out[t]);
    if (!out) continue;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int r = k * (32 / kRowLanes<DH>) + lane / kRowLanes<DH>;
      float x[8];
      values8(t ? v_word<DH>(w[t][k], oct) : w[t][k], s[t][k], x);
      if (r < n) store8(out + dst + r * a.ld_tok, x);
    }
  }
}

// ----------------------------------------------------------------------------------------------
// evict
// ----------------------------------------------------------------------------------------------
constexpr int kSelThreads = 1024;

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

__device__ __forceinline__ uint32_t row_key(const EvictArgs& a, int64_t base, int j, int safe_from, bool has_safe) {
  if (has_safe && a.s.pos[base + j] >= safe_from) return 0xffffffffu;
  const float w = a.s.weight[base + j];
  return isnan(w) ? 0u : float_key(w);
}

// Exclusive prefix sums of two flags over the block in thread order; totals in *t0, *t1.
__device__ __forceinline__ int2 block_rank(bool f0, bool f1, int2* warp_sums, int* t0, int* t1) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t m0 = __ballot_sync(0xffffffffu, f0), m1 = __ballot_sync(0xffffffffu, f1);
  if (lane == 0) warp_sums[warp] = make_int2(__popc(m0), __popc(m1));
  __syncthreads();
  int2 w = warp_sums[lane];   // 32 warps: every warp scans all sums
  int2 inc = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc.x, o), y = __shfl_up_sync(0xffffffffu, inc.y, o);
    if (lane >= o) {
      inc.x += x;
      inc.y += y;
    }
  }
  *t0 = __shfl_sync(0xffffffffu, inc.x, 31);
  *t1 = __shfl_sync(0xffffffffu, inc.y, 31);
  const int bx = __shfl_sync(0xffffffffu, inc.x - w.x, warp), by = __shfl_sync(0xffffffffu, inc.y - w.y, warp);
  __syncthreads();
  const uint32_t below = (1u << lane) - 1u;
  return make_int2(bx + __popc(m0 & below), by + __popc(m1 & below));
}

// One block per (sequence, head): the keep-th largest key by four 8-bit radix passes, then one pass
// in row order that ranks ties, holes and the rows that fill them.
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int2 warp_sums[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_want;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int64_t bh = static_cast<int64_t>(b) * a.s.H_kv + h, base = bh * a.s.cap;
  const int n = clamp_len(a.len[b], a.n_max, a.status), k = a.keep;
  if (n <= k) {
    if (tid == 0) {
      a.count[2 * bh] = a.in_place ? 0 : n;
      a.count[2 * bh + 1] = n;
    }
    if (!a.in_place)
      for (int i = tid; i < n; i += kSelThreads) a.from[bh * a.keep + i] = i;
    return;
  }
  const bool has_safe = a.recent > 0;
  const int safe_from = has_safe ? a.seen[b] - a.recent : 0;
  uint32_t prefix = 0;
  int want = k;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int j = tid; j < n; j += kSelThreads) {
      const uint32_t key = row_key(a, base, j, safe_from, has_safe);
      if (shift == 24) {
        if (key == 0u && isnan(a.s.weight[base + j])) report(a.status, SPATTEN_E_NONFINITE);
        atomicAdd(&hist[key >> 24], 1);
      } else if ((key >> (shift + 8)) == (prefix >> (shift + 8))) {
        atomicAdd(&hist[(key >> shift) & 255u], 1);
      }
    }
    __syncthreads();
    if (tid < 32) {   // the bin that holds the want-th largest key: lane l sums bins 255-8l .. 248-8l
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += (c[i] = hist[255 - 8 * tid - i]);
      int inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (tid >= o) inc += x;
      }
      int before = inc - sum;
      if (before < want && want <= inc) {
        for (int i = 0; i < 8; ++i) {
          if (want <= before + c[i]) {
            s_prefix = prefix | static_cast<uint32_t>(255 - 8 * tid - i) << shift;
            s_want = want - before;
            break;
          }
          before += c[i];
        }
      }
    }
    __syncthreads();
    prefix = s_prefix;
    want = s_want;
  }
  // rows with key > prefix stay; of those equal to it, the first `want`
  int ties = 0, moved = 0;
  int32_t* hole = a.hole + bh * a.m;
  int32_t* tail = a.tail + bh * a.m;
  int holes = 0, tails = 0;
  for (int j0 = 0; j0 < n; j0 += kSelThreads) {
    const int j = j0 + tid;
    const uint32_t key = j < n ? row_key(a, base, j, safe_from, has_safe) : 0u;
    const bool tie = j < n && key == prefix;
    int t0, t1;
    const int2 tr = block_rank(tie, false, warp_sums, &t0, &t1);
    const bool kept = j < n && (key > prefix || (tie && ties + tr.x < want));
    ties += t0;
    const bool is_hole = j < k && !kept, is_tail = j >= k && kept;
    int h0, h1;
    const int2 r = block_rank(is_hole, is_tail, warp_sums, &h0, &h1);
    if (is_hole) hole[holes + r.x] = j;
    if (is_tail) tail[tails + r.y] = j;
    if (!a.in_place && j < k && kept) a.from[bh * a.keep + j] = j;
    holes += h0;
    tails += h1;
  }
  moved = holes;
  __syncthreads();
  if (!a.in_place)
    for (int i = tid; i < moved; i += kSelThreads) a.from[bh * a.keep + hole[i]] = tail[i];
  if (tid == 0) {
    a.count[2 * bh] = a.in_place ? moved : k;
    a.count[2 * bh + 1] = k;
  }
}

// Moves the planned rows: a row's codes are 16-byte pieces, its scales, weight and position one piece
// each; consecutive lanes take the pieces of one row.
template <int DH>
__global__ void __launch_bounds__(kThreads) kv4_move_kernel(EvictArgs a) {
  constexpr int kCode = DH / 32;            // 16-byte pieces of one tensor's codes
  constexpr int kPieces = DH == 64 ? 8 : 16;   // lanes per row (128 channels: 12 in use)
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t bh = static_cast<int64_t>(b) * a.s.H_kv + h;
  const int n = a.count[2 * bh];
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) a.len_out[b] = a.count[2 * bh + 1];
  const int piece = threadIdx.x % kPieces;
  for (int i = blockIdx.x * (kThreads / kPieces) + threadIdx.x / kPieces; i < n; i += gridDim.x * (kThreads / kPieces)) {
    const int64_t from = bh * a.s.cap + (a.in_place ? a.tail[bh * a.m + i] : a.from[bh * a.keep + i]);
    const int64_t to = bh * a.d.cap + (a.in_place ? a.hole[bh * a.m + i] : i);
    if (piece < kCode) {
      reinterpret_cast<uint4*>(a.d.k_codes)[to * kCode + piece] = reinterpret_cast<const uint4*>(a.s.k_codes)[from * kCode + piece];
    } else if (piece < 2 * kCode) {
      reinterpret_cast<uint4*>(a.d.v_codes)[to * kCode + piece - kCode] =
          reinterpret_cast<const uint4*>(a.s.v_codes)[from * kCode + piece - kCode];
    } else if (piece < 2 * kCode + 2) {
      const uint16_t* s = piece == 2 * kCode ? a.s.k_scale : a.s.v_scale;
      uint16_t* d = piece == 2 * kCode ? a.d.k_scale : a.d.v_scale;
      if constexpr (DH == 64) reinterpret_cast<uint32_t*>(d)[to] = reinterpret_cast<const uint32_t*>(s)[from];
      else reinterpret_cast<uint2*>(d)[to] = reinterpret_cast<const uint2*>(s)[from];
    } else if (piece == 2 * kCode + 2) {
      a.d.weight[to] = a.s.weight[from];
    } else if (piece == 2 * kCode + 3) {
      if (a.s.pos) a.d.pos[to] = a.s.pos[from];
    }
  }
}

bool same_cache(const spatten_kv4_cache& a, const spatten_kv4_cache& b) {
  return a.cap == b.cap && a.k_codes == b.k_codes && a.k_scale == b.k_scale && a.v_codes == b.v_codes &&
         a.v_scale == b.v_scale && a.weight == b.weight && a.pos == b.pos;
}
bool any_shared(const spatten_kv4_cache& a, const spatten_kv4_cache& b) {
  return a.k_codes == b.k_codes || a.k_scale == b.k_scale || a.v_codes == b.v_codes || a.v_scale == b.v_scale ||
         (a.weight && a.weight == b.weight) || (a.pos && a.pos == b.pos);
}

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

}  // namespace
}  // namespace spt

extern "C" int32_t spatten_kv4_append(const spatten_kv4_cache* c, const void* k, const void* v, int32_t dtype,
                                      int64_t ld_tok, int32_t total, const int32_t* cu, const int32_t* len,
                                      int32_t* len_out, const int32_t* seen, int32_t* seen_out,
                                      int32_t* dev_status, void* stream) {
  spt::AbiRange nvtx_range("spatten_kv4_append");
  using namespace spt;
  if (!c || !k || !v || !len || !len_out) return SPATTEN_E_ARG;
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
  if (!c || !cu || (!k_out && !v_out)) return SPATTEN_E_ARG;
  SPT_TRY(kv4_validate(*c));
  if (dtype != SPATTEN_F32 && dtype != SPATTEN_BF16) return SPATTEN_E_ARG;
  if (total < 0) return SPATTEN_E_ARG;
  if (ld_tok < static_cast<int64_t>(c->H_kv) * c->d_h) return SPATTEN_E_SHAPE;
  const int esz = dtype == SPATTEN_BF16 ? 2 : 4;
  if (!aligned16(k_out) || !aligned16(v_out) || (ld_tok * esz) % 16 != 0) return SPATTEN_E_ALIGN;
  if (total == 0) return SPATTEN_OK;
  const ReadArgs a{*c, cu, row0, total, {k_out, v_out}, ld_tok, dev_status};
  const int64_t tasks = (static_cast<int64_t>(total) / (c->d_h == 64 ? kTaskRows<64> : kTaskRows<128>) + c->B) * c->H_kv;
  const int64_t blocks = ceil_div(tasks, kThreads / 32);
  if (blocks > INT32_MAX) return SPATTEN_E_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(blocks);
  cudaStream_t st = as_stream(stream);
  if (c->d_h == 64) {
    if (dtype == SPATTEN_BF16) kv4_read_kernel<64, __nv_bfloat16><<<grid, kThreads, 0, st>>>(a);
    else kv4_read_kernel<64, float><<<grid, kThreads, 0, st>>>(a);
  } else {
    if (dtype == SPATTEN_BF16) kv4_read_kernel<128, __nv_bfloat16><<<grid, kThreads, 0, st>>>(a);
    else kv4_read_kernel<128, float><<<grid, kThreads, 0, st>>>(a);
  }
  return launch_status();
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
  cudaStream_t st = as_stream(stream);
  kv4_select_kernel<<<dim3(src->H_kv, src->B), kSelThreads, 0, st>>>(a);
  SPT_TRY(launch_status());
  // in place at most m rows move, else `keep`; a few rows per thread group when there are many
  const int64_t rows = a.in_place ? a.m : keep;
  const int per_block = kThreads / (src->d_h == 64 ? 8 : 16);
  const int64_t want = ceil_div(rows, per_block), most = ceil_div(8 * 148, static_cast<int64_t>(src->B) * src->H_kv);
  const dim3 grid(static_cast<unsigned>(want < 1 ? 1 : (want < most ? want : most)), src->H_kv, src->B);
  if (src->d_h == 64) kv4_move_kernel<64><<<grid, kThreads, 0, st>>>(a);
  else kv4_move_kernel<128><<<grid, kThreads, 0, st>>>(a);
  return launch_status();
}
