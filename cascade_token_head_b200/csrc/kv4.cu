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
// lanes of the group share their amax.  Returns the codes as nibbles (channel i at bits 4i) and the
// scale's bfloat16 bits.
__device__ __forceinline__ uint32_t quantize8(float* x, uint32_t* scale_bits, bool* bad) {
  float amax = 0.0f;
  *bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (!isfinite(x[i])) {
      x[i] = 0.0f;
      *bad = true;
    }
    amax = fmaxf(amax, fabsf(x[i]));
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(amax, 7.0f));
  if (__bfloat162float(sb) == 0.0f) sb = __float2bfloat16_rn(1.0f);
  const float s = __bfloat162float(sb);
  *scale_bits = __bfloat16_as_ushort(sb);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // the scale is rounded to nearest, so the largest quotient may pass 7 by a little: clamp
    const int q = max(-7, min(7, __float2int_rn(__fdiv_rn(x[i], s))));
    w |= static_cast<uint32_t>(q + 8) << (4 * i);
  }
  return w;
}

// One lane's eight channels of (row `src`, head h) into cache row `row`; whole warps call it (the
// lanes of a group exchange their amax), `ok` says whether this lane has a row to store.
template <int DH, typename T>
__device__ __forceinline__ void append8(const AppendArgs& a, int tensor, int64_t src, int b, int h, int oct, int row,
                                        bool ok) {
  constexpr int G = DH / kKv4Group;
  float x[8] = {};
  if (ok) load8(static_cast<const T*>(a.x[tensor]) + src * a.ld_tok + static_cast<int64_t>(h) * DH + oct * 8, x);
  uint32_t sb;
  bool bad;
  const uint32_t w = quantize8(x, &sb, &bad);
  if (!ok) return;
  if (bad) report(a.status, SPATTEN_E_NONFINITE);
  const int g = oct >> 2, t = oct & 3;
  const int64_t at = (static_cast<int64_t>(b) * a.c.H_kv + h) * a.c.cap + row;
  if (tensor == 0) {
    reinterpret_cast<uint32_t*>(a.c.k_codes)[at * (DH / 8) + t * G + g] = w;
  } else {
    uint16_t* v = reinterpret_cast<uint16_t*>(a.c.v_codes) + at * (DH / 4);
    v[(2 * t) * G + g] = static_cast<uint16_t>(w);
    v[(2 * t + 1) * G + g] = static_cast<uint16_t>(w >> 16);
  }
  if (t == 0) (tensor == 0 ? a.c.k_scale : a.c.v_scale)[at * G + g] = static_cast<uint16_t>(sb);
}

// Packed rows: one lane per eight channels, blockIdx.y the tensor.  Lanes run along a token's heads,
// so the loads are whole lines; each row's codes leave as one 32- or 64-byte segment.
template <int DH, typename T>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(AppendArgs a, bool counts) {
  constexpr int kLanes = DH / 8;
  const int per_row = a.c.H_kv * kLanes;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t r = u / per_row;
  const int rest = static_cast<int>(u - r * per_row), h = rest / kLanes, oct = rest % kLanes;
  const int tensor = blockIdx.y;
  bool ok = r < a.total;
  int b = -1, row = 0, i = 0;
  if (ok) {
    b = owner_of_row(a.cu, a.c.B, static_cast<int>(r));
    ok = b >= 0;
  }
  if (ok) {
    const PackedRows p = packed_rows(a.cu, b, a.total);
    const int old = clamp_len(a.len[b], a.c.cap, a.status);
    i = static_cast<int>(r) - p.first;
    ok = !p.bad && i >= 0 && i < p.n;
    row = old + i;
    if (ok && row >= a.c.cap) {
      report(a.status, SPATTEN_E_INDEX);
      ok = false;
    }
  }
  append8<DH, T>(a, tensor, r, b, h, oct, row, ok);
  if (ok && oct == 0 && tensor == 0) {
    const int64_t at = (static_cast<int64_t>(b) * a.c.H_kv + h) * a.c.cap + row;
    if (a.c.weight) a.c.weight[at] = 0.0f;
    if (a.c.pos) a.c.pos[at] = a.seen[b] + i;
  }
  // the counts, where no other block still reads them (len_out and seen_out are buffers of their own)
  if (counts && blockIdx.y == 0)
    for (int64_t s = u; s < a.c.B; s += static_cast<int64_t>(gridDim.x) * kThreads) {
      const PackedRows p = packed_rows(a.cu, static_cast<int>(s), a.total);
      if (p.bad) report(a.status, SPATTEN_E_INDEX);
      const int old = clamp_len(a.len[s], a.c.cap, a.status), n = min(p.n, a.c.cap - old);
      a.len_out[s] = old + n;
      if (a.seen_out) a.seen_out[s] = a.seen[s] + n;
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
    append8<DH, T>(a, tensor, b, b, h, oct, row, ok);
    if (ok && oct == 0 && tensor == 0) {
      const int64_t at = (static_cast<int64_t>(b) * a.c.H_kv + h) * a.c.cap + row;
      if (a.c.weight) a.c.weight[at] = 0.0f;
      if (a.c.pos) a.c.pos[at] = seen + 0;
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
  const int64_t units = static_cast<int64_t>(a.total) * a.c.H_kv * (DH / 8);
  if (units > 0) {
    const dim3 grid(static_cast<unsigned>(ceil_div(units, kThreads)), 2);
    kv4_append_kernel<DH, T><<<grid, kThreads, 0, st>>>(a, apart);
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

// One lane per eight channels; lanes run along a token's heads, so the stores are whole lines.
template <int DH, typename T>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(ReadArgs a) {
  constexpr int kLanes = DH / 8, G = DH / kKv4Group;
  const int per_row = a.c.H_kv * kLanes;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t r = u / per_row;
  if (r >= a.total) return;
  const int rest = static_cast<int>(u - r * per_row), h = rest / kLanes, oct = rest % kLanes;
  const int tensor = blockIdx.y;
  T* out = static_cast<T*>(a.out[tensor]);
  if (!out) return;
  const int b = owner_of_row(a.cu, a.c.B, static_cast<int>(r));
  if (b < 0) return;
  const PackedRows p = packed_rows(a.cu, b, a.total);
  const int64_t i = r - p.first;
  if (p.bad || i < 0 || i >= p.n) {
    report(a.status, SPATTEN_E_INDEX);
    return;
  }
  const int64_t row = (a.row0 ? a.row0[b] : 0) + i;
  float x[8] = {};
  if (row < 0 || row >= a.c.cap) {
    report(a.status, SPATTEN_E_INDEX);
  } else {
    const int g = oct >> 2, t = oct & 3;
    const int64_t at = (static_cast<int64_t>(b) * a.c.H_kv + h) * a.c.cap + row;
    uint32_t w;
    if (tensor == 0) {
      w = reinterpret_cast<const uint32_t*>(a.c.k_codes)[at * (DH / 8) + t * G + g];
    } else {
      const uint16_t* v = reinterpret_cast<const uint16_t*>(a.c.v_codes) + at * (DH / 4);
      w = v[(2 * t) * G + g] | static_cast<uint32_t>(v[(2 * t + 1) * G + g]) << 16;
    }
    const float s = bf16_bits_to_float((tensor == 0 ? a.c.k_scale : a.c.v_scale)[at * G + g]);
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = s * static_cast<float>(static_cast<int>((w >> (4 * c)) & 15u) - 8);
  }
  store8(out + r * a.ld_tok + static_cast<int64_t>(h) * DH + oct * 8, x);
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
  const int64_t units = static_cast<int64_t>(total) * c->H_kv * (c->d_h / 8);
  const dim3 grid(static_cast<unsigned>(ceil_div(units, kThreads)), 2);
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
