// Prompt attention on the 5th-generation tensor cores (tcgen05 + TMEM + TMA), bfloat16; float32 operands as
// sums of three bfloat16 planes, which a first kernel splits them into, and six products of planes (24 bits;
// 16 prompts of 512, 16 heads of 64: 163 us, and 570 with multiply-adds on CUDA cores).
//
// Two kernels, and a small third one when several query heads share a key/value head:
//  OUTPUT  one pass over the visible keys in tiles of KT with the running maximum and sum of the
//          softmax.  A CTA owns NQ tiles of 128 query rows that read the same key/value head; each has
//          softmax warps (TMEM lane = row; for KT = 128 two threads a row, 64 keys of a tile each), next
//          to one TMA producer warp and one MMA warp.  Rows of 64 channels take NQ = 1, KT = 64: small CTAs,
//          of which an SM holds several that hide each other's starts and ends.  Rows of 128 take NQ = 2,
//          KT = 128: one large CTA, whose key tiles are read once for both query tiles.  S = Q K^T goes to
//          TMEM, P (bfloat16) goes back over the columns of S and is the TMEM operand of O += P V, so P
//          never touches shared memory.
//  WEIGHT  weight_j = sum_i exp(S_ij - m_i) / l_i needs final statistics, hence a second pass over the
//          scores, transposed: S^T = K Q^T puts one key on each TMEM lane, so the sum over the rows stays
//          inside a thread (no exchange between lanes) and runs in a fixed order.
//  The heads of a group add up in a third, small one.
//  Where a call has too few row tiles to fill the GPU and long sequences, each tile's keys are split over several
//  CTAs of OUTPUT, whose parts a JOIN kernel adds up with the weights exp(m_part - m).
// What bounds them: exponentials (16 per clock and SM; for the weights a quarter of them goes to the FMA
// pipe, exp2_poly.cuh) next to the tensor cores.  8192 tokens, 32 heads of 128 over 8 (550 GFLOP): output
// 487 us in a row of calls, 1127 TFLOP/s, where the power limit holds the clock down (440 us by itself, tensor pipe
// 59 %); weights 299 (268; 55 %).  Short prompts are bound by each CTA's start and end and by the diagonal
// tiles: a batch of 16, 39 and 29 us, tensor pipe 20 %.  Float32, 16 prompts of 512: 38 us to split the operands
// (DRAM 63 %), 90 and 46 for outputs and weights, tensor pipe 39 %, with the softmax of a tile between its products.
// O's rescaling is skipped while no row's maximum has grown by more than 2^8, which float32 sums and the bfloat16 P
// bear without loss (P is relative; the values' range: spatten.h).
// Every mbarrier wait is bounded: on timeout the CTA reports SPATTEN_E_TIMEOUT, waits for its own
// copies and MMAs, frees its TMEM and returns.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "attention.cuh"
#include "exp2_poly.cuh"
#include "prompt.cuh"
#include "tc_tma.cuh"

namespace spt {
namespace {

using namespace tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 128;             // rows of a query tile (and, for the weights, keys of a key tile)
constexpr int kBox = 64;               // rows of a TMA box
constexpr float kRescale = 8.0f;       // growth of a row's maximum (log2) that makes O be rescaled

// The three planes of a pair of float32: each takes the high half of what is left, cut off (a sum of 24 bits).
__device__ __forceinline__ uint32_t split_pair(float2 x, uint32_t& mid, uint32_t& low) {
  const uint32_t a = __float_as_uint(x.x), b = __float_as_uint(x.y);
  const float r0 = x.x - __uint_as_float(a & 0xffff0000u), r1 = x.y - __uint_as_float(b & 0xffff0000u);
  const uint32_t c = __float_as_uint(r0), d = __float_as_uint(r1);
  mid = __byte_perm(c, d, 0x7632);
  low = __byte_perm(__float_as_uint(r0 - __uint_as_float(c & 0xffff0000u)), __float_as_uint(r1 - __uint_as_float(d & 0xffff0000u)), 0x7632);
  return __byte_perm(a, b, 0x7632);
}

__device__ __forceinline__ float2 ex2_pair(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }
// the same by the FMA pipe for the first POLY of every four pairs (Q: the pair), which takes NaN for a small exponent
template <int Q, int POLY>
__device__ __forceinline__ float2 exp2_pair(float2 x) {
  if constexpr ((Q & 3) < POLY) return exp2_poly2(x);
  else return ex2_pair(x);
}
constexpr int kWeightPoly = 1;   // of the weights' exponentials (outputs and weights of 16 x 1024 rows of 16 heads of 64: 117 us; none 121, half 121)

__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
// whether p holds in any of the threads that share a named barrier
__device__ __forceinline__ bool group_any(bool p, int id, int threads) {
  uint32_t r;
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      "setp.ne.u32 p, %1, 0;\n"
      "bar.red.or.pred q, %2, %3, p;\n"
      "selp.u32 %0, 1, 0, q;\n"
      "}\n"
      : "=r"(r)
      : "r"(p ? 1u : 0u), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// A wait of a whole warp: the first poll does not block, so that a limit of one poll is no wait at all.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t limit) {
  bool ok = mbar_test_wait(bar, parity);
  if (!ok) {
    if (limit > 1) ok = wait_bar(bar, parity, abort_flag, limit - 1);
    else *abort_flag = 1;
  }
  return __all_sync(0xffffffffu, ok);
}

// All of a [ROWS x DH] tile: blocks of 64 channels, each the rows' 128 bytes one behind the other; of PL planes,
// whose rows are `plane` rows apart, one tile behind the other.
template <int DH, int ROWS, int PL>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, int head, int row, int plane, uint64_t* bar) {
#pragma unroll
  for (int pl = 0; pl < PL; ++pl)
#pragma unroll
    for (int c = 0; c < DH / 64; ++c)
#pragma unroll
      for (int r = 0; r < ROWS; r += kBox)
        tma_load_3d(dst + ((pl * (DH / 64) + c) * ROWS + r) * 128, map, c * 64, head, pl * plane + row + r, bar);
}

// Float32 operands are sums of three bfloat16 planes (24 bits); of their nine products those within 2^-24 of the
// largest are made, small ones first.
template <int PL> constexpr int kProducts = PL == 1 ? 1 : 6;
template <int PL>
__device__ __forceinline__ constexpr int product_a(int i) {
  return PL == 1 ? 0 : (i == 0 ? 2 : (i == 2 || i == 3 ? 1 : 0));
}
template <int PL>
__device__ __forceinline__ constexpr int product_b(int i) {
  return PL == 1 ? 0 : (i == 1 ? 2 : (i == 2 || i == 4 ? 1 : 0));
}

// The MMA warp runs its loop as a whole and elects a lane (the same one every time) for the instructions
// themselves: so operands are known to be uniform and stay in uniform registers.  Issued from a branch of
// one lane, every MMA waited some 100 cycles for its operands to be moved there, against 64 of work.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "elect.sync _|p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void commit_one(uint64_t* bar) {
  if (elect_one()) mma_commit(bar);
}

// Descriptors of a tile's first step; a later one adds its offset, in units of 16 bytes, to the address in the
// low bits.
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr) { return desc_sw128(saddr, 16, 1024); }             // K-major
template <int ROWS>
__device__ __forceinline__ uint64_t desc_cols(uint32_t saddr) { return desc_sw128(saddr, ROWS * 128u, 1024); }    // MN-major

// D[128 x N] = A B^T over DH channels, both tiles K-major
template <int DH, int N, int PL>
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t a, uint64_t b) {
  constexpr uint32_t id = idesc_bf16(128, N, false, false);
#pragma unroll
  for (int i = 0; i < kProducts<PL>; ++i)
#pragma unroll
    for (int s = 0; s < DH / 16; ++s) {
      const uint32_t at = (product_a<PL>(i) * (kRows * DH * 2u) + (s >> 2) * (kRows * 128u) + (s & 3) * 32u) >> 4;
      const uint32_t bt = (product_b<PL>(i) * (N * DH * 2u) + (s >> 2) * (N * 128u) + (s & 3) * 32u) >> 4;
      if (elect_one()) mma_f16(d, a + at, b + bt, id, i > 0 || s > 0 ? 1u : 0u);
    }
}
// O (+)= P V: P in TMEM (8 columns per 16 keys, the second 64 keys 64 columns on; further planes of P behind
// the KT columns of the scores, 32 each: KT is 64 then), V rows MN-major
template <int DH, int KT, int PL>
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t p, uint64_t v, uint32_t acc) {
  constexpr uint32_t id = idesc_bf16(128, DH, false, true);
  static_assert(PL == 1 || KT == 64, "planes of P");
#pragma unroll
  for (int i = 0; i < kProducts<PL>; ++i) {
    const int pa = product_a<PL>(i);
#pragma unroll
    for (int s = 0; s < KT / 16; ++s)
      if (elect_one())
        mma_f16_ts(d, p + (pa ? KT + (pa - 1) * 32 : 0) + (s & 3) * 8 + (s >> 2) * 64,
                   v + ((product_b<PL>(i) * (KT * DH * 2u) + s * 2048u) >> 4), id, (acc || i > 0 || s > 0) ? 1u : 0u);
  }
}

struct Maps {
  CUtensorMap q, k, v;
};

// =================================================================================================
// OUTPUT
// =================================================================================================
// NQ query tiles a CTA, tiles of KT keys.  One thread has a row and 64 keys of each tile; where a tile has 128
// keys the two threads of a row share its maximum.
template <int DH_, int NQ_, int KT_, int STAGES, int PL_ = 1>
struct OutCfg {
  static constexpr int DH = DH_, NQ = NQ_, KT = KT_, PL = PL_, kHalves = KT / 64;
  static constexpr int kStages = STAGES;                 // K and V tiles in flight, one ring
  static constexpr uint32_t kQTile = PL * kRows * DH * 2u, kTile = PL * KT * DH * 2u;
  static constexpr uint32_t oKV = NQ * kQTile;
  static constexpr uint32_t kSmem = oKV + kStages * kTile + 1024u;
  static constexpr int kGroup = 128 * kHalves;           // softmax threads of a query tile
  static constexpr int kThreads = NQ * kGroup + 64;
  static constexpr uint32_t kScores = KT + (PL - 1) * 32;   // columns of a tile's scores and further planes of P
  static constexpr uint32_t kColumns = NQ * (kScores + DH), kTmem = kColumns <= 128 ? 128 : (kColumns <= 256 ? 256 : 512);
  static constexpr int kCtas = 2 * kSmem > 226 * 1024 ? 1 : 512 / kTmem;   // per SM
  static constexpr uint32_t tS = 0, tO = NQ * kScores;
};

template <int NQ, int NST>
struct OutBars {
  uint64_t q_full, kv_full[NST], kv_empty[NST], s_full[NQ], p_ready[NQ], o_full[NQ], v_fix, drain;
};

constexpr int kSplitTiles = 2, kMaxSplits = 32;   // key tiles that a split has at least, splits at most

// What a CTA does with its tile.
template <class C>
struct OutWork {
  int head[C::NQ], row0[C::NQ], rows[C::NQ], T[C::NQ];   // of each query tile: head, rows of the sequence, key tiles seen
  int Tmax, partial;                                     // the most key tiles; the one that ends past the keys, or -1
  int key0;                                              // the first key: of all those tiles, or of split `part` of `parts`
  __device__ __forceinline__ OutWork(const PromptTile& pt, int slot, bool pair_heads, int tile_rows, int part, int parts) {
    Tmax = 0;
#pragma unroll
    for (int g = 0; g < C::NQ; ++g) {
      head[g] = pair_heads ? 2 * slot + g : slot;
      row0[g] = pt.tile * tile_rows + (pair_heads ? 0 : 128 * g);
      rows[g] = max(0, min(128, pt.q.n - row0[g]));
      const int seen = rows[g] ? max(0, min(pt.k.n, row0[g] + rows[g] + pt.k.n - pt.q.n)) : 0;   // keys the last row sees
      T[g] = (seen + C::KT - 1) / C::KT;
      Tmax = max(Tmax, T[g]);
    }
    partial = pt.k.n < Tmax * C::KT ? Tmax - 1 : -1;
    key0 = 0;
    if (parts > 1) {
      const int per = max(kSplitTiles, (Tmax + parts - 1) / parts), lo = part * per;
      key0 = lo * C::KT;
      Tmax = max(0, min(Tmax - lo, per));
#pragma unroll
      for (int g = 0; g < C::NQ; ++g) T[g] = max(0, min(T[g] - lo, per));
      partial = partial >= lo && partial - lo < Tmax ? partial - lo : -1;
    }
  }
};

// SPLIT: the CTA has a part of its row tile's keys (a kernel of its own: it costs registers, 2 % of unsplit calls)
template <class C, bool SPLIT>
__global__ void __launch_bounds__(C::kThreads, C::kCtas) prompt_out_kernel(PromptProblem p, const __grid_constant__ Maps maps) {
  constexpr int DH = C::DH, NQ = C::NQ, KT = C::KT, PL = C::PL, NST = C::kStages, kHalves = C::kHalves;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ OutBars<NQ, NST> bars;
  __shared__ float row_stat[NQ][kHalves][kRows];   // what the two halves of a row tell each other
  __shared__ uint32_t tmem_base;
  __shared__ PromptTile item;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const spatten_prompt_args& a = p.a;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int G = a.H / a.H_kv;
  // NQ = 2: two heads of a group at the same rows, or (odd groups) 256 rows of one head
  const bool pair_heads = NQ == 2 && (G & 1) == 0;
  const int tile_rows = NQ == 2 && !pair_heads ? 256 : 128;
  const int slots = pair_heads ? a.H / 2 : a.H;
  constexpr int kProducer = NQ * C::kGroup / 32, kMma = kProducer + 1;
  if (warp == kMma) {
    tmem_alloc(&tmem_base, C::kTmem);
    tmem_relinquish();   // without it no second CTA becomes resident
  } else if (warp == kProducer && lane == 0) {
    tma_prefetch_map(&maps.q);
    tma_prefetch_map(&maps.k);
    tma_prefetch_map(&maps.v);
    abort_word = 0;
    mbar_init(&bars.q_full, 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(&bars.kv_full[s], 1);
      mbar_init(&bars.kv_empty[s], 1);
    }
    for (int g = 0; g < NQ; ++g) {
      mbar_init(&bars.s_full[g], 1);
      mbar_init(&bars.p_ready[g], C::kGroup);
      mbar_init(&bars.o_full[g], 1);
    }
    mbar_init(&bars.v_fix, 32);
    mbar_init(&bars.drain, 1);
    fence_mbar_init();
  }
  grid_dep_trigger();
  grid_dep_wait();
  if (blockIdx.x == 0) report_bad_offsets(a);
  // one warp looks the tile up and starts the loads that wait for nothing, before the CTA meets
  const int parts = SPLIT ? p.splits : 1, part = SPLIT ? static_cast<int>(blockIdx.x / slots) % parts : 0;
  const int slot = blockIdx.x % slots, hk = (pair_heads ? 2 * slot : slot) / G;
  auto load_kv = [&](int x, int first) {   // the ring's x-th tile: K0 V0 K1 V1 ..
    mbar_arrive_expect_tx(&bars.kv_full[x % NST], C::kTile);
    load_tile<DH, KT, PL>(smem + C::oKV + (x % NST) * C::kTile, (x & 1) ? &maps.v : &maps.k, hk, first + (x >> 1) * KT, a.total_kv,
                          &bars.kv_full[x % NST]);
  };
  if (warp == kProducer) {
    const PromptTile pt = find_prompt_tile<false>(a, tile_rows, blockIdx.x / slots / parts);
    if (lane == 0) {
      item = pt;
      if (pt.b >= 0) {
        const OutWork<C> w(pt, slot, pair_heads, tile_rows, part, parts);
        if (w.Tmax > 0) {
          mbar_arrive_expect_tx(&bars.q_full, NQ * C::kQTile);
#pragma unroll
          for (int g = 0; g < NQ; ++g)   // a tile without rows is loaded from the first one's rows and not used
            load_tile<DH, kRows, PL>(smem + g * C::kQTile, &maps.q, w.head[g], pt.q.first + (w.rows[g] ? w.row0[g] : w.row0[0]), a.total_q,
                                     &bars.q_full);
          for (int x = 0; x < min(NST, 2 * w.Tmax); ++x) load_kv(x, pt.k.first + w.key0);
        }
      }
    }
    __syncwarp();
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0), wlim = p.wait_limit;
  const PromptTile pt = item;
  if (pt.b < 0) {   // no such tile
    if (warp == kMma) tmem_dealloc(tmem, C::kTmem);
    return;
  }
  const PackedRows qr = pt.q, kr = pt.k;
  const int shift = kr.n - qr.n;
  const OutWork<C> work(pt, slot, pair_heads, tile_rows, part, parts);
  const auto &head = work.head, &row0 = work.row0, &rows = work.rows, &T = work.T;
  const int Tmax = work.Tmax, partial = work.partial, early = min(NST, 2 * Tmax);
  bool aborted = false;

  if (warp == kProducer) {
    int issued = early;
    for (int x = 0; x < 2 * Tmax; ++x) {
      const int s = x % NST, t = x >> 1;
      const uint32_t ph = (x / NST) & 1;
      if (x >= early) {
        if (!warp_wait(&bars.kv_empty[s], ph ^ 1u, abort_flag, wlim)) {
          aborted = true;
          break;
        }
        if (lane == 0) load_kv(x, kr.first + work.key0);
        ++issued;
      }
      if ((x & 1) && t == partial) {
        uint8_t* dst = smem + C::oKV + s * C::kTile;
        // rows past the sequence's keys meet P = 0: they must be finite, so they become zeros
        if (!warp_wait(&bars.kv_full[s], ph, abort_flag, wlim)) {
          aborted = true;
          break;
        }
        const int first = kr.n - work.key0 - t * KT;
        for (int e = first * 8 + lane; e < KT * 8; e += 32)
#pragma unroll
          for (int c = 0; c < PL * DH / 64; ++c)
            *reinterpret_cast<uint4*>(dst + c * KT * 128 + sw128_offset(e >> 3, e & 7)) = make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
        mbar_arrive(&bars.v_fix);
      }
    }
    if (lane == 0 && Tmax > 0) {   // copies in flight land before shared memory is given up, whoever gave up waiting
      drain_wait(&bars.q_full, 0);
      for (int x = max(0, issued - NST); x < issued; ++x) drain_wait(&bars.kv_full[x % NST], (x / NST) & 1);
    }
  } else if (warp == kMma) {
    if (Tmax > 0) {
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!aborted && !warp_wait(bar, parity, abort_flag, wlim)) aborted = true;
        return !aborted;
      };
      constexpr uint32_t kStep = C::kTile >> 4;
      const uint64_t dQ = desc_rows(smem_u32(smem)), dK = desc_rows(smem_u32(smem + C::oKV)), dV = desc_cols<KT>(smem_u32(smem + C::oKV));
      if (wait(&bars.q_full, 0) && wait(&bars.kv_full[0], 0)) {
        tc_after_sync();
#pragma unroll
        for (int g = 0; g < NQ; ++g)
          if (T[g] > 0) {
            mma_scores<DH, KT, PL>(tmem + C::tS + g * C::kScores, dQ + g * (C::kQTile >> 4), dK);
            commit_one(&bars.s_full[g]);
          }
        commit_one(&bars.kv_empty[0]);
      }
      // One tile's P V and next scores run while the other tile's softmax does.  Between two tiles' MMAs there
      // is only the wait for P: the tensor cores idle meanwhile.  (An MMA warp per tile took 675 us where this
      // form then took 519: the tiles' MMAs alternate in the pipe.)
      int sv = 1, sk = 2 % NST, pv = 0, pk = (2 / NST) & 1;   // the ring's stages of V(t) and K(t + 1), and their phases
      for (int t = 0; t < Tmax && !aborted; ++t) {
        const bool more = t + 1 < Tmax;
        if (!wait(&bars.kv_full[sv], pv) || (t == partial && !wait(&bars.v_fix, 0)) || (more && !wait(&bars.kv_full[sk], pk))) break;
        const uint64_t dVt = dV + sv * kStep, dKt = dK + sk * kStep;
#pragma unroll
        for (int g = 0; g < NQ; ++g) {
          if (t >= T[g]) continue;
          if (!wait(&bars.p_ready[g], t & 1)) break;
          tc_after_sync();
          mma_pv<DH, KT, PL>(tmem + C::tO + g * DH, tmem + C::tS + g * C::kScores, dVt, PL == 1 && t > 0 ? 1u : 0u);
          if (t + 1 < T[g]) {
            mma_scores<DH, KT, PL>(tmem + C::tS + g * C::kScores, dQ + g * (C::kQTile >> 4), dKt);   // over the P that the MMAs before it read
            commit_one(&bars.s_full[g]);
          } else {
            commit_one(&bars.o_full[g]);
          }
        }
        if (aborted) break;
        commit_one(&bars.kv_empty[sv]);
        if (more) commit_one(&bars.kv_empty[sk]);
        if ((sv += 2) >= NST) sv -= NST, pv ^= 1;
        if ((sk += 2) >= NST) sk -= NST, pk ^= 1;
      }
      if (aborted) {   // every MMA already issued completes before TMEM is freed
        commit_one(&bars.drain);
        drain_wait(&bars.drain, 0);
      }
    }
    __syncwarp();
  } else {
    // warp (tile g, half, quadrant): 32 rows, and 64 of a tile's keys
    const int g = NQ == 1 ? 0 : warp / (4 * kHalves), half = kHalves == 1 ? 0 : (warp >> 2) & 1, r = tid & 127;
    const int my_row0 = g ? row0[NQ - 1] : row0[0], my_rows = g ? rows[NQ - 1] : rows[0], my_T = g ? T[NQ - 1] : T[0];
    const int my_head = g ? head[NQ - 1] : head[0];
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // the warp's TMEM lanes (32 (warp & 3)) << 16
    constexpr int kOCols = DH / kHalves;                            // columns of O that this thread scales and stores
    const uint32_t tS = tmem + lanes + C::tS + g * C::kScores + half * 64, tO = tmem + lanes + C::tO + g * DH + half * kOCols;
    // the last key that this row sees, and that the warp's first one does
    const int last = min(my_row0 + r + shift, kr.n - 1), warp_row = my_row0 + (warp & 3) * 32;
    const int last_first = min(warp_row + shift, kr.n - 1), last_last = min(warp_row + 31 + shift, kr.n - 1);
    const float c = a.sm_scale * kLog2e;
    const float2 cc = make_float2(c, c);
    float m = -INFINITY, l = 0.0f;   // maximum (log2 units) that P is relative to, sum of this half
    // Float32: the tensor cores cut their sums off, so an output accumulated there over hundreds of steps drifts
    // towards 0 by their number times 2^-25.  Each tile's P V (of which the small products come first) starts
    // from 0 instead, and the tiles add up here, rounded to nearest.
    float acc[PL == 3 ? DH : 1];
#pragma unroll
    for (int j = 0; j < (PL == 3 ? DH : 1); ++j) acc[j] = 0.0f;
    auto add_tile = [&]() {
#pragma unroll
      for (int ch = 0; ch < (PL == 3 ? DH : 0); ch += 32) {
        float o[32];
        tmem_ld32(tO + ch, o);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[PL == 3 ? ch + j : 0] += o[j];
      }
    };
    for (int t = 0; t < my_T; ++t) {
      const bool ok = warp_wait(&bars.s_full[g], t & 1, abort_flag, wlim);
      tc_after_sync();
      if (PL == 3 && ok && t > 0) add_tile();   // the score MMA was issued behind the previous P V
      const int j0 = work.key0 + t * KT + half * 64, lim = last - j0;   // columns 0 .. lim are seen
      const bool full = last_first - j0 >= 63;              // by every row of the warp
      float mx = -INFINITY;
      if (ok) {   // the scores are read twice: there are not registers enough to keep them over the vote
        if (full) {
          float v[64];
          tmem_ld32(tS, v);
          tmem_ld32(tS + 32, v + 32);
          tmem_ld_wait();
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[k] = v[k];
#pragma unroll
            for (int j = 1; j < 8; ++j) x[k] = fmaxf(x[k], v[k + 8 * j]);
          }
          mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        } else {
#pragma unroll 1
          for (int ch = 0; ch < 64 && last_last - j0 >= ch; ch += 32) {
            float v[32];
            tmem_ld32(tS + ch, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) mx = fmaxf(mx, ch + j <= lim ? v[j] : -INFINITY);
          }
        }
      }
      const float mt = c * mx;
      const bool grow = t == 0 || !ok || mt > m + kRescale;
      if (kHalves == 1 ? __any_sync(0xffffffffu, grow) : group_any(grow, 1 + g, C::kGroup)) {
        float mn = fmaxf(m, mt);
        if constexpr (kHalves == 1) {
          if (!ok) {
            aborted = true;
            break;
          }
        } else {
          if (group_any(!ok, 1 + g, C::kGroup)) {   // the group agrees
            aborted = true;
            break;
          }
          row_stat[g][half][r] = mt;
          named_sync(1 + g, C::kGroup);
          mn = fmaxf(mn, row_stat[g][half ^ 1][r]);
        }
        const float f = ex2(m - (mn == -INFINITY ? 0.0f : mn));
        m = mn;
        l *= f;
        // the score MMA of this tile was issued behind the previous P V, so O is complete here
        if constexpr (PL == 3) {
#pragma unroll
          for (int j = 0; j < DH; ++j) acc[j] *= f;
        } else if (t > 0 && __any_sync(0xffffffffu, f != 1.0f)) {
#pragma unroll 1
          for (int ch = 0; ch < kOCols; ch += 32) {
            float o[32];
            tmem_ld32(tO + ch, o);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t u[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(o[16 * q + j] * f);
              tmem_st16(tO + ch + 16 * q, u);
            }
          }
        }
      }
      const float base = m == -INFINITY ? 0.0f : m;
      const float2 nb = make_float2(-base, -base);
      float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
      if (full) {
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t u[16], u2[PL == 3 ? 16 : 1], u3[PL == 3 ? 16 : 1];
          float v[32];
          tmem_ld32(tS + ch * 32, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float* w = v + 2 * j;
            const float2 e0 = ex2_pair(__ffma2_rn(make_float2(w[0], w[1]), cc, nb));
            const float2 e1 = ex2_pair(__ffma2_rn(make_float2(w[2], w[3]), cc, nb));
            const float2 e2 = ex2_pair(__ffma2_rn(make_float2(w[4], w[5]), cc, nb));
            const float2 e3 = ex2_pair(__ffma2_rn(make_float2(w[6], w[7]), cc, nb));
            s0 = __fadd2_rn(s0, __fadd2_rn(e0, e2));
            s1 = __fadd2_rn(s1, __fadd2_rn(e1, e3));
            if constexpr (PL == 1) {
              u[j] = pack_bf16x2(e0.x, e0.y);
              u[j + 1] = pack_bf16x2(e1.x, e1.y);
              u[j + 2] = pack_bf16x2(e2.x, e2.y);
              u[j + 3] = pack_bf16x2(e3.x, e3.y);
            } else {
              u[j] = split_pair(e0, u2[j], u3[j]);
              u[j + 1] = split_pair(e1, u2[j + 1], u3[j + 1]);
              u[j + 2] = split_pair(e2, u2[j + 2], u3[j + 2]);
              u[j + 3] = split_pair(e3, u2[j + 3], u3[j + 3]);
            }
          }
          tmem_st16(tS + ch * 16, u);   // over this thread's own scores, read before
          if constexpr (PL == 3) {
            tmem_st16(tS + KT + ch * 16, u2);
            tmem_st16(tS + KT + 32 + ch * 16, u3);
          }
        }
      } else {   // by ex2 alone: the polynomial does not reach 0, which hidden keys need
#pragma unroll 1
        for (int ch = 0; ch < 64; ch += 32) {
          uint32_t u[16], u2[PL == 3 ? 16 : 1], u3[PL == 3 ? 16 : 1];
          if (last_last - j0 >= ch) {
            float v[32];
            tmem_ld32(tS + ch, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 x = __ffma2_rn(make_float2(v[2 * j], v[2 * j + 1]), cc, nb);
              const float2 e = make_float2(ch + 2 * j <= lim ? ex2(x.x) : 0.0f, ch + 2 * j + 1 <= lim ? ex2(x.y) : 0.0f);
              s0 = __fadd2_rn(s0, e);
              if constexpr (PL == 1) u[j] = pack_bf16x2(e.x, e.y);
              else u[j] = split_pair(e, u2[j], u3[j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              u[j] = 0u;
              if constexpr (PL == 3) u2[j] = u3[j] = 0u;
            }
          }
          tmem_st16(tS + (ch >> 1), u);
          if constexpr (PL == 3) {
            tmem_st16(tS + KT + (ch >> 1), u2);
            tmem_st16(tS + KT + 32 + (ch >> 1), u3);
          }
        }
      }
      l += (s0.x + s1.x) + (s0.y + s1.y);
      tmem_st_wait();
      tc_before_sync();
      mbar_arrive(&bars.p_ready[g]);
    }
    if (kHalves == 2 && !aborted) {   // the group agrees on that
      named_sync(1 + g, C::kGroup);   // the maxima have been read
      row_stat[g][half][r] = l;
      named_sync(1 + g, C::kGroup);
      l = row_stat[g][0][r] + row_stat[g][kHalves - 1][r];
    }
    // rows that see nothing have l = 0 and O = 0; a NaN sum stays one
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
    if (!aborted && my_T > 0 && !warp_wait(&bars.o_full[g], 0, abort_flag, wlim)) aborted = true;
    if (!aborted) {
      tc_after_sync();
      const int64_t row = static_cast<int64_t>(qr.first) + my_row0 + r;
      using T = std::conditional_t<PL == 1, __nv_bfloat16, float>;
      if (PL == 3 && my_T > 0) add_tile();
      if constexpr (SPLIT) {   // as it is: prompt_join_kernel does the rest
        const int64_t at = (static_cast<int64_t>(part) * a.H + my_head) * a.total_q + row;
        if (r < my_rows && half == 0) p.split_ml[at] = make_float2(m, l);
        if (my_T > 0) {
          float* part_o = p.split_o + at * DH + half * kOCols;
#pragma unroll
          for (int ch = 0; ch < kOCols; ch += 32) {
            float o[32];
            if constexpr (PL == 3) {
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = acc[ch + j];
            } else {
              tmem_ld32(tO + ch, o);
              tmem_ld_wait();
            }
            if (r < my_rows)
#pragma unroll
              for (int j = 0; j < 32; j += 8) {
                uint32_t u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(o[j + i]);
                store32(part_o + ch + j, u);
              }
          }
        }
      } else {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.o) + row * a.o_ld_tok + static_cast<int64_t>(my_head) * DH + half * kOCols);
        if constexpr (PL == 3) {
          if (r < my_rows)
#pragma unroll
            for (int j = 0; j < DH; j += 8) {
              uint32_t u[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(acc[j + i] * inv);
              store32(dst + j / 4, u);
            }
        } else {
#pragma unroll 1
          for (int ch = 0; ch < kOCols / 32; ++ch) {
            float o[32];
            if (my_T > 0) {
              tmem_ld32(tO + ch * 32, o);
              tmem_ld_wait();
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = 0.0f;
            }
            if (r < my_rows) {
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint32_t u[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = pack_bf16x2(o[16 * q + 2 * j] * inv, o[16 * q + 2 * j + 1] * inv);
                store32(dst + ch * 4 + 2 * q, u);
              }
            }
          }
        }
        if (p.offset && half == 0 && r < my_rows)   // exp2(c (S + offset)) = P
          p.offset[static_cast<int64_t>(my_head) * a.total_q + row] = l > 0.0f ? -(m + log2f(l)) / c : (l == 0.0f ? 0.0f : l);
      }
    }
  }
  tc_before_sync();
  const bool any_abort = __syncthreads_or(aborted);
  if (any_abort && tid == 0) report(a.dev_status, SPATTEN_E_TIMEOUT);
  if (warp == kMma) {
    tc_after_sync();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// The splits of a row joined: a warp per row and head, DH / 32 channels a lane.
template <int DH, typename T>
__global__ void __launch_bounds__(256) prompt_join_kernel(PromptProblem p) {
  grid_dep_trigger();
  grid_dep_wait();
  const spatten_prompt_args& a = p.a;
  constexpr int N = DH / 32, kInFlight = 8;
  static_assert(kMaxSplits % kInFlight == 0, "whole rounds");
  const int lane = threadIdx.x & 31;
  const int64_t x = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int row = static_cast<int>(x / a.H), h = static_cast<int>(x % a.H);
  if (row >= a.total_q) return;
  const int64_t at = static_cast<int64_t>(h) * a.total_q + row, step = static_cast<int64_t>(a.H) * a.total_q;
  static_assert(kMaxSplits <= 32, "a lane a split");
  const float2 ml = lane < p.splits ? p.split_ml[lane * step + at] : make_float2(-INFINITY, 0.0f);
  if (owner_of_row(a.cu_q, a.B, a.total_q, row) < 0) return;   // rows of no sequence stay as they are (and have no parts)
  float m = ml.x;
#pragma unroll
  for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  // a split without keys has l = 0 and left no output; a NaN goes on
  const float f = ml.y == 0.0f ? 0.0f : ex2(ml.x - (m == -INFINITY ? 0.0f : m));
  float l = 0.0f, o[N] = {};
  for (int s0 = 0; s0 < p.splits; s0 += kInFlight) {
    float v[kInFlight][N];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {   // of a split that left no output too: that is read and not used
      const float* part = p.split_o + (min(s0 + u, p.splits - 1) * step + at) * DH + lane * N;
      if constexpr (N == 4)
        asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[u][0]), "=f"(v[u][1]), "=f"(v[u][N - 2]), "=f"(v[u][N - 1]) : "l"(part));
      else
        asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(v[u][0]), "=f"(v[u][1]) : "l"(part));
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {   // splits past the last: lanes of l = 0
      const float ls = __shfl_sync(0xffffffffu, ml.y, s0 + u), fs = __shfl_sync(0xffffffffu, f, s0 + u);
      l = fmaf(ls, fs, l);
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = fmaf(ls == 0.0f ? 0.0f : v[u][i], fs, o[i]);
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
  T* dst = static_cast<T*>(a.o) + row * a.o_ld_tok + static_cast<int64_t>(h) * DH + lane * N;
#pragma unroll
  for (int i = 0; i < N; ++i) st_from_float(dst + i, o[i] * inv);
  if (p.offset && lane == 0)   // as in the output kernel
    p.offset[at] = l > 0.0f ? -(m + log2f(l)) / (a.sm_scale * kLog2e) : (l == 0.0f ? 0.0f : l);
}

// =================================================================================================
// WEIGHT
// =================================================================================================
template <int DH_, int STAGES, int BUFS_, int CTAS, int PL_ = 1>
struct WeightCfg {
  static constexpr int DH = DH_, PL = PL_;
  static constexpr int kStages = STAGES;
  static constexpr uint32_t kTile = PL * kRows * DH * 2u, kExtra = kRows * 32u;   // and 16 channels more
  static constexpr uint32_t oQ = kTile + kExtra, kStage = kTile + kExtra;
  static constexpr uint32_t kSmem = oQ + kStages * kStage + 1024u;
  static constexpr int kSoftmax = 256, kThreads = kSoftmax + 64;
  static constexpr int kBufs = BUFS_, kCtas = CTAS;   // score buffers; CTAs per SM
  static constexpr uint32_t kTmem = 128 * kBufs;
  static_assert(CTAS * (kSmem + 2048) <= 228 * 1024 && CTAS * kTmem <= 512, "CTAs per SM");
};

// The row's offset -(m + log2 l) / c enters the scores by an MMA step of 16 channels more: the keys' are three
// ones, the rows' the offset as the sum of three bfloat16 (24 bits).  So no thread reads a statistic, and a
// weight costs a multiplication, an exponential and an addition.  32-byte rows, 32-byte swizzle.
__device__ __forceinline__ uint32_t extra_at(uint32_t row, uint32_t chunk) {
  return row * 32u + ((chunk ^ ((row >> 2) & 1u)) << 4);
}
__device__ __forceinline__ uint64_t desc_extra(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>(256 >> 4) << 32;   // 8-row groups
  d |= static_cast<uint64_t>(1) << 46;          // descriptor version for tcgen05
  d |= static_cast<uint64_t>(6) << 61;          // SWIZZLE_32B
  return d;
}

template <int NST>
struct WeightBars {
  uint64_t k_full, q_full[NST], q_empty[NST], s_full[2], s_empty[2], drain;
};

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas) prompt_weight_kernel(PromptProblem p, const __grid_constant__ Maps maps) {
  constexpr int DH = C::DH, PL = C::PL, NST = C::kStages, NB = C::kBufs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ WeightBars<NST> bars;
  __shared__ float half_sum[kRows];
  __shared__ int last_nan;   // the last row whose offset is NaN: the keys that it sees get one whichever unit made their exponentials
  __shared__ uint32_t tmem_base;
  __shared__ PromptTile item;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const spatten_prompt_args& a = p.a;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  constexpr int kProducer = 8, kMma = 9;
  if (warp == kMma) {
    tmem_alloc(&tmem_base, C::kTmem);
    tmem_relinquish();   // without it no second CTA becomes resident
  } else if (warp == kProducer) {
    if (lane == 0) {
      tma_prefetch_map(&maps.q);
      tma_prefetch_map(&maps.k);
      abort_word = 0;
      mbar_init(&bars.k_full, 1);
      for (int s = 0; s < NST; ++s) {
        mbar_init(&bars.q_full[s], 33);
        mbar_init(&bars.q_empty[s], 1);
      }
      for (int s = 0; s < 2; ++s) {
        mbar_init(&bars.s_full[s], 1);
        mbar_init(&bars.s_empty[s], 8);
      }
      mbar_init(&bars.drain, 1);
      fence_mbar_init();
    }
  } else if (tid < kRows) {   // the keys' extra channels: 1, 1, 1, 0, ..
    *reinterpret_cast<uint4*>(smem + C::kTile + extra_at(tid, 0)) = make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u);
    *reinterpret_cast<uint4*>(smem + C::kTile + extra_at(tid, 1)) = make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
  }
  grid_dep_trigger();
  grid_dep_wait();
  const int h = blockIdx.x % a.H, G = a.H / a.H_kv, hk = h / G;
  auto first_tile = [](const PromptTile& pt) {   // of the row tiles that see the tile's first key
    return max(0, pt.tile * kRows - (pt.k.n - pt.q.n)) / kRows;
  };
  if (warp == kProducer) {   // one warp looks the tile up and loads its keys before the CTA meets
    const PromptTile pt = find_prompt_tile<true>(a, kRows, blockIdx.x / a.H);
    if (lane == 0) {
      item = pt;
      if (pt.b >= 0 && (pt.q.n + kRows - 1) / kRows > first_tile(pt)) {
        mbar_arrive_expect_tx(&bars.k_full, C::kTile);
        load_tile<DH, kRows, PL>(smem, &maps.k, hk, pt.k.first + pt.tile * kRows, a.total_kv, &bars.k_full);
      }
    }
    __syncwarp();
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0), wlim = p.wait_limit;
  const PromptTile pt = item;
  if (pt.b < 0) {   // no such tile
    if (warp == kMma) tmem_dealloc(tmem, C::kTmem);
    return;
  }
  const PackedRows qr = pt.q, kr = pt.k;
  const int j0 = pt.tile * kRows, shift = kr.n - qr.n;
  const bool counted = counts_rows(a, pt.b, kr.n);
  const int rt0 = first_tile(pt), NT = max(0, (qr.n + kRows - 1) / kRows - rt0);
  bool aborted = false;
  float total = 0.0f;

  if (warp == kProducer) {
    int issued = 0, nan_row = INT32_MIN;
    const float* offset = p.offset + static_cast<int64_t>(h) * a.total_q + qr.first;
    for (int t = 0; t < NT; ++t) {
      const int s = t % NST, i0 = (rt0 + t) * kRows;
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {   // rows past the sequence are masked where they are used
        const int i = i0 + lane + 32 * k;
        v[k] = i < qr.n ? offset[i] : 0.0f;
      }
      if (!warp_wait(&bars.q_empty[s], ((t / NST) & 1) ^ 1u, abort_flag, wlim)) {
        aborted = true;
        break;
      }
      uint8_t* dst = smem + C::oQ + s * C::kStage;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars.q_full[s], C::kTile);
        load_tile<DH, kRows, PL>(dst, &maps.q, h, qr.first + i0, a.total_q, &bars.q_full[s]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (isnan(v[k])) nan_row = i0 + lane + 32 * k;
        const uint32_t hi = pack_bf16x2(v[k], 0.0f);
        const float r1 = v[k] - __uint_as_float(hi << 16);
        const uint32_t mid = pack_bf16x2(r1, 0.0f);
        const float r2 = r1 - __uint_as_float(mid << 16);
        *reinterpret_cast<uint4*>(dst + C::kTile + extra_at(lane + 32 * k, 0)) =
            make_uint4((hi & 0xffffu) | mid << 16, pack_bf16x2(r2, 0.0f), 0u, 0u);
        *reinterpret_cast<uint4*>(dst + C::kTile + extra_at(lane + 32 * k, 1)) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_async_smem();
      mbar_arrive(&bars.q_full[s]);
      ++issued;
    }
    nan_row = __reduce_max_sync(0xffffffffu, nan_row);
    if (lane == 0) last_nan = nan_row;
    if (lane == 0 && NT > 0) {   // as in the output kernel
      drain_wait(&bars.k_full, 0);
      for (int x = max(0, issued - NST); x < issued; ++x) drain_wait(&bars.q_full[x % NST], (x / NST) & 1);
    }
  } else if (warp == kMma) {
    if (NT > 0) {
      const uint64_t dK = desc_rows(smem_u32(smem)), dQ = desc_rows(smem_u32(smem + C::oQ));
      const uint64_t eK = desc_extra(smem_u32(smem + C::kTile)), eQ = desc_extra(smem_u32(smem + C::oQ + C::kTile));
      constexpr uint32_t id = idesc_bf16(128, 128, false, false);
      if (!warp_wait(&bars.k_full, 0, abort_flag, wlim)) aborted = true;
      for (int t = 0; t < NT && !aborted; ++t) {
        const int s = t % NST;
        if (!warp_wait(&bars.q_full[s], (t / NST) & 1, abort_flag, wlim) ||
            !warp_wait(&bars.s_empty[t % NB], ((t / NB) & 1) ^ 1u, abort_flag, wlim)) {
          aborted = true;
          break;
        }
        tc_after_sync();
        mma_scores<DH, kRows, PL>(tmem + (t % NB) * 128, dK, dQ + s * (C::kStage >> 4));
        if (elect_one()) mma_f16(tmem + (t % NB) * 128, eK, eQ + s * (C::kStage >> 4), id, 1u);
        commit_one(&bars.s_full[t % NB]);
        commit_one(&bars.q_empty[s]);
      }
      if (aborted) {
        commit_one(&bars.drain);
        drain_wait(&bars.drain, 0);
      }
    }
    __syncwarp();
  } else {
    const int half = warp >> 2, col0 = half * 64;
    const int j = j0 + (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const float c = a.sm_scale * kLog2e;
    const float2 cc = make_float2(c, c);
    for (int t = 0; t < NT; ++t) {
      const int i0 = (rt0 + t) * kRows;
      if (!warp_wait(&bars.s_full[t % NB], (t / NB) & 1, abort_flag, wlim)) {
        aborted = true;
        break;
      }
      tc_after_sync();
      const uint32_t tS = tmem + lanes + (t % NB) * 128 + col0;
      const int lo = j - shift - i0 - col0, hi = qr.n - i0 - col0;   // columns lo .. hi - 1 see the key
      const int lo_first = lo - lane;                                // the same for the warp's first key
      float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
      if (lo_first + 31 <= 0 && hi >= 64) {   // all of the warp's
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {   // 32 at a time: registers for three CTAs
          float v[32];
          tmem_ld32(tS + ch * 32, v);
          tmem_ld_wait();
          if (ch == 1) {
            tc_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.s_empty[t % NB]);
          }
#pragma unroll
          for (int q = 0; q < 32; q += 8) {
            const float2 e0 = exp2_pair<0, kWeightPoly>(__fmul2_rn(make_float2(v[q], v[q + 1]), cc));
            const float2 e1 = exp2_pair<1, kWeightPoly>(__fmul2_rn(make_float2(v[q + 2], v[q + 3]), cc));
            const float2 e2 = exp2_pair<2, kWeightPoly>(__fmul2_rn(make_float2(v[q + 4], v[q + 5]), cc));
            const float2 e3 = exp2_pair<3, kWeightPoly>(__fmul2_rn(make_float2(v[q + 6], v[q + 7]), cc));
            s0 = __fadd2_rn(s0, __fadd2_rn(e0, e2));
            s1 = __fadd2_rn(s1, __fadd2_rn(e1, e3));
          }
        }
      } else {
#pragma unroll 1
        for (int ch = 0; ch < 64; ch += 32) {
          if (lo_first >= ch + 32 || hi <= ch) continue;   // none of the warp's
          float v[32];
          tmem_ld32(tS + ch, v);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            const float e = ch + q >= lo && ch + q < hi ? ex2(v[q] * c) : 0.0f;
            if (q & 1) s1.x += e;
            else s0.x += e;
          }
        }
        tc_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.s_empty[t % NB]);
      }
      total += (s0.x + s1.x) + (s0.y + s1.y);
    }
    if (half) half_sum[(warp & 3) * 32 + lane] = total;
  }
  tc_before_sync();
  const bool any_abort = __syncthreads_or(aborted);
  if (any_abort && tid == 0) report(a.dev_status, SPATTEN_E_TIMEOUT);
  if (tid < kRows && j0 + tid < kr.n) {
    const int j = j0 + tid;
    const float sum = any_abort ? 0.0f : (last_nan >= j - shift ? NAN : total + half_sum[tid]);
    if (G > 1) {
      p.part[static_cast<int64_t>(h) * a.total_kv + kr.first + j] = sum;
    } else if (!counted) {   // reported by the output kernel
    } else if (j < a.weight_cap) {
      a.weight[static_cast<int64_t>(pt.b) * a.weight_ld_seq + static_cast<int64_t>(hk) * a.weight_ld_head + j] += sum;
    } else {
      report(a.dev_status, SPATTEN_E_INDEX);
    }
  }
  if (warp == kMma) {
    tc_after_sync();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// =================================================================================================
// SPLIT: float32 q, k and v (blockIdx.y) into three bfloat16 planes each
// =================================================================================================
__global__ void __launch_bounds__(256) prompt_split_kernel(PromptProblem p) {
  grid_dep_trigger();
  grid_dep_wait();
  const spatten_prompt_args& a = p.a;
  const int t = blockIdx.y;
  const float* src = static_cast<const float*>(t == 0 ? a.q : (t == 1 ? a.k : a.v));
  const int64_t ld = t == 0 ? a.q_ld_tok : a.kv_ld_tok;
  const int row = (t == 0 ? a.H : a.H_kv) * a.d_h / 8;   // octets
  const int64_t octets = static_cast<int64_t>(t == 0 ? a.total_q : a.total_kv) * row;
  uint4* dst = reinterpret_cast<uint4*>(p.planes[t]);
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < octets; e += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = octets <= INT32_MAX ? static_cast<int64_t>(static_cast<uint32_t>(e) / static_cast<uint32_t>(row)) : e / row;
    const float4* x = reinterpret_cast<const float4*>(src + r * ld + (e - r * row) * 8);
    const float4 u = x[0], v = x[1];
    uint4 mid, low, hi;
    hi.x = split_pair(make_float2(u.x, u.y), mid.x, low.x);
    hi.y = split_pair(make_float2(u.z, u.w), mid.y, low.y);
    hi.z = split_pair(make_float2(v.x, v.y), mid.z, low.z);
    hi.w = split_pair(make_float2(v.z, v.w), mid.w, low.w);
    dst[e] = hi;
    dst[octets + e] = mid;
    dst[2 * octets + e] = low;
  }
}

// =================================================================================================
// host
// =================================================================================================
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeFn>(f);
}

// [rows][heads][DH] with a row stride of ld elements, read in boxes of 64 rows x 1 head x 64 channels
int32_t make_map(CUtensorMap* m, const void* base, int dh, int heads, int rows, int64_t ld) {
  const EncodeFn enc = encode_fn();
  if (!enc) return SPATTEN_E_UNSUPPORTED;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dh), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(dh) * 2, static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[3] = {64, 1, kBox}, step[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SPATTEN_OK : SPATTEN_E_UNSUPPORTED;
}

// CTAs of the output kernel that cover any offsets: a sequence's rows end in at most one partial tile.
template <class O>
int64_t out_blocks(const spatten_prompt_args& a) {
  const bool pair_heads = O::NQ == 2 && (a.H / a.H_kv) % 2 == 0;
  const int tile_rows = O::NQ == 2 && !pair_heads ? 256 : 128;
  return (static_cast<int64_t>(a.total_q) / tile_rows + a.B) * (pair_heads ? a.H / 2 : a.H);
}

// Splits of the key tiles: as many as leave all CTAs resident at once and each kSplitTiles tiles of a sequence of
// average length (outputs of 16 rows of 16 heads of 64 behind 8000 others: 21 against 111 us unsplit; 500 of 8 heads
// behind 1500: 20 against 32; float32, 16 of 8 heads of 128 behind 1000: 24, with four tiles at least 33, unsplit 63).
template <class O>
int out_splits(const spatten_prompt_args& a) {
  const int64_t most = std::min<int64_t>(O::kCtas * sm_count() / std::max<int64_t>(1, out_blocks<O>(a)), a.total_kv / std::max(1, a.B) / (kSplitTiles * O::KT));
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMaxSplits, most)));
}

template <class O, class W>
int32_t launch(const PromptProblem& p, cudaStream_t st) {
  static DeviceOnce once;
  int dev;
  SPT_TRY(once_per_device(once, &dev, [](int) -> int32_t {
    SPT_CUDA(cudaFuncSetAttribute(prompt_out_kernel<O, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, O::kSmem));
    SPT_CUDA(cudaFuncSetAttribute(prompt_out_kernel<O, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, O::kSmem));
    SPT_CUDA(cudaFuncSetAttribute(prompt_weight_kernel<W>, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kSmem));
    return SPATTEN_OK;
  }));
  const spatten_prompt_args& a = p.a;
  Maps maps;
  if constexpr (O::PL == 1) {
    SPT_TRY(make_map(&maps.q, a.q, O::DH, a.H, a.total_q, a.q_ld_tok));
    SPT_TRY(make_map(&maps.k, a.k, O::DH, a.H_kv, a.total_kv, a.kv_ld_tok));
    SPT_TRY(make_map(&maps.v, a.v, O::DH, a.H_kv, a.total_kv, a.kv_ld_tok));
  } else {
    const int64_t hd = static_cast<int64_t>(a.H) * O::DH, hkd = static_cast<int64_t>(a.H_kv) * O::DH;
    SPT_TRY(make_map(&maps.q, p.planes[0], O::DH, a.H, 3 * a.total_q, hd));
    SPT_TRY(make_map(&maps.k, p.planes[1], O::DH, a.H_kv, 3 * a.total_kv, hkd));
    SPT_TRY(make_map(&maps.v, p.planes[2], O::DH, a.H_kv, 3 * a.total_kv, hkd));
    const int64_t octets = std::max<int64_t>(hd * a.total_q, hkd * a.total_kv) / 8;
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(ceil_div(octets, 256), 16 * sm_count()));
    SPT_TRY(launch_chained(prompt_split_kernel, dim3(blocks, 3), dim3(256), 0, st, 1, p));
  }
  const int64_t q_blocks = out_blocks<O>(a) * p.splits;
  const int64_t k_blocks = (static_cast<int64_t>(a.total_kv) / kRows + a.B) * a.H;
  if (q_blocks > INT32_MAX || k_blocks > INT32_MAX) return SPATTEN_E_UNSUPPORTED;
  const auto out = p.splits > 1 ? prompt_out_kernel<O, true> : prompt_out_kernel<O, false>;
  SPT_TRY(launch_chained(out, dim3(static_cast<unsigned>(q_blocks)), dim3(O::kThreads), O::kSmem, st, 1, p, maps));
  if (p.splits > 1) {
    const auto join = prompt_join_kernel<O::DH, std::conditional_t<O::PL == 1, __nv_bfloat16, float>>;
    SPT_TRY(launch_chained(join, dim3(static_cast<unsigned>(ceil_div(static_cast<int64_t>(a.total_q) * a.H, 8))), dim3(256), 0, st, 1, p));
  }
  if (!a.weight) return SPATTEN_OK;
  SPT_TRY(launch_chained(prompt_weight_kernel<W>, dim3(static_cast<unsigned>(k_blocks)), dim3(W::kThreads), W::kSmem, st, 1, p, maps));
  if (a.H == a.H_kv) return SPATTEN_OK;
  return prompt_reduce_launch(p, st);
}

}  // namespace

bool prompt_tc_supported(const spatten_prompt_args& a) {
  if (a.total_kv < 1) return false;
  // a tensor map holds row strides below 2^40 bytes; float32 operands are planes of a block each, 3 blocks of rows
  return a.dtype == SPATTEN_BF16 ? a.q_ld_tok < (1LL << 38) && a.kv_ld_tok < (1LL << 38)
                                 : a.total_q <= INT32_MAX / 4 && a.total_kv <= INT32_MAX / 4;
}

namespace {

// The tiles of a type and head size: call(output tiles, weight tiles).
template <typename F>
auto with_tiles(const spatten_prompt_args& a, F&& call) {
  if (a.dtype == SPATTEN_BF16)
    return a.d_h == 64 ? call(OutCfg<64, 1, 64, 4>{}, WeightCfg<64, 2, 1, 3>{}) : call(OutCfg<128, 2, 128, 4>{}, WeightCfg<128, 1, 1, 3>{});
  return a.d_h == 64 ? call(OutCfg<64, 1, 64, 2, 3>{}, WeightCfg<64, 1, 2, 2, 3>{}) : call(OutCfg<128, 1, 64, 2, 3>{}, WeightCfg<128, 1, 2, 1, 3>{});
}

}  // namespace

int prompt_tc_splits(const spatten_prompt_args& a) {
  return with_tiles(a, [&](auto o, auto) { return out_splits<decltype(o)>(a); });
}

int32_t prompt_tc_launch(const PromptProblem& p, cudaStream_t st) {
  return with_tiles(p.a, [&](auto o, auto w) { return launch<decltype(o), decltype(w)>(p, st); });
}

}  // namespace spt
