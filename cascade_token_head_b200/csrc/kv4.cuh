// The 4-bit cache's row layout and the bounds shared by its kernels (see spatten.h).
#pragma once

#include "chained.cuh"

namespace spt {

constexpr int kKv4Group = 32;   // channels per scale

// bytes of one row's codes, and its scales
__host__ __device__ constexpr int kv4_row_bytes(int d_h) { return d_h / 2; }
__host__ __device__ constexpr int kv4_groups(int d_h) { return d_h / kKv4Group; }

int32_t kv4_validate(const spatten_kv4_cache& c);

// Rows of sequence b in a packed block: cu[b] .. cu[b+1]-1 (one row per sequence when cu is NULL).
// Offsets that decrease or leave [0, total] give an empty sequence; `bad` says so.
struct PackedRows {
  int first, n;
  bool bad;
};
__device__ __forceinline__ PackedRows packed_rows(const int32_t* cu, int b, int total) {
  if (!cu) return {b, 1, false};
  const int s = cu[b], e = cu[b + 1];
  if (s < 0 || e < s || e > total) return {0, 0, true};
  return {s, e - s, false};
}

// The first sequence that packed row r belongs to (-1: none), by the whole warp: each sequence is asked, so that
// one with bad offsets hides no other.
__device__ __forceinline__ int owner_of_row(const int32_t* cu, int B, int total, int r) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int b0 = 0; b0 < B; b0 += 32) {
    const PackedRows p = b0 + lane < B ? packed_rows(cu, b0 + lane, total) : PackedRows{0, 0, false};
    const uint32_t in = __ballot_sync(0xffffffffu, r >= p.first && r - p.first < p.n);
    if (in) return b0 + __ffs(in) - 1;
  }
  return -1;
}
// The same for a row of each lane's own (rows past total have none).  A binary search finds it where offsets do
// not decrease; rows that it does not find are looked for one by one if a sequence has bad offsets.
__device__ __forceinline__ int owner_of_lanes_row(const int32_t* cu, int B, int total, int r) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= r) lo = mid;
    else hi = mid;
  }
  const PackedRows p = packed_rows(cu, lo, total);
  const bool found = r >= p.first && r - p.first < p.n;
  uint32_t missing = __ballot_sync(0xffffffffu, !found && r < total);
  int b = found ? lo : -1;
  if (!missing) return b;
  bool bad = false;
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < B; i += 32) bad |= packed_rows(cu, i, total).bad;
  if (!__any_sync(0xffffffffu, bad)) return b;
#pragma unroll 1
  for (; missing; missing &= missing - 1) {
    const int lane = __ffs(missing) - 1, owner = owner_of_row(cu, B, total, __shfl_sync(0xffffffffu, r, lane));
    if (lane == (threadIdx.x & 31)) b = owner;
  }
  return b;
}

// The sequence and tile number t, for tiles of `rows` packed rows that start anew at each sequence:
// tiles are counted from the last sequence's last tile backwards, so that a sequence's late rows, which
// see the most keys, are started first (FRONT: from the first sequence's first tile).  Every warp calls
// it whole; b = -1 past the last tile.
struct SeqTile {
  int b, tile;
};
template <bool FRONT = false>
__device__ __forceinline__ SeqTile find_seq_tile(const int32_t* cu, int B, int total, int rows, int t) {
  const int lane = threadIdx.x & 31;
  int all = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    int c = b0 + lane < B ? (packed_rows(cu, b0 + lane, total).n + rows - 1) / rows : 0;
    all += warp_sum_int(c);
  }
  int want = FRONT ? t : all - 1 - t;
  if (want < 0 || want >= all) return {-1, 0};
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int c = b0 + lane < B ? (packed_rows(cu, b0 + lane, total).n + rows - 1) / rows : 0;
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const int sum = __shfl_sync(0xffffffffu, inc, 31);
    if (want < sum) {
      const uint32_t past = __ballot_sync(0xffffffffu, want < inc);
      const int l = __ffs(past) - 1;
      const int before = __shfl_sync(0xffffffffu, inc - c, l);
      return {b0 + l, want - before};
    }
    want -= sum;
  }
  return {-1, 0};
}

// A row count from the device, held to [0, most]; a count outside is reported.
__device__ __forceinline__ int clamp_len(int n, int most, int32_t* status) {
  if (n < 0 || n > most) {
    report(status, SPATTEN_E_INDEX);
    n = n < 0 ? 0 : most;
  }
  return n;
}

__device__ __forceinline__ float bf16_bits_to_float(uint32_t b) { return __uint_as_float(b << 16); }

}  // namespace spt
