// Rows sorted by group whose offsets stay on the device: the grid is an upper
// bound of the tiles (a group adds at most one partial tile), every wave finds
// its tile from the offsets by two wave-wide prefix sums, and workgroups past
// the last tile end at once.
#pragma once

#include "moe_gemm.h"

namespace moe {

struct Groups {
  const int32_t* offsets;
  int32_t* status;
  int groups, rows;
};

// Rows are cut at the edges 0, offsets[0..groups], rows: entry e = g + 1 is
// group g, the first and last entries are the rows of no group. Edges are
// clamped to [0, rows], so that no offsets lead outside the buffers.
__device__ __forceinline__ int edge(const Groups& a, int e) {
  if (e <= 0) return 0;
  if (e > a.groups + 1) return a.rows;
  return min(max(a.offsets[e - 1], 0), a.rows);
}

struct Tile {
  int group;        // groups or -1: the rows of no group
  int row, rows;    // first row and rows of the tile (0: no tile)
  int p;            // tile along the output's columns
};

// The tile of this workgroup: `np` column tiles for every BQ rows of an entry.
// Lane l sums the tiles of the entries U l .. U l + U - 1; the wave's prefix
// sums give the lane, and the prefix sums of that lane's entries the entry.
template <int BQ>
__device__ __forceinline__ Tile find_tile(const Groups& a, int np) {
  const int lane = threadIdx.x & 63, entries = a.groups + 2, U = (entries + 63) / 64;
  auto tiles = [](int lo, int hi) { return hi > lo ? (hi - lo + BQ - 1) / BQ : 0; };
  int sum = 0;
  const int lo0 = edge(a, lane * U);
  int lo = lo0;
  for (int u = 0; u < U; ++u) {
    const int e = lane * U + u;
    if (e >= entries) break;
    const int hi = edge(a, e + 1);
    sum += tiles(lo, hi);
    lo = hi;
  }
  const int incl = wave_scan(sum, lane);
  const int64_t total = (int64_t)__builtin_amdgcn_readlane(incl, 63) * np;
  const int64_t place = xcd_order(blockIdx.x, total);
  if (place >= total) return {0, 0, 0, 0};
  const int t = (int)(place / np);
  const uint64_t lanes = __ballot(incl > t);
  if (!lanes) return {0, 0, 0, 0};   // (counts of offsets that do not ascend may wrap)
  const int sel = __builtin_ctzll(lanes);
  // the sums of the entries before, and the entry's own tiles and rows
  int s = 0, first = __builtin_amdgcn_readlane(incl - sum, sel), n_rt, glo, ghi;
  if (U == 1) {   // (a lane has one entry: its edges are there)
    n_rt = __builtin_amdgcn_readlane(sum, sel);
    glo = __builtin_amdgcn_readlane(lo0, sel);
    ghi = __builtin_amdgcn_readlane(lo, sel);
  } else {
    const int e = sel * U + lane;
    const bool mine = lane < U && e < entries;
    const int elo = mine ? edge(a, e) : 0, ehi = mine ? edge(a, e + 1) : 0;
    const int cnt = tiles(elo, ehi);
    const int incl2 = first + wave_scan(cnt, lane);
    const uint64_t hits = __ballot(incl2 > t);
    if (!hits) return {0, 0, 0, 0};
    s = __builtin_ctzll(hits);
    first = __builtin_amdgcn_readlane(incl2 - cnt, s);
    n_rt = __builtin_amdgcn_readlane(cnt, s);
    glo = __builtin_amdgcn_readlane(elo, s);
    ghi = __builtin_amdgcn_readlane(ehi, s);
  }
  int rt, pt;
  tile_at(place - (int64_t)first * np, n_rt, np, rt, pt);
  if (rt < 0 || rt >= n_rt) return {0, 0, 0, 0};
  return {sel * U + s - 1, glo + rt * BQ, min(BQ, ghi - (glo + rt * BQ)), pt};
}

// The workgroup's tile in scalar registers (it is the same in every lane).
template <typename G>
__device__ __forceinline__ Tile my_tile(const Groups& a, int width) {
  Tile t = find_tile<G::kQ>(a, (width + G::kP - 1) / G::kP);
  t.group = __builtin_amdgcn_readfirstlane(t.group);
  t.row = __builtin_amdgcn_readfirstlane(t.row);
  t.rows = __builtin_amdgcn_readfirstlane(t.rows);
  t.p = __builtin_amdgcn_readfirstlane(t.p);
  return t;
}

// (Of operands that need not lie in one allocation.)
template <typename T>
__device__ __forceinline__ int64_t elements_between(const T* a, const T* b) {
  return ((int64_t)(intptr_t)b - (int64_t)(intptr_t)a) / (int64_t)sizeof(T);
}

// The first workgroup reports offsets that do not ascend or leave [0, rows].
__device__ __forceinline__ void report(const Groups& a) {
  if (!a.status || blockIdx.x) return;
  bool bad = false;
  for (int g = threadIdx.x; g < a.groups; g += blockDim.x) {
    const int lo = a.offsets[g], hi = a.offsets[g + 1];
    bad = bad || lo < 0 || hi < lo || hi > a.rows;
  }
  if (bad) atomicOr(a.status, MOE_STATUS_BAD_OFFSETS);
}

// No rows: nothing to write, but the offsets are looked at.
static __global__ __launch_bounds__(64) void k_offsets(Groups a) { report(a); }

inline int launch_offsets(const char* what, const Groups& a, hipStream_t s) {
  k_offsets<<<dim3(1), dim3(64), 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MOE_OK : hip_fail(e, what);
}

template <auto Kernel, typename G, typename... A>
int launch_rows_of_tiles(const char* what, int64_t tiles, hipStream_t s, A... args) {
  const int64_t blocks = tile_blocks(tiles, G::NT);
  if (!blocks) return fail(MOE_EUNSUPPORTED, "%s: too many tiles for one launch (%lld)", what, tiles);
  return launch_tiles<Kernel>(what, dim3((unsigned)blocks), G::NT, G::kLds, s, args...);
}

// At most so many row tiles of q rows: a group adds at most one partial tile.
inline int64_t row_tiles(const Groups& a, int q) {
  const int64_t some = a.groups + 2 < a.rows ? a.groups + 2 : a.rows;   // entries that can have rows
  return (a.rows + (q - 1) * some) / q;
}

// About so many: half a partial tile a group. (What a launch rule compares; the grid is the bound.)
inline int64_t likely_row_tiles(const Groups& a, int q) {
  return a.groups == 1 ? (a.rows + q - 1) / q : a.rows / q + (a.groups < a.rows ? a.groups : a.rows) / 2;
}

// Rounds of `tiles` workgroups of which `at_once` run at a time. (The tiles of several groups are guessed: on a tie there is one more.)
inline int64_t rounds(const Groups& a, int64_t tiles, int at_once) {
  return a.groups == 1 ? (tiles + at_once - 1) / at_once : tiles / at_once + 1;
}

}  // namespace moe
