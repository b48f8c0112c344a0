// Products grouped by expert (moe_grouped_*): rows sorted by group, group g's
// rows offsets[g] .. offsets[g+1] against its own 16-bit weight W[g] (n x k).
//
//   forward  y[r]  = W[g(r)] x[r]                    P = W rows,    Q = x rows,  sum over k
//   input    dx[r] = W[g(r)]^T dy[r]                 P = W columns, Q = dy rows, sum over n
//   weight   dW[g] = sum over g's rows dy[r] x[r]^T  P = x columns, Q = dy columns
//
// Few rows a group: bound by HBM, every used weight is read once (48 rows over
// 384 groups of 2048 x 4096: 135 us, 6.0 TB/s; 12288 rows: 1120 us, 5.9 TB/s).
// Many: by the matrix instructions and what the ragged groups leave of them
// (16384 rows over 32 groups of 4096 x 2048: input gradient 335 to 353 us from
// card to card, 780 to 820 TFLOP/s, forward 333; four even groups of 4096 x
// 4096: 1150 TFLOP/s; a library product of this size class reaches 1355 to 1450
// on even sizes). The weight gradient of the same rows writes 1.07 GB in f32:
// 546 to 555 us, 341 without its stores.
//
// The offsets stay on the device: the grid is an upper bound of the tiles (a
// group adds at most one partial tile), every wave finds its tile from the
// offsets by two wave-wide prefix sums, and workgroups past the last tile end
// at once.
#include <hip/hip_runtime.h>

#include "moe_gemm.h"
#include "moe_host.h"

namespace moe {
namespace {

struct GroupedArgs {
  const int32_t* offsets;
  int32_t* status;
  int groups, rows;
  int n, k;
  int f32;   // outputs in f32
  int64_t x_stride, y_stride, w_stride, w_group;
};

// Rows are cut at the edges 0, offsets[0..groups], rows: entry e = g + 1 is
// group g, the first and last entries are the rows of no group. Edges are
// clamped to [0, rows], so that no offsets lead outside the buffers.
__device__ __forceinline__ int edge(const GroupedArgs& a, int e) {
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
__device__ __forceinline__ Tile find_tile(const GroupedArgs& a, int np) {
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

// The first workgroup reports offsets that do not ascend or leave [0, rows].
__device__ __forceinline__ void report(const GroupedArgs& a) {
  if (!a.status || blockIdx.x) return;
  bool bad = false;
  for (int g = threadIdx.x; g < a.groups; g += blockDim.x) {
    const int lo = a.offsets[g], hi = a.offsets[g + 1];
    bad = bad || lo < 0 || hi < lo || hi > a.rows;
  }
  if (bad) atomicOr(a.status, MOE_STATUS_BAD_OFFSETS);
}

// No rows: nothing to write, but the offsets are looked at.
__global__ __launch_bounds__(64) void k_grouped_offsets(GroupedArgs a) { report(a); }

// Forward (WCOL false): in = x, out = y. Input gradient (WCOL true): in = dy, out = dx.
template <typename T, bool WCOL, typename G>
__global__ __launch_bounds__(G::NT, 2) void k_grouped(GroupedArgs a, const T* __restrict__ in, const T* __restrict__ w,
                                                   void* __restrict__ out) {
  extern __shared__ __align__(16) uint8_t lds[];
  report(a);
  const int width = WCOL ? a.k : a.n, red = WCOL ? a.n : a.k;
  Tile t = find_tile<G::kQ>(a, (width + G::kP - 1) / G::kP);
  // (the same in every lane: into scalar registers)
  t.group = __builtin_amdgcn_readfirstlane(t.group);
  t.row = __builtin_amdgcn_readfirstlane(t.row);
  t.rows = __builtin_amdgcn_readfirstlane(t.rows);
  t.p = __builtin_amdgcn_readfirstlane(t.p);
  if (t.rows <= 0) return;
  const bool none = t.group < 0 || t.group >= a.groups;
  const int p0 = t.p * G::kP;
  const int64_t in_stride = WCOL ? a.y_stride : a.x_stride, out_stride = WCOL ? a.x_stride : a.y_stride;
  const Operand<T> P = {w + (none ? 0 : t.group) * a.w_group + (WCOL ? p0 : p0 * a.w_stride), a.w_stride, WCOL ? width - p0 : min(G::kP, width - p0), nullptr,
                        a.k >= 8};
  const Operand<T> Q = {in + t.row * in_stride, in_stride, t.rows, nullptr, red >= 8};
  typename G::Acc acc = {};
  G::run(P, Q, none ? 0 : red, lds, acc);
  uint8_t* o = (uint8_t*)out + (t.row * out_stride + p0) * (a.f32 ? 4 : 2);
  G::store(acc, o, a.f32, out_stride, width - p0, [&](int q) { return q < t.rows ? q : -1; });
}

template <typename T, typename G>
__global__ __launch_bounds__(G::NT, 2) void k_grouped_dw(GroupedArgs a, const T* __restrict__ dy, const T* __restrict__ x,
                                                      void* __restrict__ dw) {
  extern __shared__ __align__(16) uint8_t lds[];
  report(a);
  const int np = (a.k + G::kP - 1) / G::kP, nq = (a.n + G::kQ - 1) / G::kQ;
  const int64_t total = (int64_t)np * nq * a.groups, place = xcd_order(blockIdx.x, total);
  if (place >= total) return;
  const int g = (int)(place / (np * nq)), in = (int)(place % (np * nq));
  int qt, pt;
  tile_at(in, nq, np, qt, pt);
  const int p0 = pt * G::kP, q0 = qt * G::kQ;
  const int lo = edge(a, g + 1), hi = max(lo, edge(a, g + 2));
  const Operand<T> P = {x + lo * a.x_stride + p0, a.x_stride, a.k - p0, nullptr, a.k >= 8};
  const Operand<T> Q = {dy + lo * a.y_stride + q0, a.y_stride, a.n - q0, nullptr, a.n >= 8};
  typename G::Acc acc = {};
  G::run(P, Q, hi - lo, lds, acc);
  uint8_t* o = (uint8_t*)dw + (g * a.w_group + q0 * a.w_stride + p0) * (a.f32 ? 4 : 2);
  G::store(acc, o, a.f32, a.w_stride, a.k - p0, [&](int q) { return q0 + q < a.n ? q : -1; });
}

// The weight gradients' tiles in chunks of `wide` x `tall` (q x p) tiles of one
// group. Chunks go to the XCDs in turn, so that each finds a chunk's operands in
// its own L2 and gets a share of every group's work; its workgroups take its tiles in turn.
// The tiles follow one another without a pause (Gemm::run_on): the sum of a
// group of 512 rows is 8 steps, as long as a tile's start and end take.
struct Chunks {
  int wide, tall, nq, np;   // tiles of a chunk, chunks of a group
};

template <typename T, typename G>
__global__ __launch_bounds__(G::NT, 2) void k_grouped_dw_ring(GroupedArgs a, Chunks ch, const T* __restrict__ dy,
                                                              const T* __restrict__ x, void* __restrict__ dw) {
  extern __shared__ __align__(16) uint8_t lds[];
  report(a);
  const int np = (a.k + G::kP - 1) / G::kP, nq = (a.n + G::kQ - 1) / G::kQ;
  const int per = ch.wide * ch.tall, chunks = a.groups * ch.nq * ch.np, stride = gridDim.x / 8;
  struct Place {
    int g, p0, q0;
  };
  auto same = [](int v) { return __builtin_amdgcn_readfirstlane(v); };   // (divisions are done in vector registers)
  int t = (int)(blockIdx.x / 8) - stride;
  typename G::Ring ring(lds);
  Place cur = {}, then = {};
  auto next = [&]() -> int {
    for (;;) {
      t += stride;
      const int c = same(t / per) * 8 + (int)(blockIdx.x % 8), in = t - t / per * per;
      if (c >= chunks) return 0;
      const int g = same(c / (ch.nq * ch.np)), rest = c % (ch.nq * ch.np);
      const int qt = same(rest / ch.np * ch.wide + in / ch.tall), pt = same(rest % ch.np * ch.tall + in % ch.tall);
      if (qt >= nq || pt >= np) continue;
      then = {g, pt * G::kP, qt * G::kQ};
      const int lo = same(edge(a, g + 1)), hi = same(edge(a, g + 2));
      ring.start({x + lo * a.x_stride + then.p0, a.x_stride, a.k - then.p0, nullptr, true},
                 {dy + lo * a.y_stride + then.q0, a.y_stride, a.n - then.q0, nullptr, true}, max(hi - lo, 0));
      return 1;
    }
  };
  for (int more = next(); more;) {
    cur = then;
    typename G::Acc acc = {};
    more = G::run_on(ring, acc, next);
    uint8_t* o = (uint8_t*)dw + (cur.g * a.w_group + cur.q0 * a.w_stride + cur.p0) * (a.f32 ? 4 : 2);
    G::store(acc, o, a.f32, a.w_stride, a.k - cur.p0, [&](int q) { return cur.q0 + q < a.n ? q : -1; });
    ring.stores = cur.q0 + G::kQ <= a.n && cur.p0 + G::kP <= a.k ? G::kStores : 0;
  }
}

enum Way { kForward, kInput, kWeight };

int check_grouped(const moe_grouped* g, int64_t rows) {
  if (!g) return fail(MOE_EINVAL, "grouped is NULL%s%lld");
  if (g->type != MOE_TYPE_BF16 && g->type != MOE_TYPE_FP16)
    return fail(MOE_EINVAL, "grouped: type must be MOE_TYPE_BF16 or MOE_TYPE_FP16%s (%lld)", "", g->type);
  if (g->out_type != g->type && g->out_type != MOE_TYPE_F32)
    return fail(MOE_EINVAL, "grouped: out_type must be type or MOE_TYPE_F32%s (%lld)", "", g->out_type);
  if (g->n_groups < 1) return fail(MOE_EINVAL, "grouped: n_groups must be >= 1%s (%lld)", "", g->n_groups);
  if (g->n_groups > MOE_GROUPED_MAX_GROUPS)
    return fail(MOE_EUNSUPPORTED, "grouped: n_groups above MOE_GROUPED_MAX_GROUPS%s (%lld)", "", g->n_groups);
  if (g->n < 1 || g->k < 1) return fail(MOE_EINVAL, "grouped: n and k must be >= 1%s%lld");
  if (g->x_stride < g->k || g->y_stride < g->n || g->w_stride < g->k)
    return fail(MOE_EINVAL, "grouped: a row stride is below its row%s%lld");
  if (g->w_group_stride < (int64_t)(g->n - 1) * g->w_stride + g->k)
    return fail(MOE_EINVAL, "grouped: w_group_stride is below one weight%s (%lld)", "", g->w_group_stride);
  if (g->x_stride > MOE_GROUPED_MAX_STRIDE || g->y_stride > MOE_GROUPED_MAX_STRIDE ||
      g->w_stride > MOE_GROUPED_MAX_STRIDE)
    return fail(MOE_EUNSUPPORTED, "grouped: a row stride above MOE_GROUPED_MAX_STRIDE%s%lld");
  if (rows < 0) return fail(MOE_EINVAL, "grouped: rows must be >= 0%s (%lld)", "", rows);
  if (rows > MOE_GROUPED_MAX_ROWS)   // (row numbers rounded up to a tile or a step stay within 32 bits)
    return fail(MOE_EUNSUPPORTED, "grouped: rows above MOE_GROUPED_MAX_ROWS%s (%lld)", "", rows);
  return MOE_OK;
}

GroupedArgs grouped_args(const moe_grouped& g, const int32_t* offsets, int64_t rows, int32_t* status) {
  return {offsets, status, g.n_groups, (int)rows, g.n, g.k, g.out_type == MOE_TYPE_F32,
          g.x_stride, g.y_stride, g.w_stride, g.w_group_stride};
}

template <auto Kernel, typename G, typename... A>
int launch(int64_t tiles, hipStream_t s, A... args) {
  const int64_t blocks = tile_blocks(tiles, G::NT);
  if (!blocks) return fail(MOE_EUNSUPPORTED, "grouped: too many tiles for one launch%s (%lld)", "", tiles);
  return launch_tiles<Kernel>("grouped", dim3((unsigned)blocks), G::NT, G::kLds, s, args...);
}

// At most so many row tiles of q rows: a group adds at most one partial tile.
int64_t row_tiles(const GroupedArgs& a, int q) {
  const int64_t some = a.groups + 2 < a.rows ? a.groups + 2 : a.rows;   // entries that can have rows
  return (a.rows + (q - 1) * some) / q;
}

template <typename T, bool WCOL, typename G>
int launch_rows(const GroupedArgs& a, const void* in, const void* w, void* out, hipStream_t s) {
  const int width = WCOL ? a.k : a.n;
  return launch<k_grouped<T, WCOL, G>, G>(row_tiles(a, G::kQ) * ((width + G::kP - 1) / G::kP), s, a, (const T*)in,
                                          (const T*)w, out);
}

template <typename T, bool WCOL, bool DMA>
int launch_rows_as(const GroupedArgs& a, const void* in, const void* w, void* out, hipStream_t s) {
  // (The offsets are on the device: the tile goes by the mean of the groups. Where few groups have most of the rows
  // it is too small: 5000 rows, all but 800 in one of 384 groups of 2048 x 4096, take 339 us in tiles of 16 rows, 166 of 64.)
  const int64_t mean = a.rows / a.groups;
  const int width = WCOL ? a.k : a.n;
  if (mean < 16) return launch_rows<T, WCOL, Gemm<T, WCOL, false, 128, 16, 4, 1, 4, DMA>>(a, in, w, out, s);
  // Few tiles: smaller ones, so that more CUs share the work. 100 rows of one group of 2048 x 2048: 10.5 us in
  // tiles of 16 rows, 15 of 64, 20 of 128; 1200 rows over 4 groups of 1024 x 2048: 15.5 us of 64, 23.5 of 128.
  if (row_tiles(a, 64) * ((width + 127) / 128) < 96)
    return launch_rows<T, WCOL, Gemm<T, WCOL, false, 128, 16, 4, 1, 4, DMA>>(a, in, w, out, s);
  if (mean < 64 || row_tiles(a, 128) * ((width + 127) / 128) < 300)
    return launch_rows<T, WCOL, Gemm<T, WCOL, false, 128, 64, 2, 2, 3, DMA>>(a, in, w, out, s);
  if constexpr (DMA) {
    // One workgroup a CU with a third step in flight, where there are three
    // tiles a CU and sums long enough for its fill and drain; otherwise two
    // workgroups a CU. 16384 rows over 32 groups of 4096 x 2048: forward 333 us
    // against 342, input gradient 337 against 341; forward of 8000 over 16 of 4096 x 512: 69 against 63.
    const int red = WCOL ? a.n : a.k;
    if (row_tiles(a, 128) * ((width + 255) / 256) >= 768 && red >= 1024)
      return launch_rows<T, WCOL, Gemm<T, WCOL, false, 256, 128, 4, 2, 3, DMA>>(a, in, w, out, s);
  }
  return launch_rows<T, WCOL, Gemm<T, WCOL, false, 128, 128, 2, 2, 2, DMA>>(a, in, w, out, s);
}

template <typename T, typename G>
int launch_dw(const GroupedArgs& a, const void* dy, const void* x, void* dw, hipStream_t s) {
  const int64_t tiles = (int64_t)((a.k + G::kP - 1) / G::kP) * ((a.n + G::kQ - 1) / G::kQ) * a.groups;
  return launch<k_grouped_dw<T, G>, G>(tiles, s, a, (const T*)dy, (const T*)x, dw);
}

template <typename T, typename G>
int launch_dw_ring(const GroupedArgs& a, int at_once, const void* dy, const void* x, void* dw, hipStream_t s) {
  const int np = (a.k + G::kP - 1) / G::kP, nq = (a.n + G::kQ - 1) / G::kQ;
  int wide = nq < 8 ? nq : 8, tall = np;
  auto parts = [](int n, int d) { return (n + d - 1) / d; };
  while ((int64_t)a.groups * parts(nq, wide) * parts(np, tall) < 64 && wide * tall > 1) {   // a share for every XCD
    if (tall > wide || wide == 1) tall = parts(tall, 2);
    else wide = parts(wide, 2);
  }
  const Chunks ch = {wide, tall, parts(nq, wide), parts(np, tall)};
  const int64_t tiles = (int64_t)np * nq * a.groups;
  if ((int64_t)a.groups * ch.nq * ch.np * wide * tall >= INT32_MAX / 16)
    return fail(MOE_EUNSUPPORTED, "grouped: too many tiles for one launch%s (%lld)", "", tiles);
  return launch_tiles<k_grouped_dw_ring<T, G>>("grouped", dim3(tiles < at_once ? (tiles + 7) / 8 * 8 : at_once),
                                               G::NT, G::kLds, s, a, ch, (const T*)dy, (const T*)x, dw);
}

template <typename T>
int launch_dw_aligned(const GroupedArgs& a, const void* dy, const void* x, void* dw, hipStream_t s) {
  // Four tiles a CU and more: the larger tile, one workgroup a CU with a third step in flight. 16384 rows over 32
  // groups of 4096 x 2048 (16384 small tiles): 551 us against 612; 4000 over 8 of 512 x 1024 (256): 21 against 16.
  const int64_t tiles = (int64_t)((a.k + 255) / 256) * ((a.n + 127) / 128) * a.groups;
  if (tiles >= 1024) return launch_dw_ring<T, Gemm<T, true, true, 256, 128, 4, 2, 3, true>>(a, 256, dy, x, dw, s);
  return launch_dw_ring<T, Gemm<T, true, true, 128, 128, 2, 2, 2, true>>(a, 512, dy, x, dw, s);
}

template <typename T>
int launch_way(Way way, const GroupedArgs& a, const void* in, const void* w, void* out, hipStream_t s) {
  if (way == kForward)
    return rows16(in, a.x_stride) && rows16(w, a.w_stride) && a.w_group % 8 == 0
               ? launch_rows_as<T, false, true>(a, in, w, out, s)
               : launch_rows_as<T, false, false>(a, in, w, out, s);
  if (way == kInput)
    return rows16(in, a.y_stride) && rows16(w, a.w_stride) && a.w_group % 8 == 0 && a.k % 8 == 0
               ? launch_rows_as<T, true, true>(a, in, w, out, s)
               : launch_rows_as<T, true, false>(a, in, w, out, s);
  return rows16(in, a.y_stride) && rows16(w, a.x_stride) && a.n % 8 == 0 && a.k % 8 == 0
             ? launch_dw_aligned<T>(a, in, w, out, s)
             : launch_dw<T, Gemm<T, true, true, 128, 128, 2, 2, 2, false>>(a, in, w, out, s);
}

int grouped(Way way, const moe_grouped* g, const void* in, const void* w, const int32_t* offsets, int64_t rows,
            void* out, int32_t* status, void* stream) {
  if (int r = check_grouped(g, rows)) return r;
  if (!offsets) return fail(MOE_EINVAL, "grouped: offsets must be non-NULL%s%lld");
  if (way != kWeight && rows == 0) {   // nothing to write
    if (!status) return MOE_OK;
    if ((uintptr_t)offsets % 4 || (uintptr_t)status % 4)
      return fail(MOE_EINVAL, "grouped: a pointer is not aligned to its elements%s%lld");
    k_grouped_offsets<<<dim3(1), dim3(64), 0, (hipStream_t)stream>>>(grouped_args(*g, offsets, rows, status));
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? MOE_OK : hip_fail(e, "grouped");
  }
  if ((rows && !in) || ((rows || way != kWeight) && !w) || !out)
    return fail(MOE_EINVAL, "grouped: operands and output must be non-NULL%s%lld");
  const size_t es = elem_bytes(g->out_type);
  if ((uintptr_t)in % 2 || (uintptr_t)w % 2 || (uintptr_t)out % es || (uintptr_t)offsets % 4 || (uintptr_t)status % 4)
    return fail(MOE_EINVAL, "grouped: a pointer is not aligned to its elements%s%lld");
  const GroupedArgs a = grouped_args(*g, offsets, rows, status);
  const hipStream_t s = (hipStream_t)stream;
  return g->type == MOE_TYPE_BF16 ? launch_way<bf16_t>(way, a, in, w, out, s)
                                  : launch_way<fp16_t>(way, a, in, w, out, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_grouped_forward(const moe_grouped* g, const void* x, const void* w, const int32_t* offsets, int64_t rows,
                        void* y, int32_t* status, void* stream) {
  return grouped(kForward, g, x, w, offsets, rows, y, status, stream);
}

int moe_grouped_backward_x(const moe_grouped* g, const void* dy, const void* w, const int32_t* offsets, int64_t rows,
                           void* dx, int32_t* status, void* stream) {
  return grouped(kInput, g, dy, w, offsets, rows, dx, status, stream);
}

int moe_grouped_backward_w(const moe_grouped* g, const void* dy, const void* x, const int32_t* offsets, int64_t rows,
                           void* dw, int32_t* status, void* stream) {
  return grouped(kWeight, g, dy, x, offsets, rows, dw, status, stream);
}

}  // extern "C"
