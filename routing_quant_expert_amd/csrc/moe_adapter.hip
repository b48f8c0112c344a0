// A shared projection with one low-rank adapter per token (moe_adapter_project):
//   out[t] = W x[t] + factor[a] B[a] (A[a] x[t]),  a = index[t] (-1: W x[t] alone).
//
// Few tokens (or few tiles): the call reads every weight once, so the long
// sums over k are cut into slices, enough for all CUs to read at once
// (k_adapter_part: W and the A of the adapters in use, f32 partial sums), and a
// second launch adds them up with the short products by B (k_adapter_sum, all in f32).
//
// More tokens: they are sorted by adapter (k_adapter_sort), u = factor A x is
// made in f32 by 16 tokens of one adapter (k_adapter_low), and the tiles of
// the projection run over the sorted tokens (k_adapter_main): after its sum
// over k a tile goes on with the products of u and B, adapter by adapter, and
// adds them to the outputs of that adapter's tokens alone: no other token's
// values meet its weights. u enters those products as two 16-bit terms, its
// rounded value and the rounded rest (three where a bf16 product makes an f32
// output), which leave at most 2^-16 of u (bf16 outputs), 2^-24 (f32 of bf16) or
// 2^-22 (fp16, f32 outputs too: the size of the roundings of its own f32 sums; a
// third term costs 5% of 700 tokens of 4096 x 256, rank 64). fp16 has few
// exponents, so a token's u of 64 ranks is scaled by a power of two that brings
// its largest value to their top: nothing is lost above 2^-39 of that value.
//
// One token of 2048 x 4096, rank 16: 9.8 us a call, 4.5 in the reading launch
// (3.7 TB/s) and 4.9 in the joining one, whose time is latency. Workgroups of
// adapters that no token uses end at once, but are launched: 16.8 us beside 1024
// adapters. 48 tokens, 24 adapters of rank 32: 12.4 us. 4096 tokens of 4096 x
// 2048, rank 64: 93 to 98 us (730 to 770 TFLOP/s): sort 7 (in one workgroup), u
// 13 (reading A again for every 16 tokens), tiles 79, where the plain product
// alone takes a library 52.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "moe_gemm.h"
#include "moe_host.h"

namespace moe {
namespace {

constexpr int kTokenTile = 64;   // a wave's lanes hold one token each in k_adapter_part
constexpr int kRowTile = 128;    // the sorted tokens are padded to the largest tile

struct AdapterArgs {
  int adapters, rank, n, k;
  int f32;   // outputs in f32
  int m;
  int64_t x_stride, w_stride, out_stride, a_stride, a_group, b_stride, b_group;
  const float* factor;
  const int32_t* index;
  int32_t* status;
};

// Token t's adapter, -1 for none (and for an index that names none).
__device__ __forceinline__ int adapter_of(const AdapterArgs& a, int t) {
  const int i = a.index[t];
  return (uint32_t)i < (uint32_t)a.adapters ? i : -1;
}
__device__ __forceinline__ bool bad_index(const AdapterArgs& a, int t) {
  const int i = a.index[t];
  return i < -1 || i >= a.adapters;
}
__device__ __forceinline__ float factor_of(const AdapterArgs& a, int i) { return a.factor ? a.factor[i] : 1.0f; }

// ---- few tokens -----------------------------------------------------------

// Whether m tokens take the sliced sums: 64 tokens, or so few tiles of 64 x 64
// that most CUs would have one at most, where the joining launch has no more
// than 2^24 products by B to add. 300 tokens of 2048 x 2048, rank 16: 18.3 us
// against 23.3 sorted; of 901 x 1503: 18 against 42; 500 tokens of 1024 x 1024, rank 64 (2^25): 30 against 21.
bool few_tokens(int n, int rank, int64_t m) {
  return m <= kTokenTile ||
         (m <= 512 && (m + 63) / 64 * ((n + 63) / 64) <= 320 && (double)m * n * rank <= (double)(1 << 24));
}

// Slices of the sum over k: `count` of `len` (a multiple of a step). Two
// workgroups a CU for the projection's own tiles where tokens are few (one
// token of 2048 x 4096: all of W is asked for at once), one where the partial sums themselves are much to move.
struct Slices {
  int count, len;
};
Slices slices_of(int n, int k, int64_t m) {
  const int64_t tiles = (int64_t)((n + 63) / 64) * ((m + kTokenTile - 1) / kTokenTile);
  const int64_t most = (k + 255) / 256, want = ((m <= 16 ? 512 : 256) + tiles - 1) / tiles;
  const int count = (int)(want < most ? want : most);
  const int len = ((k + count - 1) / count + kStep - 1) / kStep * kStep;
  return {(k + len - 1) / len, len};
}

// Tile `t` of a slice: the W tiles, then each adapter's A tiles; partial sums
// [slice][m][n] of W x and [slice][m][rank] of A x (of a token's own adapter).
template <typename T, typename G>
__global__ __launch_bounds__(G::NT, 2) void k_adapter_part(AdapterArgs a, Slices sl, const T* __restrict__ x,
                                                        const T* __restrict__ w, const T* __restrict__ wa,
                                                        float* __restrict__ part, float* __restrict__ upart) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int wt = (a.n + G::kP - 1) / G::kP, rt = (a.rank + G::kP - 1) / G::kP;
  const int slice = blockIdx.y, tile = blockIdx.x, t0 = blockIdx.z * kTokenTile, tokens = min(a.m - t0, kTokenTile);
  const int mine = lane < tokens ? adapter_of(a, t0 + lane) : -1;
  if (a.status && tile == 0 && slice == 0 && threadIdx.x < 64 && lane < tokens && bad_index(a, t0 + lane))
    atomicOr(a.status, MOE_STATUS_BAD_ADAPTER);
  const bool base = tile < wt;
  const int adapter = base ? -1 : (tile - wt) / rt;
  const uint64_t users = __ballot(mine == adapter);
  if (!base && !users) return;   // an adapter that no token uses is not read
  const int p0 = (base ? tile : (tile - wt) % rt) * G::kP, width = base ? a.n : a.rank;
  const int k0 = slice * sl.len, red = min(sl.len, a.k - k0);
  const Operand<T> P = {base ? w + p0 * a.w_stride + k0 : wa + adapter * a.a_group + p0 * a.a_stride + k0,
                        base ? a.w_stride : a.a_stride, min(G::kP, width - p0), nullptr, a.k >= 8};
  const Operand<T> Q = {x + t0 * a.x_stride + k0, a.x_stride, tokens, nullptr, a.k >= 8};
  typename G::Acc acc = {};
  G::run(P, Q, red, lds, acc);
  float* out = (base ? part : upart) + ((int64_t)slice * a.m + t0) * width + p0;
  G::store(acc, out, true, width, width - p0,
           [&](int q) { return q < tokens && (base || (users >> q & 1)) ? q : -1; });
}

// 256 columns of one token: the slices' sums, in order, then the rank terms.
template <typename T, typename U>
__global__ __launch_bounds__(256) void k_adapter_sum(AdapterArgs a, int slices, const T* __restrict__ wb,
                                                     const float* __restrict__ part, const float* __restrict__ upart,
                                                     U* __restrict__ out) {
  __shared__ float u[MOE_ADAPTER_MAX_RANK];
  const int t = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x, col = min(c, a.n - 1);
  const int mine = adapter_of(a, t);
  auto total = [&](const float* from, int width) {
    from += (int64_t)t * width;
    float s = 0.0f;
#pragma unroll 8
    for (int i = 0; i < slices; ++i) s += from[(int64_t)i * a.m * width];
    return s;
  };
  constexpr int kFirst = 4;   // the first 32 ranks of B are asked for with the sums
  const T* b = wb + max(mine, 0) * a.b_group + col * a.b_stride;
  oct<T> first[kFirst];
#pragma unroll
  for (int i = 0; i < kFirst; ++i) first[i] = raw_oct(b + 8 * i, mine >= 0 ? a.rank - 8 * i : 0, a.rank >= 8);
  float s = total(part + col, a.n);
  if (mine >= 0) {
    for (int j = threadIdx.x; j < a.rank; j += 256) u[j] = factor_of(a, mine) * total(upart + j, a.rank);
  }
  __syncthreads();
  if (mine >= 0) {
    auto add = [&](oct<T> o, int j) {
      const f32x8 v = to_f32(o);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i < a.rank) s = fmaf(u[j + i], v[i], s);
    };
#pragma unroll
    for (int i = 0; i < kFirst; ++i) add(placed_oct<T>(first[i], a.rank - 8 * i, a.rank >= 8), 8 * i);
    for (int j = 8 * kFirst; j < a.rank; j += 8) add(load_oct(b + j, a.rank - j, a.rank >= 8), j);
  }
  if (c < a.n) out[t * a.out_stride + c] = (U)s;
}

// ---- more tokens ----------------------------------------------------------

// The tokens in the order of their adapters (those without one first), filled
// up to a tile with rows of no token; and the same rows again adapter by
// adapter in slots, each adapter's filled up to 16 (row -1).
struct Sorted {
  int32_t* token;   // [padded] or -1
  int32_t* owner;   // [padded] the row's adapter, or -1
  int32_t* slots;   // [1] number of slots, a multiple of 16
  int32_t* row;     // [most slots] sorted row, or -1
  int32_t* user;    // [most slots / 16] adapter of 16 slots
  float* u;         // [padded][rank_pad]: factor A x
  int rank_pad;
};

int64_t padded_rows(int64_t m) { return (m + kRowTile - 1) / kRowTile * kRowTile; }
int64_t most_slots(int64_t m, int adapters) {
  const int64_t used = adapters < m ? adapters : m;
  return (m + 15 * used) / 16 * 16;
}
int rank_pad(int rank) { return (rank + kStep - 1) / kStep * kStep; }

// One workgroup: counts, starts and places (of bucket 0, the tokens without an
// adapter, then bucket by bucket). The order of an adapter's tokens depends
// on the order of the atomics; a token's outputs do not depend on its place.
__global__ __launch_bounds__(1024) void k_adapter_sort(AdapterArgs a, Sorted so, int padded) {
  __shared__ int count[MOE_ADAPTER_MAX_ADAPTERS + 1], start[MOE_ADAPTER_MAX_ADAPTERS + 1], slot[MOE_ADAPTER_MAX_ADAPTERS + 1];
  const int tid = threadIdx.x, lane = tid & 63, buckets = a.adapters + 1;
  for (int b = tid; b < buckets; b += 1024) count[b] = 0;
  __syncthreads();
  // Counts the lanes that are there in their buckets (by one lane where all have the same): the lane's place in its own.
  auto add = [&](bool there, int b) -> int {
    const uint64_t lanes = __ballot(there);
    if (!lanes) return 0;
    const int leader = __builtin_ctzll(lanes), first = __shfl(b, leader);
    if (lanes != __ballot(there && b == first)) return there ? atomicAdd(&count[b], 1) : 0;
    int at = 0;
    if (lane == leader) at = atomicAdd(&count[b], __popcll(lanes));
    return __shfl(at, leader) + (int)__popcll(lanes & ((1ull << lane) - 1));
  };
  constexpr int kHeld = 4;   // tokens whose bucket and place a thread keeps
  int held[kHeld], place[kHeld];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int t = tid + 1024 * i;
    held[i] = t < a.m ? adapter_of(a, t) + 1 : 0;
    bad = bad || (t < a.m && bad_index(a, t));
  }
#pragma unroll
  for (int i = 0; i < kHeld; ++i) place[i] = add(tid + 1024 * i < a.m, held[i]);
  if (a.m > 1024 * kHeld) __syncthreads();   // the held tokens take the first places
  for (int t0 = 1024 * kHeld; t0 < a.m; t0 += 1024) {
    const int t = t0 + tid;
    add(t < a.m, t < a.m ? adapter_of(a, t) + 1 : 0);
    bad = bad || (t < a.m && bad_index(a, t));
  }
  if (a.status && bad) atomicOr(a.status, MOE_STATUS_BAD_ADAPTER);
  __syncthreads();
  if (tid < 64) {
    int rows = 0, slots = 0;
    for (int b0 = 0; b0 < buckets; b0 += 64) {
      const int b = b0 + tid, v = b < buckets ? count[b] : 0, w = b > 0 ? (v + 15) / 16 * 16 : 0;
      const int rows_to = wave_scan(v, tid), slots_to = wave_scan(w, tid);
      if (b < buckets) {
        start[b] = rows + rows_to - v;
        slot[b] = slots + slots_to - w;
      }
      rows += __shfl(rows_to, 63);
      slots += __shfl(slots_to, 63);
    }
    if (tid == 0) *so.slots = slots;
  }
  __syncthreads();
  for (int i = a.m + tid; i < padded; i += 1024) {
    so.token[i] = -1;
    so.owner[i] = -1;
  }
  for (int b = 1 + tid; b < buckets; b += 1024) {
    const int v = count[b], end = (v + 15) / 16 * 16;
    for (int i = v; i < end; ++i) so.row[slot[b] + i] = -1;
    for (int i = 0; i < end; i += 16) so.user[(slot[b] + i) / 16] = b - 1;
  }
  auto put = [&](int t, int b, int at) {
    const int row = start[b] + at;
    so.token[row] = t;
    so.owner[row] = b - 1;
    if (b > 0) so.row[slot[b] + at] = row;
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (tid + 1024 * i < a.m) put(tid + 1024 * i, held[i], place[i]);
  if (a.m <= 1024 * kHeld) return;
  // the others' places: counted again, from the held tokens' numbers up
  __syncthreads();
  for (int b = tid; b < buckets; b += 1024) count[b] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kHeld; ++i) add(true, held[i]);
  __syncthreads();
  for (int t0 = 1024 * kHeld; t0 < a.m; t0 += 1024) {
    const int t = t0 + tid, b = t < a.m ? adapter_of(a, t) + 1 : 0;
    const int at = add(t < a.m, b);
    if (t < a.m) put(t, b, at);
  }
}

// u of 16 slots and 64 ranks: the eight waves take every eighth 32 of k, their sums meet in LDS.
constexpr int kLowWaves = 8;
template <typename T, int NA>
__global__ __launch_bounds__(64 * kLowWaves) void k_adapter_low(AdapterArgs a, Sorted so, const T* __restrict__ x,
                                                                const T* __restrict__ wa) {
  __shared__ float red[kLowWaves][16][NA * 16 + 1];
  const int s = blockIdx.x, r0 = blockIdx.y * kStep;
  if (16 * s >= *so.slots) return;
  const int mine = so.user[s];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, part = 8 * (lane >> 4);
  const T* xr = x + max(so.token[max(so.row[16 * s + row], 0)], 0) * a.x_stride + part;
  const T* ar[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i)
    ar[i] = wa + mine * a.a_group + min(r0 + 16 * i + row, a.rank - 1) * a.a_stride + part;
  f32x4 acc[NA] = {};
  int k = 32 * wave;
  auto some = [&](auto count) {   // `count` of the wave's 32 k, all loads at once
    oct<T> xv[count], av[count][NA];
#pragma unroll
    for (int n = 0; n < count; ++n) {
      __builtin_memcpy(&xv[n], xr + k + 32 * kLowWaves * n, 16);
#pragma unroll
      for (int i = 0; i < NA; ++i) __builtin_memcpy(&av[n][i], ar[i] + k + 32 * kLowWaves * n, 16);
    }
#pragma unroll
    for (int n = 0; n < count; ++n)
#pragma unroll
      for (int i = 0; i < NA; ++i) acc[i] = mfma16(av[n][i], xv[n], acc[i]);
    k += 32 * kLowWaves * count;
  };
  while (k + 3 * 32 * kLowWaves + 32 <= a.k) some(std::integral_constant<int, 4>());
  while (k + 32 <= a.k) some(std::integral_constant<int, 1>());
  if (k < a.k) {
    const oct<T> xv = load_oct(xr + k, a.k - k - part, a.k >= 8);
#pragma unroll
    for (int i = 0; i < NA; ++i) acc[i] = mfma16(load_oct(ar[i] + k, a.k - k - part, a.k >= 8), xv, acc[i]);
  }
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][row][16 * i + 4 * (lane >> 4) + r] = acc[i][r];
  __syncthreads();
  const float f = factor_of(a, mine);
  for (int i = threadIdx.x; i < 16 * kStep; i += 64 * kLowWaves) {
    const int slot = i / kStep, j = i % kStep, to = so.row[16 * s + slot];
    if (to < 0) continue;
    float v = 0.0f;
    if (j < NA * 16 && r0 + j < a.rank) {
#pragma unroll
      for (int w = 0; w < kLowWaves; ++w) v += red[w][slot][j];
      v *= f;
    }
    so.u[(int64_t)to * so.rank_pad + r0 + j] = v;
  }
}

// u of a tile's rows and 64 ranks as `PIECES` 16-bit tiles whose sum it is.
// fp16: a row is scaled by the power of two (row_scale) that brings its largest
// finite value to [2^14, 2^15), and its products back: unscaled, values above 65504
// would be infinite, and the second term of values below 2^-3 would meet the
// type's smallest step (a u of 1e-4 kept to 2e-4 of itself). The exponent stays
// within 126, where the scale and its inverse are normal numbers.
template <typename T, typename G, int PIECES>
__device__ __forceinline__ void stage_u(const Sorted& so, int row0, int r0, uint8_t* tiles, float* row_scale) {
  typedef typename G::QT QT;
#pragma unroll
  for (int k = 0; k < QT::kPer; ++k) {
    const int i = QT::position(k);
    int r, row;
    QT::place(i, r, row);
    f32x8 v = {};
    if (so.owner[row0 + row] >= 0) v = load_oct(so.u + (int64_t)(row0 + row) * so.rank_pad + r0 + r, 8, true);
    if constexpr (std::is_same_v<T, fp16_t>) {
      float most = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) most = fmaxf(most, __builtin_isinf(v[e]) ? 0.0f : fabsf(v[e]));
#pragma unroll
      for (int d = 1; d < 8; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
      float scale = 1.0f;
      if (most > 0.0f) scale = ldexpf(1.0f, min(14 - ilogbf(most), 126));
      v = v * scale;
      if (r == 0) row_scale[row] = scale;   // (chunk 0 of the row, wherever it is stored)
    }
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const oct<T> t = __builtin_convertvector(v, oct<T>);
      *reinterpret_cast<oct<T>*>(tiles + p * QT::kBytes + 16 * i) = t;
      const f32x8 back = to_f32(t);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __builtin_isinf(back[e]) ? 0.0f : v[e] - back[e];
    }
  }
}

template <typename T, typename G, int PIECES>
__global__ __launch_bounds__(G::NT, 2) void k_adapter_main(AdapterArgs a, Sorted so, const T* __restrict__ x,
                                                           const T* __restrict__ w, const T* __restrict__ wb,
                                                           void* __restrict__ out) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ float row_scale[G::kQ];
  static_assert(G::PT::kBytes + PIECES * G::QT::kBytes <= G::kLds, "the tiles of u and B fit the ring's LDS");
  const int np = (a.n + G::kP - 1) / G::kP, nq = (a.m + G::kQ - 1) / G::kQ;
  const int64_t total = (int64_t)np * nq, place = xcd_order(blockIdx.x, total);
  if (place >= total) return;
  int qt, pt;
  tile_at(place, nq, np, qt, pt);
  const int p0 = pt * G::kP, row0 = qt * G::kQ, lane = threadIdx.x & 63;
  const Operand<T> P = {w + p0 * a.w_stride, a.w_stride, min(G::kP, a.n - p0), nullptr, a.k >= 8};
  const Operand<T> Q = {x, a.x_stride, G::kQ, so.token + row0, a.k >= 8};
  constexpr int kOwners = (G::kQ + 63) / 64;
  int owner[kOwners];   // of row 64 i + lane of the tile: ascending, but for rows of no token at the end
#pragma unroll
  for (int i = 0; i < kOwners; ++i) owner[i] = so.owner[row0 + 64 * i + lane];
  int mine[G::NQ];      // of the rows whose outputs this lane holds
#pragma unroll
  for (int j = 0; j < G::NQ; ++j) mine[j] = so.owner[row0 + G::wave_q() + 16 * j + (lane & 15)];
  typename G::Acc acc = {};
  G::run(P, Q, a.k, lds, acc);

  // the first adapter of the tile above `done`, or -1
  auto after = [&](int done) {
    int next = -1;
#pragma unroll
    for (int i = kOwners - 1; i >= 0; --i) {
      const uint64_t rows = __ballot(owner[i] > done);
      if (rows) next = __builtin_amdgcn_readlane(owner[i], __builtin_ctzll(rows));
    }
    return next;
  };
  const int first = after(-1);
  oct<T> bv[G::PT::kPer];
  auto b_of = [&](int adapter, int r0) -> Operand<T> {
    return {wb + adapter * a.b_group + p0 * a.b_stride + r0, a.b_stride, min(G::kP, a.n - p0), nullptr, a.rank >= 8};
  };
  auto ask_b = [&](int adapter, int r0) {
    const Operand<T> B = b_of(adapter, r0);
    typename G::PT::Off off[G::PT::kPer];
    G::PT::template offsets<false>(B, off);
    G::PT::load(B, B.base, off, a.rank - r0, bv);
  };
  for (int r0 = 0; first >= 0 && r0 < a.rank; r0 += kStep) {
    uint8_t* const ut = lds + G::PT::kBytes;
    ask_b(first, r0);
    lds_barrier();
    stage_u<T, G, PIECES>(so, row0, r0, ut, row_scale);
    for (int next = first, then; next >= 0; next = then) {
      G::PT::store(b_of(next, r0), a.rank - r0, bv, lds);
      then = after(next);
      if (then >= 0) ask_b(then, r0);   // on its way while this one's products run
      lds_barrier();
#pragma unroll
      for (int j = 0; j < G::NQ; ++j) {
        if (!__ballot(mine[j] == next)) continue;
        f32x4 low[G::NP] = {};
        G::template multiply_row<PIECES>(lds, ut, j, low);
        float back = 1.0f;
        if constexpr (std::is_same_v<T, fp16_t>) back = 1.0f / row_scale[G::wave_q() + 16 * j + (lane & 15)];
#pragma unroll
        for (int i = 0; i < G::NP; ++i)
          if (mine[j] == next) acc[i][j] = acc[i][j] + low[i] * back;
      }
      lds_barrier();
    }
  }
  uint8_t* o = (uint8_t*)out + (int64_t)p0 * (a.f32 ? 4 : 2);
  G::store(acc, o, a.f32, a.out_stride, a.n - p0, [&](int q) { return so.token[row0 + q]; });
}

int check_adapters(const moe_adapters* p, int64_t m) {
  if (!p) return fail(MOE_EINVAL, "adapters is NULL%s%lld");
  if (p->type != MOE_TYPE_BF16 && p->type != MOE_TYPE_FP16)
    return fail(MOE_EINVAL, "adapters: type must be MOE_TYPE_BF16 or MOE_TYPE_FP16%s (%lld)", "", p->type);
  if (p->out_type != p->type && p->out_type != MOE_TYPE_F32)
    return fail(MOE_EINVAL, "adapters: out_type must be type or MOE_TYPE_F32%s (%lld)", "", p->out_type);
  if (p->n_adapters < 1 || p->rank < 1 || p->n < 1 || p->k < 1)
    return fail(MOE_EINVAL, "adapters: n_adapters, rank, n and k must be >= 1%s%lld");
  if (p->n_adapters > MOE_ADAPTER_MAX_ADAPTERS || p->rank > MOE_ADAPTER_MAX_RANK)
    return fail(MOE_EUNSUPPORTED, "adapters: more adapters or a larger rank than the limits%s%lld");
  if (p->x_stride < p->k || p->w_stride < p->k || p->a_stride < p->k || p->b_stride < p->rank || p->out_stride < p->n)
    return fail(MOE_EINVAL, "adapters: a row stride is below its row%s%lld");
  if (p->a_group_stride < (int64_t)(p->rank - 1) * p->a_stride + p->k ||
      p->b_group_stride < (int64_t)(p->n - 1) * p->b_stride + p->rank)
    return fail(MOE_EINVAL, "adapters: the distance of two adapters is below one%s%lld");
  for (int64_t v : {p->x_stride, p->w_stride, p->a_stride, p->b_stride, p->out_stride})
    if (v > MOE_GROUPED_MAX_STRIDE) return fail(MOE_EUNSUPPORTED, "adapters: a row stride is too large%s (%lld)", "", v);
  if (!p->a || !p->b) return fail(MOE_EINVAL, "adapters: a and b must be non-NULL%s%lld");
  if ((uintptr_t)p->a % 2 || (uintptr_t)p->b % 2 || (uintptr_t)p->factor % 4)
    return fail(MOE_EINVAL, "adapters: a pointer is not aligned to its elements%s%lld");
  if (m < 1) return fail(MOE_EINVAL, "m must be >= 1%s (m %lld)", "", m);
  if (m > MOE_ADAPTER_MAX_TOKENS) return fail(MOE_EUNSUPPORTED, "adapters: too many tokens%s (m %lld)", "", m);
  return MOE_OK;
}

size_t round256(size_t v) { return (v + 255) & ~(size_t)255; }

// Bytes of the parts of the workspace: few tokens: the partial sums; more: the sorted rows and u.
struct AdapterWs {
  size_t part, upart, owner, slots, row, user, u, total;
};
AdapterWs adapter_ws(const moe_adapters& p, int64_t m) {
  AdapterWs w = {};
  if (few_tokens(p.n, p.rank, m)) {
    const Slices s = slices_of(p.n, p.k, m);
    w.upart = round256((size_t)s.count * m * p.n * 4);
    w.total = w.upart + round256((size_t)s.count * m * p.rank * 4);
  } else {
    const size_t rows = (size_t)padded_rows(m), slots = (size_t)most_slots(m, p.n_adapters);
    w.owner = rows * 4;
    w.slots = 2 * w.owner;
    w.row = w.slots + 256;
    w.user = w.row + round256(slots * 4);
    w.u = w.user + round256(slots / 16 * 4);
    w.total = w.u + rows * rank_pad(p.rank) * 4;
  }
  return w;
}

template <typename T, bool DMA, int BQ>
int launch_part(const AdapterArgs& a, Slices sl, const T* x, const T* w, const T* wa, float* part, float* upart,
                hipStream_t s) {
  typedef Gemm<T, false, false, 64, BQ, 4, 1, 4, DMA> G;
  const int64_t tiles = (a.n + 63) / 64 + (int64_t)a.adapters * ((a.rank + 63) / 64);
  return launch_tiles<k_adapter_part<T, G>>("adapters", dim3((unsigned)tiles, sl.count, (a.m + kTokenTile - 1) / kTokenTile),
                                            G::NT, G::kLds, s, a, sl, x, w, wa, part, upart);
}

template <typename T, bool DMA>
int launch_few(const AdapterArgs& a, const T* x, const T* w, const T* wa, const T* wb, void* out, uint8_t* ws,
               const AdapterWs& l, hipStream_t s) {
  const Slices sl = slices_of(a.n, a.k, a.m);
  float *part = (float*)(ws + l.part), *upart = (float*)(ws + l.upart);
  const int r = a.m <= 16   ? launch_part<T, DMA, 16>(a, sl, x, w, wa, part, upart, s)
                : a.m <= 32 ? launch_part<T, DMA, 32>(a, sl, x, w, wa, part, upart, s)
                            : launch_part<T, DMA, 64>(a, sl, x, w, wa, part, upart, s);
  if (r) return r;
  const dim3 grid((a.n + 255) / 256, a.m);
  if (a.f32) k_adapter_sum<T, float><<<grid, dim3(256), 0, s>>>(a, sl.count, wb, part, upart, (float*)out);
  else k_adapter_sum<T, T><<<grid, dim3(256), 0, s>>>(a, sl.count, wb, part, upart, (T*)out);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MOE_OK : hip_fail(e, "adapters");
}

template <typename T, typename G>
int launch_main(const AdapterArgs& a, const Sorted& so, const T* x, const T* w, const T* wb, void* out, hipStream_t s) {
  const int64_t tiles = (int64_t)((a.m + G::kQ - 1) / G::kQ) * ((a.n + G::kP - 1) / G::kP);
  const int64_t blocks = tile_blocks(tiles, G::NT);
  if (!blocks) return fail(MOE_EUNSUPPORTED, "adapters: too many tiles for one launch%s (%lld)", "", tiles);
  const dim3 grid((unsigned)blocks);
  if constexpr (std::is_same_v<T, bf16_t>) {
    if (a.f32) return launch_tiles<k_adapter_main<T, G, 3>>("adapters", grid, G::NT, G::kLds, s, a, so, x, w, wb, out);
  }
  return launch_tiles<k_adapter_main<T, G, 2>>("adapters", grid, G::NT, G::kLds, s, a, so, x, w, wb, out);
}

template <typename T, bool DMA>
int launch_many(const AdapterArgs& a, const T* x, const T* w, const T* wa, const T* wb, void* out, uint8_t* ws,
                const AdapterWs& l, hipStream_t s) {
  const Sorted so = {(int32_t*)ws, (int32_t*)(ws + l.owner), (int32_t*)(ws + l.slots), (int32_t*)(ws + l.row),
                     (int32_t*)(ws + l.user), (float*)(ws + l.u), rank_pad(a.rank)};
  k_adapter_sort<<<dim3(1), dim3(1024), 0, s>>>(a, so, (int)padded_rows(a.m));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_fail(e, "adapters");
  const dim3 grid((unsigned)(most_slots(a.m, a.adapters) / 16), (a.rank + kStep - 1) / kStep), threads(64 * kLowWaves);
  if (a.rank <= 16) k_adapter_low<T, 1><<<grid, threads, 0, s>>>(a, so, x, wa);
  else if (a.rank <= 32) k_adapter_low<T, 2><<<grid, threads, 0, s>>>(a, so, x, wa);
  else k_adapter_low<T, 4><<<grid, threads, 0, s>>>(a, so, x, wa);
  e = hipGetLastError();
  if (e != hipSuccess) return hip_fail(e, "adapters");
  // Tiles by their number, as for the grouped products: 64 x 64 where larger ones would leave CUs idle (1000 tokens of
  // 1024 x 1024: 19 us), 256 x 128 from three a CU on with long sums (at two a CU, 4096 tokens of 4096 x 2048: 95 us of either).
  const int64_t rows = (a.m + 127) / 128;
  if (rows * ((a.n + 127) / 128) < 256)
    return launch_main<T, Gemm<T, false, false, 64, 64, 2, 2, 4, DMA, true>>(a, so, x, w, wb, out, s);
  if constexpr (DMA) {
    if (rows * ((a.n + 255) / 256) >= 768 && a.k >= 1024)
      return launch_main<T, Gemm<T, false, false, 256, 128, 4, 2, 3, DMA, true>>(a, so, x, w, wb, out, s);
  }
  return launch_main<T, Gemm<T, false, false, 128, 128, 2, 2, 2, DMA, true>>(a, so, x, w, wb, out, s);
}

template <typename T>
int launch_adapters(const moe_adapters& p, const AdapterArgs& a, const void* x, const void* w, void* out, uint8_t* ws,
                    hipStream_t s) {
  const AdapterWs l = adapter_ws(p, a.m);
  const T *xt = (const T*)x, *wt = (const T*)w, *wa = (const T*)p.a, *wb = (const T*)p.b;
  const bool dma = rows16(x, a.x_stride) && rows16(w, a.w_stride);
  if (!few_tokens(a.n, a.rank, a.m))
    return dma ? launch_many<T, true>(a, xt, wt, wa, wb, out, ws, l, s)
               : launch_many<T, false>(a, xt, wt, wa, wb, out, ws, l, s);
  return dma && rows16(p.a, a.a_stride) && a.a_group % 8 == 0
             ? launch_few<T, true>(a, xt, wt, wa, wb, out, ws, l, s)
             : launch_few<T, false>(a, xt, wt, wa, wb, out, ws, l, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_adapter_workspace_bytes(const moe_adapters* p, int64_t max_m) {
  if (check_adapters(p, max_m)) return 0;
  // (the number of slices falls where m grows)
  size_t most = adapter_ws(*p, max_m).total;
  for (int64_t m = 1; m < max_m && few_tokens(p->n, p->rank, m); ++m) most = std::max(most, adapter_ws(*p, m).total);
  return most;
}

int moe_adapter_project(const moe_adapters* p, const void* x, const void* w, const int32_t* index, int64_t m,
                        void* out, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  if (int r = check_adapters(p, m)) return r;
  if (!x || !w || !index || !out) return fail(MOE_EINVAL, "adapters: x, w, index and out must be non-NULL%s%lld");
  if ((uintptr_t)x % 2 || (uintptr_t)w % 2 || (uintptr_t)out % elem_bytes(p->out_type) || (uintptr_t)index % 4 ||
      (uintptr_t)status % 4)
    return fail(MOE_EINVAL, "adapters: a pointer is not aligned to its elements%s%lld");
  if (!ws) return fail(MOE_EINVAL, "workspace is NULL%s%lld");
  if ((uintptr_t)ws & 255) return fail(MOE_EINVAL, "workspace must be 256-byte aligned%s%lld");
  const size_t need = adapter_ws(*p, m).total;
  if (ws_bytes < need) return fail(MOE_EWORKSPACE, "workspace too small%s: need %lld bytes", "", (long long)need);
  const AdapterArgs a = {p->n_adapters, p->rank, p->n, p->k, p->out_type == MOE_TYPE_F32, (int)m,
                         p->x_stride, p->w_stride, p->out_stride, p->a_stride, p->a_group_stride, p->b_stride,
                         p->b_group_stride, p->factor, index, status};
  return p->type == MOE_TYPE_BF16
             ? launch_adapters<bf16_t>(*p, a, x, w, out, (uint8_t*)ws, (hipStream_t)stream)
             : launch_adapters<fp16_t>(*p, a, x, w, out, (uint8_t*)ws, (hipStream_t)stream);
}

}  // extern "C"
