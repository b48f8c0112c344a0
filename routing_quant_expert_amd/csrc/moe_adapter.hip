// A shared projection with one low-rank adapter per token (moe_adapter_project):
//   out[t] = W x[t] + factor[a] B[a] (A[a] x[t]),  a = index[t] (-1: W x[t] alone).
//
// Few tokens (m <= 64): the call reads every weight once, so the long sums over
// k are cut into slices, enough for all CUs to read at once (k_adapter_part: W
// and the A of the adapters in use, f32 partial sums), and a second launch adds
// them up with the short products by B (k_adapter_sum, all in f32).
//
// More tokens: they are sorted by adapter (k_adapter_sort), every adapter's
// tokens filled up to whole 16-row slots, u = factor A x is made once per slot
// in f32 (k_adapter_low), and the tiles of the projection run over the sorted
// slots (k_adapter_main): after its sum over k a tile goes on with u and B as
// further terms of the same sums, adapter by adapter, only in the 16-row slots
// of that adapter: no other token's values meet its weights. u enters those
// products as two 16-bit terms, its rounded value and the rounded rest (three
// where a bf16 product makes an f32 output), so that it is exact to 2^-16 of
// itself at least (2^-24 for f32 outputs of either type, 2^-22 for fp16).
#include <hip/hip_runtime.h>

#include "moe_gemm.h"
#include "moe_host.h"

namespace moe {
namespace {

constexpr int kFewTokens = 64;        // a wave's lanes hold one token each in k_adapter_part
constexpr int kSlotTile = 128;        // the sorted slots are padded to the largest tile

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

// Slices of the sum over k: `count` of `len` (a multiple of a step).
struct Slices {
  int count, len;
};
Slices slices_of(int n, int k) {
  const int tiles = (n + 63) / 64, most = (k + 255) / 256;
  int count = (384 + tiles - 1) / tiles;
  count = count < most ? count : most;
  const int len = ((k + count - 1) / count + kStep - 1) / kStep * kStep;
  return {(k + len - 1) / len, len};
}

// Tile `t` of a slice: the W tiles, then each adapter's A tiles; partial sums
// [slice][m][n] of W x and [slice][m][rank] of A x (of a token's own adapter).
template <typename T, typename G>
__global__ __launch_bounds__(G::NT) void k_adapter_part(AdapterArgs a, Slices sl, const T* __restrict__ x,
                                                        const T* __restrict__ w, const T* __restrict__ wa,
                                                        float* __restrict__ part, float* __restrict__ upart) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int wt = (a.n + G::kP - 1) / G::kP, rt = (a.rank + G::kP - 1) / G::kP;
  const int slice = blockIdx.y, tile = blockIdx.x;
  const int mine = lane < a.m ? adapter_of(a, lane) : -1;
  if (a.status && tile == 0 && slice == 0 && threadIdx.x < 64 && lane < a.m && bad_index(a, lane))
    atomicOr(a.status, MOE_STATUS_BAD_ADAPTER);
  const bool base = tile < wt;
  const int adapter = base ? -1 : (tile - wt) / rt;
  const uint64_t users = __ballot(mine == adapter);
  if (!base && !users) return;   // an adapter that no token uses is not read
  const int p0 = (base ? tile : (tile - wt) % rt) * G::kP, width = base ? a.n : a.rank;
  const int k0 = slice * sl.len, red = min(sl.len, a.k - k0);
  const Operand<T> P = {base ? w + p0 * a.w_stride + k0 : wa + adapter * a.a_group + p0 * a.a_stride + k0,
                        base ? a.w_stride : a.a_stride, min(G::kP, width - p0), nullptr};
  const Operand<T> Q = {x + k0, a.x_stride, a.m, nullptr};
  typename G::Acc acc = {};
  G::run(P, Q, red, lds, acc);
  float* out = (base ? part : upart) + (int64_t)slice * a.m * width + p0;
  G::store(acc, out, true, width, width - p0,
           [&](int q) { return q < a.m && (base || (users >> q & 1)) ? q : -1; });
}

template <typename T, typename U>
__global__ __launch_bounds__(256) void k_adapter_sum(AdapterArgs a, int slices, const T* __restrict__ wb,
                                                     const float* __restrict__ part, const float* __restrict__ upart,
                                                     U* __restrict__ out) {
  __shared__ float u[MOE_ADAPTER_MAX_RANK];
  const int t = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
  const int mine = adapter_of(a, t);
  if (mine >= 0) {
    for (int j = threadIdx.x; j < a.rank; j += 256) {
      float s = 0.0f;
      for (int i = 0; i < slices; ++i) s += upart[((int64_t)i * a.m + t) * a.rank + j];
      u[j] = factor_of(a, mine) * s;
    }
  }
  __syncthreads();
  if (c >= a.n) return;
  float s = 0.0f;
  for (int i = 0; i < slices; ++i) s += part[((int64_t)i * a.m + t) * a.n + c];
  if (mine >= 0) {
    const T* b = wb + mine * a.b_group + c * a.b_stride;
    for (int j = 0; j < a.rank; j += 8) {
      const f32x8 v = to_f32(load_oct(b + j, a.rank - j));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i < a.rank) s = fmaf(u[j + i], v[i], s);
    }
  }
  out[t * a.out_stride + c] = (U)s;
}

// ---- more tokens ----------------------------------------------------------

// The sorted slots: tokens without an adapter, then adapter by adapter, each
// filled up to 16 slots with empty ones (token -1), the whole up to a tile.
struct Sorted {
  int32_t* slots;   // [1] their number, a multiple of 16
  int32_t* token;   // [most]
  int32_t* owner;   // [most / 16] adapter of 16 slots, or -1
  float* u;         // [most][rank_pad]: factor A x
  int rank_pad;
};

int64_t most_slots(int64_t m, int adapters) {
  const int64_t used = adapters + 1 < m ? adapters + 1 : m;
  return (m + 15 * used + kSlotTile - 1) / kSlotTile * kSlotTile;
}
int rank_pad(int rank) { return (rank + kStep - 1) / kStep * kStep; }

// One workgroup: counts, starts and places. The places of an adapter's tokens
// among its own slots depend on the order of the atomics; a token's outputs do not depend on its place.
__global__ __launch_bounds__(1024) void k_adapter_sort(AdapterArgs a, Sorted so) {
  __shared__ int count[MOE_ADAPTER_MAX_ADAPTERS + 1], start[MOE_ADAPTER_MAX_ADAPTERS + 2];
  const int tid = threadIdx.x, buckets = a.adapters + 1;
  for (int b = tid; b < buckets; b += 1024) count[b] = 0;
  __syncthreads();
  bool bad = false;
  for (int t = tid; t < a.m; t += 1024) {
    atomicAdd(&count[adapter_of(a, t) + 1], 1);
    bad = bad || bad_index(a, t);
  }
  if (a.status && bad) atomicOr(a.status, MOE_STATUS_BAD_ADAPTER);
  __syncthreads();
  if (tid < 64) {
    int sum = 0;
    for (int b0 = 0; b0 < buckets; b0 += 64) {
      const int v = b0 + tid < buckets ? (count[b0 + tid] + 15) / 16 * 16 : 0;
      const int incl = wave_scan(v, tid);
      if (b0 + tid < buckets) start[b0 + tid] = sum + incl - v;
      sum += __shfl(incl, 63);
    }
    if (tid == 0) start[buckets] = sum;
  }
  __syncthreads();
  const int total = start[buckets], padded = (total + kSlotTile - 1) / kSlotTile * kSlotTile;
  for (int b = tid; b < buckets; b += 1024)
    for (int i = start[b] + count[b]; i < start[b + 1]; ++i) so.token[i] = -1;
  for (int i = total + tid; i < padded; i += 1024) so.token[i] = -1;
  for (int s = tid; s < padded / 16; s += 1024) {
    int lo = 0, hi = buckets;   // the last bucket that starts at or before the 16 slots
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (start[mid] <= 16 * s) lo = mid;
      else hi = mid;
    }
    so.owner[s] = 16 * s < total ? lo - 1 : -1;
  }
  if (tid == 0) *so.slots = total;
  __syncthreads();
  for (int t = tid; t < a.m; t += 1024) {
    const int b = adapter_of(a, t) + 1;
    so.token[start[b] + atomicSub(&count[b], 1) - 1] = t;
  }
}

// u of 16 slots and 64 ranks: the four waves take every fourth 32 of k, their sums meet in LDS.
template <typename T, int NA>
__global__ __launch_bounds__(256) void k_adapter_low(AdapterArgs a, Sorted so, const T* __restrict__ x,
                                                     const T* __restrict__ wa) {
  __shared__ float red[4][16][NA * 16 + 1];
  const int s = blockIdx.x, r0 = blockIdx.y * kStep;
  if (16 * s >= *so.slots) return;
  const int mine = so.owner[s];
  if (mine < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, part = 8 * (lane >> 4);
  const T* xr = x + max(so.token[16 * s + row], 0) * a.x_stride + part;
  const T* ar[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i)
    ar[i] = wa + mine * a.a_group + min(r0 + 16 * i + row, a.rank - 1) * a.a_stride + part;
  f32x4 acc[NA] = {};
  int k = 32 * wave;
#pragma unroll 4
  for (; k + 32 <= a.k; k += 128) {
    oct<T> xv, av[NA];
    __builtin_memcpy(&xv, xr + k, 16);
#pragma unroll
    for (int i = 0; i < NA; ++i) __builtin_memcpy(&av[i], ar[i] + k, 16);
#pragma unroll
    for (int i = 0; i < NA; ++i) acc[i] = mfma16(av[i], xv, acc[i]);
  }
  if (k < a.k) {
    const oct<T> xv = load_oct(xr + k, a.k - k - part);
#pragma unroll
    for (int i = 0; i < NA; ++i) acc[i] = mfma16(load_oct(ar[i] + k, a.k - k - part), xv, acc[i]);
  }
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][row][16 * i + 4 * (lane >> 4) + r] = acc[i][r];
  __syncthreads();
  const float f = factor_of(a, mine);
  for (int i = threadIdx.x; i < 16 * kStep; i += 256) {
    const int slot = i / kStep, j = i % kStep;
    float v = 0.0f;
    if (j < NA * 16 && r0 + j < a.rank)
      v = f * ((red[0][slot][j] + red[1][slot][j]) + (red[2][slot][j] + red[3][slot][j]));
    so.u[(int64_t)(16 * s + slot) * so.rank_pad + r0 + j] = v;
  }
}

// u of a tile's slots and 64 ranks as `PIECES` 16-bit tiles whose sum it is.
// fp16: a row whose largest value would pass the type's range is scaled by a
// power of two (row_scale), and its sums beside it.
template <typename T, typename G, int PIECES>
__device__ __forceinline__ void stage_u(const Sorted& so, int slot0, int r0, uint8_t* tiles, float* row_scale) {
  typedef typename G::QT QT;
#pragma unroll
  for (int k = 0; k < QT::kPer; ++k) {
    const int i = QT::position(k);
    int r, row;
    QT::place(i, r, row);
    f32x8 v = {};
    if (so.owner[(slot0 + row) / 16] >= 0) v = load_oct(so.u + (int64_t)(slot0 + row) * so.rank_pad + r0 + r, 8);
    if constexpr (std::is_same_v<T, fp16_t>) {
      float most = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(v[e]));
#pragma unroll
      for (int d = 1; d < 8; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
      float scale = 1.0f;
      if (most > 32768.0f && most < INFINITY) scale = ldexpf(1.0f, 14 - ilogbf(most));
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
__global__ __launch_bounds__(G::NT) void k_adapter_main(AdapterArgs a, Sorted so, const T* __restrict__ x,
                                                        const T* __restrict__ w, const T* __restrict__ wb,
                                                        void* __restrict__ out) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ float row_scale[G::kQ];
  static_assert(G::PT::kBytes + PIECES * G::QT::kBytes <= G::kLds, "the tiles of u and B fit the ring's LDS");
  const int np = (a.n + G::kP - 1) / G::kP, nq = (*so.slots + G::kQ - 1) / G::kQ;
  const int64_t total = (int64_t)np * nq, place = xcd_order(blockIdx.x, total);
  if (place >= total) return;
  int qt, pt;
  tile_at(place, nq, np, qt, pt);
  const int p0 = pt * G::kP, slot0 = qt * G::kQ;
  const Operand<T> P = {w + p0 * a.w_stride, a.w_stride, min(G::kP, a.n - p0), nullptr};
  const Operand<T> Q = {x, a.x_stride, G::kQ, so.token + slot0};
  typename G::Acc acc = {};
  G::run(P, Q, a.k, lds, acc);

  int owner[G::kQ / 16], any = -1;
#pragma unroll
  for (int j = 0; j < G::kQ / 16; ++j) {
    owner[j] = __builtin_amdgcn_readfirstlane(so.owner[slot0 / 16 + j]);
    any = max(any, owner[j]);
  }
  for (int r0 = 0; any >= 0 && r0 < a.rank; r0 += kStep) {
    uint8_t* const ut = lds + G::PT::kBytes;
    lds_barrier();
    stage_u<T, G, PIECES>(so, slot0, r0, ut, row_scale);
    bool scaled = false;
    if constexpr (std::is_same_v<T, fp16_t>) {
      lds_barrier();
#pragma unroll
      for (int j = 0; j < G::NQ; ++j) {
        const float s = row_scale[G::wave_q() + 16 * j + (threadIdx.x & 15)];
        if (__ballot(s != 1.0f)) {
          scaled = true;
#pragma unroll
          for (int i = 0; i < G::NP; ++i) acc[i][j] = acc[i][j] * s;
        }
      }
    }
    for (int done = -1;;) {   // the adapters of the tile, ascending
      int next = INT32_MAX;
#pragma unroll
      for (int j = 0; j < G::kQ / 16; ++j)
        if (owner[j] > done) next = min(next, owner[j]);
      if (next == INT32_MAX) break;
      uint32_t some = 0;
#pragma unroll
      for (int j = 0; j < G::kQ / 16; ++j) some |= owner[j] == next ? 1u << j : 0u;
      const Operand<T> B = {wb + next * a.b_group + p0 * a.b_stride + r0, a.b_stride, min(G::kP, a.n - p0), nullptr};
      typename G::PT::Off off[G::PT::kPer];
      oct<T> v[G::PT::kPer];
      G::PT::template offsets<false>(B, off);
      G::PT::load(B, B.base, off, a.rank - r0, v);
      G::PT::store(v, lds);
      lds_barrier();
#pragma unroll
      for (int p = 0; p < PIECES; ++p) G::compute_some(lds, ut + p * G::QT::kBytes, some, acc);
      lds_barrier();
      done = next;
    }
    if constexpr (std::is_same_v<T, fp16_t>) {
      if (scaled) {
#pragma unroll
        for (int j = 0; j < G::NQ; ++j) {
          const float s = 1.0f / row_scale[G::wave_q() + 16 * j + (threadIdx.x & 15)];
#pragma unroll
          for (int i = 0; i < G::NP; ++i) acc[i][j] = acc[i][j] * s;
        }
      }
    }
  }
  uint8_t* o = (uint8_t*)out + (int64_t)p0 * (a.f32 ? 4 : 2);
  G::store(acc, o, a.f32, a.out_stride, a.n - p0, [&](int q) { return so.token[slot0 + q]; });
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

// Bytes of the parts of the workspace: few tokens: the partial sums; more: slots, tokens, owners, u.
struct AdapterWs {
  size_t part, upart, slots, token, owner, u, total;
};
AdapterWs adapter_ws(const moe_adapters& p, int64_t m) {
  AdapterWs w = {};
  if (m <= kFewTokens) {
    const Slices s = slices_of(p.n, p.k);
    w.upart = round256((size_t)s.count * m * p.n * 4);
    w.total = w.upart + round256((size_t)s.count * m * p.rank * 4);
  } else {
    const size_t most = (size_t)most_slots(m, p.n_adapters);
    w.token = 256;
    w.owner = w.token + round256(most * 4);
    w.u = w.owner + round256(most / 16 * 4);
    w.total = w.u + round256(most * rank_pad(p.rank) * 4);
  }
  return w;
}

template <typename T, bool DMA, int BQ>
int launch_part(const AdapterArgs& a, Slices sl, const T* x, const T* w, const T* wa, float* part, float* upart,
                hipStream_t s) {
  typedef Gemm<T, false, false, 64, BQ, 4, 1, 6, DMA> G;
  const int64_t tiles = (a.n + 63) / 64 + (int64_t)a.adapters * ((a.rank + 63) / 64);
  return launch_tiles<k_adapter_part<T, G>>("adapters", dim3((unsigned)tiles, sl.count), G::NT, G::kLds, s, a, sl, x, w,
                                            wa, part, upart);
}

template <typename T, bool DMA>
int launch_few(const AdapterArgs& a, const T* x, const T* w, const T* wa, const T* wb, void* out, uint8_t* ws,
               const AdapterWs& l, hipStream_t s) {
  const Slices sl = slices_of(a.n, a.k);
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

template <typename T, typename G, int PIECES>
int launch_main(const AdapterArgs& a, const Sorted& so, const T* x, const T* w, const T* wb, void* out, hipStream_t s) {
  const int64_t tiles = most_slots(a.m, a.adapters) / G::kQ * ((a.n + G::kP - 1) / G::kP);
  const int64_t blocks = tile_blocks(tiles, G::NT);
  if (!blocks) return fail(MOE_EUNSUPPORTED, "adapters: too many tiles for one launch%s (%lld)", "", tiles);
  return launch_tiles<k_adapter_main<T, G, PIECES>>("adapters", dim3((unsigned)blocks), G::NT, G::kLds, s, a, so, x, w,
                                                    wb, out);
}

template <typename T, bool DMA>
int launch_many(const AdapterArgs& a, const T* x, const T* w, const T* wa, const T* wb, void* out, uint8_t* ws,
                const AdapterWs& l, hipStream_t s) {
  const Sorted so = {(int32_t*)ws, (int32_t*)(ws + l.token), (int32_t*)(ws + l.owner), (float*)(ws + l.u),
                     rank_pad(a.rank)};
  k_adapter_sort<<<dim3(1), dim3(1024), 0, s>>>(a, so);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_fail(e, "adapters");
  const dim3 grid((unsigned)(most_slots(a.m, a.adapters) / 16), (a.rank + kStep - 1) / kStep);
  if (a.rank <= 16) k_adapter_low<T, 1><<<grid, dim3(256), 0, s>>>(a, so, x, wa);
  else if (a.rank <= 32) k_adapter_low<T, 2><<<grid, dim3(256), 0, s>>>(a, so, x, wa);
  else k_adapter_low<T, 4><<<grid, dim3(256), 0, s>>>(a, so, x, wa);
  e = hipGetLastError();
  if (e != hipSuccess) return hip_fail(e, "adapters");
  typedef Gemm<T, false, false, 64, 64, 2, 2, 4, DMA, true> Small;
  typedef Gemm<T, false, false, 128, 128, 2, 2, 2, DMA, true> Large;
  const bool small = a.m <= 512;
  if (std::is_same_v<T, bf16_t> && a.f32)
    return small ? launch_main<T, Small, 3>(a, so, x, w, wb, out, s) : launch_main<T, Large, 3>(a, so, x, w, wb, out, s);
  return small ? launch_main<T, Small, 2>(a, so, x, w, wb, out, s) : launch_main<T, Large, 2>(a, so, x, w, wb, out, s);
}

template <typename T>
int launch_adapters(const moe_adapters& p, const AdapterArgs& a, const void* x, const void* w, void* out, uint8_t* ws,
                    hipStream_t s) {
  const AdapterWs l = adapter_ws(p, a.m);
  const T *xt = (const T*)x, *wt = (const T*)w, *wa = (const T*)p.a, *wb = (const T*)p.b;
  const bool dma = rows16(x, a.x_stride) && rows16(w, a.w_stride);
  if (a.m > kFewTokens)
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
  const size_t few = adapter_ws(*p, max_m < kFewTokens ? max_m : kFewTokens).total;
  const size_t all = adapter_ws(*p, max_m).total;
  return few > all ? few : all;
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
