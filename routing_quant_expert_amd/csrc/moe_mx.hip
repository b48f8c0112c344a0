// Microscaled 4-bit floats (moe_mx_*): rows to and from the format, and
// products grouped by expert with both operands in it.
//
//   quantise    block of 32: t = max |v|; X = 2^(floor(log2 t) - 2), or the least power of two with t <= 6 X;
//               element = v / X to the nearest of 0 .5 1 1.5 2 3 4 6, ties to even, 6 past it
//   forward     y[r] = W[e] x[r]                               P = W rows, Q = x rows, sum over k
//   gated       h[r] = act(Wg[e] x[r]) * (Wu[e] x[r])          P = 16 rows of Wg and 16 of Wu in turn
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "moe_activation.h"
#include "moe_groups.h"
#include "moe_host.h"
#include "moe_mx_gemm.h"

namespace moe {
namespace {

// ---- rows ------------------------------------------------------------------------
// A thread takes 8 neighbouring elements, four threads a block of 32, and each
// thread kChunksEach such chunks at once: bound by HBM (65536 x 4096 bf16 there and back in 252 us, 5.4 TB/s;
// with 2 chunks 266, with 8 261).
constexpr int kRowThreads = 256, kChunksEach = 4;

struct RowArgs {
  int64_t rows, x_stride, code_stride, scale_stride;
  int k, chunks;      // chunks of 8 in a row, whole blocks
  uint32_t over;      // ceil(2^32 / chunks)
  int ceil;
};

struct Chunk {
  int64_t row;
  int at;   // its first element
  int n;    // elements there (below 1: none)
};

// The thread's u-th chunk: chunks are counted through the rows; a workgroup's first one in 64 bits, the others from there.
struct Chunks {
  int64_t row0;
  uint32_t in0;
  __device__ explicit Chunks(const RowArgs& a) {
    const int64_t first = (int64_t)blockIdx.x * (kRowThreads * kChunksEach);
    row0 = first / a.chunks;
    in0 = (uint32_t)(first - row0 * a.chunks);
  }
  __device__ __forceinline__ Chunk operator()(const RowArgs& a, int u) const {
    const uint32_t t = in0 + threadIdx.x + kRowThreads * u;
    uint32_t row = __umulhi(t, a.over);   // at most one too large (t < 2^32)
    int in = (int)(t - row * a.chunks);
    if (in < 0) {
      --row;
      in += a.chunks;
    }
    const int64_t r = row0 + row;
    return {r, 8 * in, r < a.rows ? a.k - 8 * in : 0};
  }
};

__device__ __forceinline__ uint32_t max_of_four(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppXor1, 0xf, 0xf, true));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppXor2, 0xf, 0xf, true));
}

// The largest magnitude of 8 elements, as an f32's bits: they order like the values, infinities and NaN above all. (So do
// those of the 16-bit types, two at a time.)
template <typename T>
__device__ __forceinline__ uint32_t top_of(oct<T> v) {
  if constexpr (sizeof(T) == 2) {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    uint32_t w[4];
    __builtin_memcpy(w, &v, sizeof(w));
    u16x2 m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu);
    m[0] = __builtin_elementwise_max(__builtin_elementwise_max(m[0], m[1]), __builtin_elementwise_max(m[2], m[3]));
    const unsigned short lo = m[0][0], hi = m[0][1], top = lo > hi ? lo : hi;
    if constexpr (std::is_same_v<T, bf16_t>) return (uint32_t)top << 16;
    else return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(fp16_t, top));
  } else {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float one = v[e];   // (a bit cast of the vector's element itself takes the first one's bits)
      top = max(top, __builtin_bit_cast(uint32_t, one) & 0x7fffffffu);
    }
    return top;
  }
}

// 8 elements divided by `by`, a power of two, to codes (rounds to nearest even, 6 at most).
template <typename T>
__device__ __forceinline__ uint32_t codes_of(oct<T> v, float by) {
  uint32_t q = 0;
  if constexpr (sizeof(T) == 4) {
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], by, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], by, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], by, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], by, 3);
  } else {
    typedef T pair __attribute__((ext_vector_type(2)));
    pair p[4];
    __builtin_memcpy(p, &v, sizeof(p));
    if constexpr (std::is_same_v<T, bf16_t>) {
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, p[0], by, 0);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, p[1], by, 1);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, p[2], by, 2);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, p[3], by, 3);
    } else {
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, p[0], by, 0);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, p[1], by, 1);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, p[2], by, 2);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, p[3], by, 3);
    }
  }
  return q;
}

// WHOLE: k is a multiple of 8, a chunk all there or not at all. (65536 x 4096 bf16 148 us; 158 with the elements made f32
// first and every chunk's end looked at.)
template <typename T, bool WHOLE>
__global__ __launch_bounds__(kRowThreads) void k_mx_quantise(RowArgs a, const T* __restrict__ x, uint8_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
  const Chunks chunks(a);
  const bool room = WHOLE || a.k >= 8;
  oct<T> raw[kChunksEach];
  Chunk c[kChunksEach];
#pragma unroll
  for (int u = 0; u < kChunksEach; ++u) {
    c[u] = chunks(a, u);
    raw[u] = raw_oct(x + c[u].row * a.x_stride + c[u].at, WHOLE && c[u].n > 0 ? 8 : c[u].n, room);
  }
#pragma unroll
  for (int u = 0; u < kChunksEach; ++u) {
    const oct<T> v = WHOLE ? raw[u] : placed_oct<T>(raw[u], c[u].n, room);   // (zeros where nothing is there)
    const uint32_t top = max_of_four(top_of<T>(v));
    // (past 1.5 times its power of two, t is more than 6 of the scale that floor gives; below 2^-125 the scale is 2^-127)
    int scale = max((int)(top >> 23) - 2 + (a.ceil && (top & 0x7fffffu) > 0x400000u ? 1 : 0), 0);
    uint32_t q = codes_of<T>(v, __builtin_bit_cast(float, scale ? (uint32_t)scale << 23 : 0x00400000u));
    if (top >= 0x7f800000u) {   // an infinity or NaN: the block is NaN
      scale = 255;
      q = 0;
    }
    uint8_t* const to = codes + c[u].row * a.code_stride + c[u].at / 2;
    if (WHOLE ? c[u].n > 0 : c[u].n >= 8) {
      __builtin_memcpy(to, &q, 4);
    } else if (!WHOLE) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (2 * i < c[u].n) to[i] = (uint8_t)(q >> (8 * i));
    }
    if (c[u].n > 0 && c[u].at % kMxBlock == 0) scales[c[u].row * a.scale_stride + c[u].at / kMxBlock] = (uint8_t)scale;
  }
}

template <typename T>
__global__ __launch_bounds__(kRowThreads) void k_mx_dequantise(RowArgs a, const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, T* __restrict__ x) {
  const Chunks chunks(a);
  uint32_t q[kChunksEach];
  int s[kChunksEach];
#pragma unroll
  for (int u = 0; u < kChunksEach; ++u) {
    const Chunk c = chunks(a, u);
    const uint8_t* const from = codes + c.row * a.code_stride + c.at / 2;
    q[u] = 0;
    s[u] = 0;
    if (c.n >= 8) {
      __builtin_memcpy(&q[u], from, 4);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (2 * i < c.n) q[u] |= (uint32_t)from[i] << (8 * i);
    }
    if (c.n > 0) s[u] = scales[c.row * a.scale_stride + c.at / kMxBlock];
  }
#pragma unroll
  for (int u = 0; u < kChunksEach; ++u) {
    const Chunk c = chunks(a, u);
    if (c.n <= 0) continue;
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.0f, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.0f, 3)};
    const float by = __builtin_bit_cast(float, s[u] == 255 ? 0x7fc00000u : s[u] ? (uint32_t)s[u] << 23 : 0x00400000u);
    f32x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = p[e / 2][e % 2] * by;   // exact in f32
    store_oct<T>(x + c.row * a.x_stride + c.at, v, c.n);
  }
}

int check_rows(const moe_mx_rows* p, int64_t rows) {
  if (!p) return fail(MOE_EINVAL, "mx rows: the description is NULL%s%lld");
  if (p->type != MOE_TYPE_BF16 && p->type != MOE_TYPE_FP16 && p->type != MOE_TYPE_F32)
    return fail(MOE_EINVAL, "mx rows: type must be MOE_TYPE_BF16, MOE_TYPE_FP16 or MOE_TYPE_F32%s (%lld)", "", p->type);
  if (p->scale != MOE_MX_FLOOR && p->scale != MOE_MX_CEIL)
    return fail(MOE_EINVAL, "mx rows: scale must be MOE_MX_FLOOR or MOE_MX_CEIL%s (%lld)", "", p->scale);
  if (p->k < 1) return fail(MOE_EINVAL, "mx rows: k must be >= 1%s (%lld)", "", p->k);
  if (p->k > MOE_MX_MAX_K) return fail(MOE_EUNSUPPORTED, "mx rows: k above MOE_MX_MAX_K%s (%lld)", "", p->k);
  if (p->x_stride < p->k || p->code_stride < (p->k + 1) / 2 || p->scale_stride < (p->k + kMxBlock - 1) / kMxBlock)
    return fail(MOE_EINVAL, "mx rows: a row stride is below its row%s%lld");
  if (rows < 0) return fail(MOE_EINVAL, "mx rows: rows must be >= 0%s (%lld)", "", rows);
  if (rows > MOE_MX_MAX_ROWS) return fail(MOE_EUNSUPPORTED, "mx rows: rows above MOE_MX_MAX_ROWS%s (%lld)", "", rows);
  return MOE_OK;
}

// `launch` is given the arguments and the number of workgroups.
template <typename Launch>
int row_call(const moe_mx_rows* p, const void* x, const void* codes, const void* scales, int64_t rows, Launch&& launch) {
  if (int r = check_rows(p, rows)) return r;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales) return fail(MOE_EINVAL, "mx rows: x, codes and scales must be non-NULL%s%lld");
  if ((uintptr_t)x % elem_bytes(p->type)) return fail(MOE_EINVAL, "mx rows: a pointer is not aligned to its elements%s%lld");
  const int chunks = 4 * ((p->k + kMxBlock - 1) / kMxBlock);
  const int64_t per = kRowThreads * kChunksEach, blocks = (rows * chunks + per - 1) / per;
  if (blocks >= (int64_t)1 << 24) return fail(MOE_EUNSUPPORTED, "mx rows: too many elements for one launch%s%lld");
  const RowArgs a = {rows, p->x_stride, p->code_stride, p->scale_stride, p->k, chunks,
                     (uint32_t)((((uint64_t)1 << 32) + chunks - 1) / chunks), p->scale == MOE_MX_CEIL};
  launch(a, (unsigned)blocks);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MOE_OK : hip_fail(e, "mx rows");
}

// ---- products ----------------------------------------------------------------------
struct MxArgs : Groups {
  int n, k;
  int out_type;
  Gate gate;
  int64_t x_stride, x_scale, y_stride, w_stride, w_group, w_scale, w_scale_group;
};

template <typename G, bool GATED>
__global__ __launch_bounds__(G::NT, 2) void k_mx(MxArgs a, const uint8_t* __restrict__ x, const uint8_t* __restrict__ xs,
                                              const uint8_t* __restrict__ w, const uint8_t* __restrict__ ws,
                                              const uint8_t* __restrict__ w2, const uint8_t* __restrict__ ws2,
                                              void* __restrict__ out) {
  extern __shared__ __align__(16) uint8_t lds[];
  report(a);
  const Tile t = my_tile<G>(a, a.n);
  if (t.rows <= 0) return;
  const bool none = t.group < 0 || t.group >= a.groups;
  const int p0 = t.p * G::kP, pn = a.n - p0;
  const int64_t at = (none ? 0 : t.group) * a.w_group + p0 * a.w_stride;
  const int64_t at_scale = (none ? 0 : t.group) * a.w_scale_group + p0 * a.w_scale;
  const MxOperand P = {w + at, ws + at_scale, a.w_stride, a.w_scale, min(G::kP, pn), GATED ? elements_between(w, w2) : 0,
                       GATED ? elements_between(ws, ws2) : 0};
  const MxOperand Q = {x + t.row * a.x_stride, xs + t.row * a.x_scale, a.x_stride, a.x_scale, t.rows};
  typename G::Acc acc = {};
  G::run(P, Q, none ? 0 : a.k, lds, acc);
  auto row = [&](int q) { return q < t.rows ? q : -1; };
  auto store = [&](const auto& sums) {
    const int64_t to = t.row * a.y_stride + p0;
    if (a.out_type == MOE_TYPE_F32) G::store_to(sums, (float*)out + to, a.y_stride, pn, row);
    else if (a.out_type == MOE_TYPE_BF16) G::store_to(sums, (bf16_t*)out + to, a.y_stride, pn, row);
    else G::store_to(sums, (fp16_t*)out + to, a.y_stride, pn, row);
  };
  if constexpr (GATED) {
    f32x4 g[G::NP / 2][G::NQ], u[G::NP / 2][G::NQ];
    G::part(acc, g, u);
#pragma unroll
    for (int i = 0; i < G::NP / 2; ++i)
#pragma unroll
      for (int j = 0; j < G::NQ; ++j) g[i][j] = gated_all(a.gate, g[i][j], u[i][j]);
    store(g);
  } else {
    store(acc);
  }
}

// The same in wide tiles.
template <typename G, bool GATED, int ACT>
__global__ __launch_bounds__(256, 1) void k_mx_wide(MxArgs a, const uint8_t* __restrict__ x, const uint8_t* __restrict__ xs,
                                                   const uint8_t* __restrict__ w, const uint8_t* __restrict__ ws,
                                                   const uint8_t* __restrict__ w2, const uint8_t* __restrict__ ws2,
                                                   void* __restrict__ out) {
  extern __shared__ __align__(16) uint8_t lds[];
  report(a);
  const Tile t = my_tile<G>(a, a.n);
  if (t.rows <= 0) return;
  const bool none = t.group < 0 || t.group >= a.groups;
  const int p0 = t.p * G::kP, pn = a.n - p0;
  const int64_t at = (none ? 0 : t.group) * a.w_group + p0 * a.w_stride;
  const int64_t at_scale = (none ? 0 : t.group) * a.w_scale_group + p0 * a.w_scale;
  const MxOperand P = {w + at, ws + at_scale, a.w_stride, a.w_scale, min(G::kP, pn), GATED ? elements_between(w, w2) : 0,
                       GATED ? elements_between(ws, ws2) : 0};
  const MxOperand Q = {x + t.row * a.x_stride, xs + t.row * a.x_scale, a.x_stride, a.x_scale, t.rows};
  by_rows(t.rows, [&](auto parts) {
    constexpr int NQ = parts, N = GATED ? 4 : 8;
    f32x4 acc[8][NQ] = {};
    if (!none) G::run(P, Q, a.k, lds, acc);
    f32x4 sums[N][NQ];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < NQ; ++j) {
        if constexpr (GATED) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sums[i][j][e] = gated<ACT>(acc[2 * i][j][e], acc[2 * i + 1][j][e], a.gate.limit);
        } else {
          sums[i][j] = acc[i][j];
        }
      }
    const int64_t to = t.row * a.y_stride + p0;
    if (a.out_type == MOE_TYPE_F32) G::store(sums, (float*)out + to, a.y_stride, pn, t.rows);
    else if (a.out_type == MOE_TYPE_BF16) G::store(sums, (bf16_t*)out + to, a.y_stride, pn, t.rows);
    else G::store(sums, (fp16_t*)out + to, a.y_stride, pn, t.rows);
  });
}

struct MxTensors {
  const void *x, *xs, *w, *ws, *w2, *ws2;
  void* out;
};

template <bool GATED, bool DMA, int BP, int BQ, int WP, int WQ, int ST, int STEPS, bool ONCE = false>
int launch_tile(const MxArgs& a, const MxTensors& v, hipStream_t s) {
  typedef MxGemm<BP, BQ, WP, WQ, ST, STEPS, DMA, GATED, ONCE> G;
  auto u8 = [](const void* p) { return (const uint8_t*)p; };
  return launch_rows_of_tiles<k_mx<G, GATED>, G>("mx", row_tiles(a, G::kQ) * ((a.n + G::kP - 1) / G::kP), s, a, u8(v.x), u8(v.xs),
                                                 u8(v.w), u8(v.ws), u8(v.w2), u8(v.ws2), v.out);
}

template <bool GATED>
int launch_wide(const MxArgs& a, const MxTensors& v, hipStream_t s) {
  typedef WideMx<GATED> G;
  const int64_t tiles = row_tiles(a, G::kQ) * ((a.n + G::kP - 1) / G::kP);
  auto with = [&](auto act) {
    constexpr int ACT = act;
    auto u8 = [](const void* p) { return (const uint8_t*)p; };
    return launch_rows_of_tiles<k_mx_wide<G, GATED, ACT>, G>("mx", tiles, s, a, u8(v.x), u8(v.xs), u8(v.w), u8(v.ws), u8(v.w2),
                                                             u8(v.ws2), v.out);
  };
  return GATED && a.gate.act == MOE_ACT_GELU ? with(std::integral_constant<int, GATED ? MOE_ACT_GELU : MOE_ACT_SILU>())
                                             : with(std::integral_constant<int, MOE_ACT_SILU>());
}

// Which tiles, by the same reckoning as the 16-bit products' (moe_gated.h). The times are at n = 2048, k = 4096, in us.
// The counts of tiles are points among the sizes that were timed; where the times cross differs by width.
// Few tiles: plain in 64 x 16, 32 of 8 8.6 against 12.2 in 128 x 64, 1 of 1 7.1 (11.4); gated in 64 x 32, 1 of 1 8.1 (11.9).
// Plain up to 192 tiles of 128 x 64: 256 of 1 (96) 9.1 (11.8), 1024 of 1, 1001 and 1003 wide (144), 11.4 (11.7), 600 of 32, 515 and
// 1001 wide (210), 8.7 (11.0); but 512 of 1 (160) 15.8 (11.9), 640 of 1 (192) 18.5 (12.6). Gated up to 1024 of its own: 400 of 8,
// n = 1024, k = 2048 (704), 8.5 (8.9), 384 of 1 (896) 13.0 (12.8), 512 of 1 (1152) 17.7 (13.2).
// More of them, but few rows a group: 128 x 32, whose codes of the weights are read once, gated 48 of 384 70.3 (74.0; 78.0 with
// loads that stay in the caches), 2000 of 384 518 (581; 562), 4000 of 384 550 (608; 585), plain 280 (314; 305); but plain
// 500 of 32, of fewer tiles, 31 (26), and 12288 of 384 gated 777 (711; 741). Plain from 512 tiles on for under 6 rows a group: 64 of
// 32 (544) 23.1 in them, 26.5 in 64 x 16, 32 of 32 (512) 19.2 (16.6); from 1024 for more rows, where 128 x 64 comes near: 400 of 60
// (1152) 44.0 (50.5), 1000 of 64 (1520) 54.3 (55.1), 384 of 32 (704) 23.9 (25.8).
// Wide tiles: 12288 rows of 64 groups plain 112 (130), gated 190 (238), 12288 of 384 gated 682 (711 in 128 x 64); but 4000 of 384
// 640 (607), 8192 of 16 plain 67 (63). They take sums of whole groups of 1024: 16384 of 32, n = 4096, k = 2048 118 (142), but
// k = 2560 167 in 128 x 128, k = 1536 122. 128 x 64 or 128 x 128: under 256 tiles of 128 x 128, plain 1024 of 1 (160) 13.0 (17.1),
// 1536 of 1 (224) 18.7 (17.4), 2048 of 1 (288) 19.7 (18.1), gated 512 of 1 (192) 13.2 (17.2), 768 of 1 (256) 18.4 (17.5). With few of them from a sum of 2048 on, 8000 of 8, n = 4096, 64 (67); at k = 1024
// 16384 of 16, n = 1024, 30.4 (26.6), but 16384 of 32, n = 4096, 86 (104).
template <bool GATED, bool DMA>
int launch_mx(const MxArgs& a, const MxTensors& v, hipStream_t s) {
  const int64_t mean = a.rows / a.groups;
  const int wide = GATED ? 2 * a.n : a.n;   // columns of P
  auto columns = [&](int p) { return (wide + p - 1) / p; };
  if constexpr (GATED) {
    if (row_tiles(a, 32) * columns(64) <= 1024) return launch_tile<GATED, DMA, 64, 32, 2, 2, 3, 4>(a, v, s);
    if (mean < 24) return launch_tile<GATED, DMA, 128, 32, 4, 1, 3, 4, true>(a, v, s);
  } else {
    if (mean < 24 && row_tiles(a, 32) * columns(128) > (mean < 6 ? 512 : 1024))
      return launch_tile<GATED, DMA, 128, 32, 4, 1, 3, 4, true>(a, v, s);
    if (mean < 6 || row_tiles(a, 64) * columns(128) <= 192) return launch_tile<GATED, DMA, 64, 16, 4, 1, 4, 2>(a, v, s);
  }
  if constexpr (DMA) {
    const int64_t tiles = likely_row_tiles(a, 256) * columns(256), small = likely_row_tiles(a, 128) * columns(128);
    const bool pays = tiles >= 768 ? mean >= 24 : mean >= 64 && 3 * rounds(a, tiles, 256) < 2 * rounds(a, small, 512);
    if (pays && (tiles >= 768 || a.k >= 2048) && a.k % WideMx<GATED>::kGroup == 0) return launch_wide<GATED>(a, v, s);
  }
  if (mean < 64 || row_tiles(a, 128) * columns(128) < 256) return launch_tile<GATED, DMA, 128, 64, 2, 2, 3, 2>(a, v, s);
  return launch_tile<GATED, DMA, 128, 128, 2, 2, 2, 4>(a, v, s);
}

int check_mx(const moe_mx* m, int64_t rows, bool with_act) {
  if (!m) return fail(MOE_EINVAL, "mx is NULL%s%lld");
  if (m->out_type != MOE_TYPE_BF16 && m->out_type != MOE_TYPE_FP16 && m->out_type != MOE_TYPE_F32)
    return fail(MOE_EINVAL, "mx: out_type must be MOE_TYPE_BF16, MOE_TYPE_FP16 or MOE_TYPE_F32%s (%lld)", "", m->out_type);
  if (with_act) {
    if (m->act != MOE_ACT_SILU && m->act != MOE_ACT_GELU)
      return fail(MOE_EINVAL, "mx: act must be MOE_ACT_SILU or MOE_ACT_GELU%s (%lld)", "", m->act);
    if (!(m->limit >= 0) || std::isinf(m->limit)) return fail(MOE_EINVAL, "mx: limit must be finite and >= 0%s%lld");
  }
  if (m->n_groups < 1) return fail(MOE_EINVAL, "mx: n_groups must be >= 1%s (%lld)", "", m->n_groups);
  if (m->n_groups > MOE_GROUPED_MAX_GROUPS)
    return fail(MOE_EUNSUPPORTED, "mx: n_groups above MOE_GROUPED_MAX_GROUPS%s (%lld)", "", m->n_groups);
  if (m->n < 1 || m->k < 1) return fail(MOE_EINVAL, "mx: n and k must be >= 1%s%lld");
  if (m->k > MOE_MX_MAX_K) return fail(MOE_EUNSUPPORTED, "mx: k above MOE_MX_MAX_K%s (%lld)", "", m->k);
  const int64_t bytes = (m->k + 1) / 2, blocks = (m->k + kMxBlock - 1) / kMxBlock;
  if (m->x_stride < bytes || m->w_stride < bytes || m->x_scale_stride < blocks || m->w_scale_stride < blocks || m->y_stride < m->n)
    return fail(MOE_EINVAL, "mx: a row stride is below its row%s%lld");
  if (m->w_group_stride < (int64_t)(m->n - 1) * m->w_stride + bytes ||
      m->w_scale_group_stride < (int64_t)(m->n - 1) * m->w_scale_stride + blocks)
    return fail(MOE_EINVAL, "mx: a group stride is below one weight%s%lld");
  const int64_t most = MOE_GROUPED_MAX_STRIDE;
  if (m->x_stride > most || m->w_stride > most || m->x_scale_stride > most || m->w_scale_stride > most || m->y_stride > most)
    return fail(MOE_EUNSUPPORTED, "mx: a row stride above MOE_GROUPED_MAX_STRIDE%s%lld");
  if (rows < 0) return fail(MOE_EINVAL, "mx: rows must be >= 0%s (%lld)", "", rows);
  if (rows > MOE_GROUPED_MAX_ROWS) return fail(MOE_EUNSUPPORTED, "mx: rows above MOE_GROUPED_MAX_ROWS%s (%lld)", "", rows);
  return MOE_OK;
}

template <bool GATED>
int mx_call(const moe_mx* m, const MxTensors& v, const int32_t* offsets, int64_t rows, int32_t* status, void* stream) {
  if (int r = check_mx(m, rows, GATED)) return r;
  if (!offsets) return fail(MOE_EINVAL, "mx: offsets must be non-NULL%s%lld");
  if ((uintptr_t)offsets % 4 || (uintptr_t)status % 4)
    return fail(MOE_EINVAL, "mx: a pointer is not aligned to its elements%s%lld");
  const MxArgs a = {{offsets, status, m->n_groups, (int)rows},
                    m->n,
                    m->k,
                    m->out_type,
                    {m->act, m->limit > 0 ? m->limit : INFINITY},
                    m->x_stride,
                    m->x_scale_stride,
                    m->y_stride,
                    m->w_stride,
                    m->w_group_stride,
                    m->w_scale_stride,
                    m->w_scale_group_stride};
  const hipStream_t s = (hipStream_t)stream;
  if (rows == 0) return status ? launch_offsets("mx", a, s) : MOE_OK;   // nothing to write, but the offsets are looked at
  if (!v.x || !v.xs || !v.w || !v.ws || !v.out || (GATED && (!v.w2 || !v.ws2)))
    return fail(MOE_EINVAL, "mx: operands, scales and output must be non-NULL%s%lld");
  if ((uintptr_t)v.out % elem_bytes(m->out_type))
    return fail(MOE_EINVAL, "mx: a pointer is not aligned to its elements%s%lld");
  const uintptr_t codes = (uintptr_t)v.x | (uintptr_t)v.w | (uintptr_t)v.w2 | a.x_stride | a.w_stride | a.w_group;
  const uintptr_t scales = (uintptr_t)v.xs | (uintptr_t)v.ws | (uintptr_t)v.ws2 | a.x_scale | a.w_scale | a.w_scale_group;
  return codes % 16 == 0 && scales % 4 == 0 ? launch_mx<GATED, true>(a, v, s) : launch_mx<GATED, false>(a, v, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_mx_quantise(const moe_mx_rows* p, const void* x, int64_t rows, void* codes, void* scales, void* stream) {
  return row_call(p, x, codes, scales, rows, [&](const RowArgs& a, unsigned blocks) {
    const hipStream_t s = (hipStream_t)stream;
    uint8_t *c = (uint8_t*)codes, *e = (uint8_t*)scales;
    auto with = [&](auto whole, const auto* from) {
      typedef std::remove_const_t<std::remove_pointer_t<decltype(from)>> T;
      k_mx_quantise<T, whole><<<blocks, kRowThreads, 0, s>>>(a, from, c, e);
    };
    auto of = [&](const auto* from) { p->k % 8 ? with(std::false_type(), from) : with(std::true_type(), from); };
    if (p->type == MOE_TYPE_BF16) of((const bf16_t*)x);
    else if (p->type == MOE_TYPE_FP16) of((const fp16_t*)x);
    else of((const float*)x);
  });
}

int moe_mx_dequantise(const moe_mx_rows* p, const void* codes, const void* scales, int64_t rows, void* x, void* stream) {
  return row_call(p, x, codes, scales, rows, [&](const RowArgs& a, unsigned blocks) {
    const hipStream_t s = (hipStream_t)stream;
    const uint8_t *c = (const uint8_t*)codes, *e = (const uint8_t*)scales;
    if (p->type == MOE_TYPE_BF16) k_mx_dequantise<<<blocks, kRowThreads, 0, s>>>(a, c, e, (bf16_t*)x);
    else if (p->type == MOE_TYPE_FP16) k_mx_dequantise<<<blocks, kRowThreads, 0, s>>>(a, c, e, (fp16_t*)x);
    else k_mx_dequantise<<<blocks, kRowThreads, 0, s>>>(a, c, e, (float*)x);
  });
}

int moe_mx_forward(const moe_mx* m, const void* x, const void* x_scale, const void* w, const void* w_scale,
                   const int32_t* offsets, int64_t rows, void* y, int32_t* status, void* stream) {
  return mx_call<false>(m, {x, x_scale, w, w_scale, nullptr, nullptr, y}, offsets, rows, status, stream);
}

int moe_mx_gated(const moe_mx* m, const void* x, const void* x_scale, const void* w_gate, const void* w_gate_scale,
                 const void* w_up, const void* w_up_scale, const int32_t* offsets, int64_t rows, void* h, int32_t* status,
                 void* stream) {
  return mx_call<true>(m, {x, x_scale, w_gate, w_gate_scale, w_up, w_up_scale, h}, offsets, rows, status, stream);
}

}  // extern "C"
