// The experts' gated feed-forward on 16-bit weights (moe_gated_*), rows sorted
// by group as for the grouped products:
//
//   forward     h[r] = act(Wg[e] x[r]) * (Wu[e] x[r])      P = 16 rows of Wg and 16 of Wu in turn, Q = x rows, sum over k
//   backward_h  dh[r] = Wd[e]^T dy[r], never stored:       P = Wd columns, Q = dy rows, sum over k
//               dgate, dup (and h again) from dh, gate, up
//   backward_x  dx[r] = Wg[e]^T dgate[r] + Wu[e]^T dup[r]  P = Wg, then Wu columns, Q = dgate, then dup rows, two sums over n
//
// A lane of the forward tile holds the sums of the same outputs of both
// projections, so that activation and product are its own work; the backward
// pass applies their derivatives to dh while it is still in registers.
#include <hip/hip_runtime.h>

#include <cmath>

#include "moe_activation.h"
#include "moe_gemm.h"
#include "moe_groups.h"
#include "moe_host.h"

namespace moe {
namespace {

struct GatedArgs : Groups {
  int n, k;
  int f32;   // dx in f32
  Gate gate;
  int64_t x_stride, h_stride, gate_stride, y_stride, w_stride, w_group, down_stride, down_group;
};

template <typename T, typename G>
__global__ __launch_bounds__(G::NT, 2) void k_gated(GatedArgs a, const T* __restrict__ x, const T* __restrict__ wg,
                                                 const T* __restrict__ wu, T* __restrict__ h, T* __restrict__ gate,
                                                 T* __restrict__ up) {
  extern __shared__ __align__(16) uint8_t lds[];
  report(a);
  const Tile t = my_tile<G>(a, a.n);
  if (t.rows <= 0) return;
  const bool none = t.group < 0 || t.group >= a.groups;
  const int p0 = t.p * G::kP, pn = a.n - p0;
  const Operand<T> P = {(G::second_rows() ? wu : wg) + (none ? 0 : t.group) * a.w_group + p0 * a.w_stride, a.w_stride,
                        min(G::kP, pn), nullptr, a.k >= 8};
  const Operand<T> Q = {x + t.row * a.x_stride, a.x_stride, t.rows, nullptr, a.k >= 8};
  typename G::Acc acc = {};
  G::run(P, Q, none ? 0 : a.k, lds, acc);
  f32x4 g[G::NP / 2][G::NQ], u[G::NP / 2][G::NQ];
  G::part(acc, g, u);
  auto row = [&](int q) { return q < t.rows ? q : -1; };
  if (gate) {
    G::store_to(g, gate + t.row * a.gate_stride + p0, a.gate_stride, pn, row);
    G::store_to(u, up + t.row * a.gate_stride + p0, a.gate_stride, pn, row);
  }
#pragma unroll
  for (int i = 0; i < G::NP / 2; ++i)
#pragma unroll
    for (int j = 0; j < G::NQ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) g[i][j][e] = gated(a.gate, g[i][j][e], u[i][j][e]);
  G::store_to(g, h + t.row * a.h_stride + p0, a.h_stride, pn, row);
}

// (gate and dgate, and up and dup, may be the same memory.)
template <typename T, typename G>
__global__ __launch_bounds__(G::NT, 2) void k_gated_dh(GatedArgs a, const T* __restrict__ dy, const T* __restrict__ wd,
                                                    const T* gate, const T* up, T* dgate, T* dup, T* __restrict__ h) {
  extern __shared__ __align__(16) uint8_t lds[];
  report(a);
  const Tile t = my_tile<G>(a, a.n);
  if (t.rows <= 0) return;
  const bool none = t.group < 0 || t.group >= a.groups;
  const int p0 = t.p * G::kP, pn = a.n - p0;
  const Operand<T> P = {wd + (none ? 0 : t.group) * a.down_group + p0, a.down_stride, pn, nullptr, a.n >= 8};
  const Operand<T> Q = {dy + t.row * a.y_stride, a.y_stride, t.rows, nullptr, a.k >= 8};
  typename G::Acc acc = {};
  G::run(P, Q, none ? 0 : a.k, lds, acc);
  const int64_t first = t.row * a.gate_stride + p0;
  struct Kept {
    f32x4 g, u;
  };
  G::each_quad(
      acc, pn, [&](int q) { return q < t.rows ? q : -1; },
      [&](int64_t q, int p, int n) -> Kept {
        const int64_t at = first + q * a.gate_stride + p;
        return {G::load_quad(gate + at, n), G::load_quad(up + at, n)};
      },
      [&](int64_t q, int p, int n, f32x4 dh, const Kept& kept) {
        f32x4 dg, du, v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x, y;
          v[e] = gated_back(a.gate, kept.g[e], kept.u[e], dh[e], x, y);
          // rows of no group have no gradients, whatever is kept there
          dg[e] = none ? 0.0f : x;
          du[e] = none ? 0.0f : y;
          v[e] = none ? 0.0f : v[e];
        }
        const int64_t at = first + q * a.gate_stride + p;
        G::store_quad(dgate + at, dg, n);
        G::store_quad(dup + at, du, n);
        if (h) G::store_quad(h + (t.row + q) * a.h_stride + p0 + p, v, n);
      });
}

template <typename T, typename G>
__global__ __launch_bounds__(G::NT, 2) void k_gated_dx(GatedArgs a, const T* __restrict__ dgate, const T* __restrict__ dup,
                                                    const T* __restrict__ wg, const T* __restrict__ wu,
                                                    void* __restrict__ dx) {
  extern __shared__ __align__(16) uint8_t lds[];
  report(a);
  const Tile t = my_tile<G>(a, a.k);
  if (t.rows <= 0) return;
  const bool none = t.group < 0 || t.group >= a.groups;
  const int p0 = t.p * G::kP, pn = a.k - p0;
  const Operand<T> P = {wg + (none ? 0 : t.group) * a.w_group + p0, a.w_stride, pn, nullptr, a.k >= 8,
                        elements_between(wg, wu)};
  const Operand<T> Q = {dgate + t.row * a.gate_stride, a.gate_stride, t.rows, nullptr, a.n >= 8,
                        elements_between(dgate, dup)};
  typename G::Acc acc = {};
  G::run(P, Q, none ? 0 : a.n, lds, acc);
  uint8_t* o = (uint8_t*)dx + (t.row * a.x_stride + p0) * (a.f32 ? 4 : 2);
  G::store(acc, o, a.f32, a.x_stride, pn, [&](int q) { return q < t.rows ? q : -1; });
}

enum Way { kForward, kHidden, kInput };

// What a call was given, in the order of its entry point.
struct Tensors {
  const void *in, *in2;   // x; dy; dgate and dup
  const void *w, *w2;     // w_gate and w_up; w_down
  const void *gate, *up;  // kept by the forward pass
  void *out, *out2, *h;   // h (gate and up kept as out and out2); dgate and dup, h; dx
};

template <Way W, typename T, bool DMA, int BP, int BQ, int WP, int WQ, int ST>
int launch_tile(const GatedArgs& a, const Tensors& v, hipStream_t s) {
  typedef Gemm<T, W != kForward, false, BP, BQ, WP, WQ, ST, DMA, false,
               W == kForward ? kRowPairs : W == kInput ? kTwoSums : kSingle> G;
  const int width = W == kInput ? a.k : a.n;
  const int64_t tiles = row_tiles(a, G::kQ) * ((width + G::kP - 1) / G::kP);
  if constexpr (W == kForward)
    return launch_rows_of_tiles<k_gated<T, G>, G>("gated", tiles, s, a, (const T*)v.in, (const T*)v.w, (const T*)v.w2,
                                                  (T*)v.h, (T*)v.out, (T*)v.out2);
  else if constexpr (W == kHidden)
    return launch_rows_of_tiles<k_gated_dh<T, G>, G>("gated", tiles, s, a, (const T*)v.in, (const T*)v.w,
                                                     (const T*)v.gate, (const T*)v.up, (T*)v.out, (T*)v.out2, (T*)v.h);
  else
    return launch_rows_of_tiles<k_gated_dx<T, G>, G>("gated", tiles, s, a, (const T*)v.in, (const T*)v.in2,
                                                     (const T*)v.w, (const T*)v.w2, v.out);
}

template <Way W, typename T, bool DMA>
int launch_rows(const GatedArgs& a, const Tensors& v, hipStream_t s) {
  const int64_t mean = a.rows / a.groups;
  const int width = W == kInput ? a.k : a.n, wide = W == kForward ? 2 * width : width;   // columns of P
  if (mean < 16 || row_tiles(a, 64) * ((wide + 127) / 128) < 96) return launch_tile<W, T, DMA, 128, 16, 4, 1, 4>(a, v, s);
  if (mean < 64 || row_tiles(a, 128) * ((wide + 127) / 128) < 300)
    return launch_tile<W, T, DMA, 128, 64, 2, 2, 3>(a, v, s);
  if constexpr (DMA) {
    if (row_tiles(a, 128) * ((wide + 255) / 256) >= 768 && (W == kInput ? a.n : a.k) >= 1024)
      return launch_tile<W, T, DMA, 256, 128, 4, 2, 3>(a, v, s);
  }
  return launch_tile<W, T, DMA, 128, 128, 2, 2, 2>(a, v, s);
}

template <Way W, typename T>
int launch_way(const GatedArgs& a, const Tensors& v, hipStream_t s) {
  bool aligned;
  if (W == kForward)
    aligned = rows16(v.in, a.x_stride) && rows16(v.w, a.w_stride) && rows16(v.w2, a.w_stride) && a.w_group % 8 == 0;
  else if (W == kHidden)
    aligned = rows16(v.in, a.y_stride) && rows16(v.w, a.down_stride) && a.down_group % 8 == 0 && a.n % 8 == 0;
  else
    aligned = rows16(v.in, a.gate_stride) && rows16(v.in2, a.gate_stride) && rows16(v.w, a.w_stride) &&
              rows16(v.w2, a.w_stride) && a.w_group % 8 == 0 && a.k % 8 == 0;
  return aligned ? launch_rows<W, T, true>(a, v, s) : launch_rows<W, T, false>(a, v, s);
}

int check_gated(const moe_gated* g, int64_t rows, Way way) {
  if (!g) return fail(MOE_EINVAL, "gated is NULL%s%lld");
  if (g->type != MOE_TYPE_BF16 && g->type != MOE_TYPE_FP16)
    return fail(MOE_EINVAL, "gated: type must be MOE_TYPE_BF16 or MOE_TYPE_FP16%s (%lld)", "", g->type);
  if (g->dx_type != g->type && g->dx_type != MOE_TYPE_F32)
    return fail(MOE_EINVAL, "gated: dx_type must be type or MOE_TYPE_F32%s (%lld)", "", g->dx_type);
  if (g->act != MOE_ACT_SILU && g->act != MOE_ACT_GELU)
    return fail(MOE_EINVAL, "gated: act must be MOE_ACT_SILU or MOE_ACT_GELU%s (%lld)", "", g->act);
  if (!(g->limit >= 0) || std::isinf(g->limit)) return fail(MOE_EINVAL, "gated: limit must be finite and >= 0%s%lld");
  if (g->n_groups < 1) return fail(MOE_EINVAL, "gated: n_groups must be >= 1%s (%lld)", "", g->n_groups);
  if (g->n_groups > MOE_GROUPED_MAX_GROUPS)
    return fail(MOE_EUNSUPPORTED, "gated: n_groups above MOE_GROUPED_MAX_GROUPS%s (%lld)", "", g->n_groups);
  if (g->n < 1 || g->k < 1) return fail(MOE_EINVAL, "gated: n and k must be >= 1%s%lld");
  // only the strides that this call uses
  const bool x = way != kHidden, h = way != kInput, gate = true, y = way == kHidden, w = way != kHidden;
  if ((x && g->x_stride < g->k) || (h && g->h_stride < g->n) || (gate && g->gate_stride < g->n) ||
      (y && g->y_stride < g->k) || (w && g->w_stride < g->k) || (!w && g->down_stride < g->n))
    return fail(MOE_EINVAL, "gated: a row stride is below its row%s%lld");
  if (w ? g->w_group_stride < (int64_t)(g->n - 1) * g->w_stride + g->k
        : g->down_group_stride < (int64_t)(g->k - 1) * g->down_stride + g->n)
    return fail(MOE_EINVAL, "gated: a group stride is below one weight%s%lld");
  const int64_t most = MOE_GROUPED_MAX_STRIDE;
  if ((x && g->x_stride > most) || (h && g->h_stride > most) || g->gate_stride > most || (y && g->y_stride > most) ||
      (w ? g->w_stride : g->down_stride) > most)
    return fail(MOE_EUNSUPPORTED, "gated: a row stride above MOE_GROUPED_MAX_STRIDE%s%lld");
  if (rows < 0) return fail(MOE_EINVAL, "gated: rows must be >= 0%s (%lld)", "", rows);
  if (rows > MOE_GROUPED_MAX_ROWS)
    return fail(MOE_EUNSUPPORTED, "gated: rows above MOE_GROUPED_MAX_ROWS%s (%lld)", "", rows);
  return MOE_OK;
}

template <Way W>
int gated_call(const moe_gated* g, const Tensors& v, const int32_t* offsets, int64_t rows, int32_t* status, void* stream) {
  if (int r = check_gated(g, rows, W)) return r;
  if (!offsets) return fail(MOE_EINVAL, "gated: offsets must be non-NULL%s%lld");
  if ((uintptr_t)offsets % 4 || (uintptr_t)status % 4)
    return fail(MOE_EINVAL, "gated: a pointer is not aligned to its elements%s%lld");
  const GatedArgs a = {{offsets, status, g->n_groups, (int)rows},
                       g->n,
                       g->k,
                       g->dx_type == MOE_TYPE_F32,
                       {g->act, g->limit > 0 ? g->limit : INFINITY},
                       g->x_stride,
                       g->h_stride,
                       g->gate_stride,
                       g->y_stride,
                       g->w_stride,
                       g->w_group_stride,
                       g->down_stride,
                       g->down_group_stride};
  const hipStream_t s = (hipStream_t)stream;
  if (rows == 0) return status ? launch_offsets("gated", a, s) : MOE_OK;   // nothing to write, but the offsets are looked at
  const bool there = W == kForward  ? v.in && v.w && v.w2 && v.h && !v.out == !v.out2
                     : W == kHidden ? v.in && v.w && v.gate && v.up && v.out && v.out2
                                    : v.in && v.in2 && v.w && v.w2 && v.out;
  if (!there)
    return fail(MOE_EINVAL, W == kForward ? "gated: operands and h must be non-NULL, gate and up both or neither%s%lld"
                                          : "gated: operands and outputs must be non-NULL%s%lld");
  const uintptr_t halves = (uintptr_t)v.in | (uintptr_t)v.in2 | (uintptr_t)v.w | (uintptr_t)v.w2 | (uintptr_t)v.gate |
                           (uintptr_t)v.up | (uintptr_t)v.out | (uintptr_t)v.out2 | (uintptr_t)v.h;
  if (halves % 2 || (W == kInput && a.f32 && (uintptr_t)v.out % 4))
    return fail(MOE_EINVAL, "gated: a pointer is not aligned to its elements%s%lld");
  return g->type == MOE_TYPE_BF16 ? launch_way<W, bf16_t>(a, v, s) : launch_way<W, fp16_t>(a, v, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_gated_forward(const moe_gated* g, const void* x, const void* w_gate, const void* w_up, const int32_t* offsets,
                      int64_t rows, void* h, void* gate, void* up, int32_t* status, void* stream) {
  return gated_call<kForward>(g, {x, nullptr, w_gate, w_up, nullptr, nullptr, gate, up, h}, offsets, rows, status, stream);
}

int moe_gated_backward_h(const moe_gated* g, const void* dy, const void* w_down, const void* gate, const void* up,
                         const int32_t* offsets, int64_t rows, void* dgate, void* dup, void* h, int32_t* status,
                         void* stream) {
  return gated_call<kHidden>(g, {dy, nullptr, w_down, nullptr, gate, up, dgate, dup, h}, offsets, rows, status, stream);
}

int moe_gated_backward_x(const moe_gated* g, const void* dgate, const void* dup, const void* w_gate, const void* w_up,
                         const int32_t* offsets, int64_t rows, void* dx, int32_t* status, void* stream) {
  return gated_call<kInput>(g, {dgate, dup, w_gate, w_up, nullptr, nullptr, dx, nullptr, nullptr}, offsets, rows, status,
                            stream);
}

}  // extern "C"
