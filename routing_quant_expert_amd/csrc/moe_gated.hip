// The gated feed-forward's forward pass, and the entry points of all three calls (moe_gated.h).
//
// Few rows are bound by the weights' reading (48 rows of 384 groups of 2048 x 4096: 265 us, 6.1 TB/s), many by the matrix
// instructions (16384 rows of 4 equal groups: 402 us, 1370 TFLOP/s; of 32 ragged ones, with gate and up kept, 530 us, 1040).
#include "moe_gated.h"
#include <cmath>

#include "moe_host.h"

namespace moe {
namespace {

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
    for (int j = 0; j < G::NQ; ++j) g[i][j] = gated_all(a.gate, g[i][j], u[i][j]);
  G::store_to(g, h + t.row * a.h_stride + p0, a.h_stride, pn, row);
}

template <typename T, typename G, int ACT>
__global__ __launch_bounds__(256, 1) void k_gated_wide(GatedArgs a, const T* __restrict__ x, const T* __restrict__ wg,
                                                      const T* __restrict__ wu, T* __restrict__ h, T* __restrict__ gate,
                                                      T* __restrict__ up) {
  extern __shared__ __align__(16) uint8_t lds[];
  report(a);
  const Tile t = my_tile<G>(a, a.n);
  if (t.rows <= 0) return;
  const bool none = t.group < 0 || t.group >= a.groups;
  const int p0 = t.p * G::kP, pn = a.n - p0;
  const Operand<T> P = {(G::second_rows() ? wu : wg) + (none ? 0 : t.group) * a.w_group + p0 * a.w_stride, a.w_stride,
                        min(G::kP, pn), nullptr, true};
  const Operand<T> Q = {x + t.row * a.x_stride, a.x_stride, t.rows, nullptr, true};
  by_rows(t.rows, [&](auto parts) {
    constexpr int NQ = parts;
    f32x4 acc[8][NQ] = {};
    if (!none) G::run(P, Q, a.k, lds, acc, [] {});
    f32x4 g[4][NQ], u[4][NQ];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < NQ; ++j) {
        g[i][j] = acc[2 * i][j];
        u[i][j] = acc[2 * i + 1][j];
      }
    if (gate) {
      G::store(g, gate + t.row * a.gate_stride + p0, a.gate_stride, pn, t.rows);
      G::store(u, up + t.row * a.gate_stride + p0, a.gate_stride, pn, t.rows);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) g[i][j][e] = gated<ACT>(g[i][j][e], u[i][j][e], a.gate.limit);
    G::store(g, h + t.row * a.h_stride + p0, a.h_stride, pn, t.rows);
  });
}

struct Kernels {
  template <typename T, typename G>
  static int narrow(int64_t tiles, const GatedArgs& a, const GatedTensors& v, hipStream_t s) {
    return launch_rows_of_tiles<k_gated<T, G>, G>("gated", tiles, s, a, (const T*)v.in, (const T*)v.w, (const T*)v.w2, (T*)v.h,
                                                  (T*)v.out, (T*)v.out2);
  }
  template <typename T, typename G>
  static int wide(int64_t tiles, const GatedArgs& a, const GatedTensors& v, hipStream_t s) {
    return a.gate.act == MOE_ACT_SILU ? wide_with<T, G, MOE_ACT_SILU>(tiles, a, v, s) : wide_with<T, G, MOE_ACT_GELU>(tiles, a, v, s);
  }
  template <typename T, typename G, int ACT>
  static int wide_with(int64_t tiles, const GatedArgs& a, const GatedTensors& v, hipStream_t s) {
    return launch_rows_of_tiles<k_gated_wide<T, G, ACT>, G>("gated", tiles, s, a, (const T*)v.in, (const T*)v.w, (const T*)v.w2,
                                                            (T*)v.h, (T*)v.out, (T*)v.out2);
  }
};


// kept: the call has gate and up (the forward pass may go without).
int check_gated(const moe_gated* g, int64_t rows, GatedWay way, bool kept) {
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
  const bool x = way != kHidden, h = way != kInput, y = way == kHidden, w = way != kHidden;
  if ((x && g->x_stride < g->k) || (h && g->h_stride < g->n) || (kept && g->gate_stride < g->n) ||
      (y && g->y_stride < g->k) || (w && g->w_stride < g->k) || (!w && g->down_stride < g->n))
    return fail(MOE_EINVAL, "gated: a row stride is below its row%s%lld");
  if (w ? g->w_group_stride < (int64_t)(g->n - 1) * g->w_stride + g->k
        : g->down_group_stride < (int64_t)(g->k - 1) * g->down_stride + g->n)
    return fail(MOE_EINVAL, "gated: a group stride is below one weight%s%lld");
  const int64_t most = MOE_GROUPED_MAX_STRIDE;
  if ((x && g->x_stride > most) || (h && g->h_stride > most) || (kept && g->gate_stride > most) || (y && g->y_stride > most) ||
      (w ? g->w_stride : g->down_stride) > most)
    return fail(MOE_EUNSUPPORTED, "gated: a row stride above MOE_GROUPED_MAX_STRIDE%s%lld");
  if (rows < 0) return fail(MOE_EINVAL, "gated: rows must be >= 0%s (%lld)", "", rows);
  if (rows > MOE_GROUPED_MAX_ROWS)
    return fail(MOE_EUNSUPPORTED, "gated: rows above MOE_GROUPED_MAX_ROWS%s (%lld)", "", rows);
  return MOE_OK;
}

template <GatedWay W>
int gated_call(const moe_gated* g, const GatedTensors& v, const int32_t* offsets, int64_t rows, int32_t* status, void* stream) {
  if (int r = check_gated(g, rows, W, W != kForward || v.out || v.out2)) return r;
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
  return W == kForward  ? gated_forward(a, v, g->type, s)
         : W == kHidden ? gated_hidden(a, v, g->type, s)
                        : gated_input(a, v, g->type, s);
}

}  // namespace

int gated_forward(const GatedArgs& a, const GatedTensors& v, int type, hipStream_t s) {
  return launch_gated<kForward, Kernels>(a, v, type, s);
}

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
