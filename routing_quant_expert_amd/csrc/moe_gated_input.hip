// The gated feed-forward's gradient of the input (moe_gated.h).
//
// One sum over both products: half the launches, and no rounding or second reading of a partial sum. 16384 rows of 32 groups
// of 2048 x 4096 in 520 us (1060 TFLOP/s; 1360 on 4 equal groups), bound by the matrix instructions.
#include "moe_gated.h"

namespace moe {
namespace {

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

template <typename T, typename G>
__global__ __launch_bounds__(256, 1) void k_gated_dx_wide(GatedArgs a, const T* __restrict__ dgate, const T* __restrict__ dup,
                                                         const T* __restrict__ wg, const T* __restrict__ wu,
                                                         void* __restrict__ dx) {
  extern __shared__ __align__(16) uint8_t lds[];
  report(a);
  const Tile t = my_tile<G>(a, a.k);
  if (t.rows <= 0) return;
  const bool none = t.group < 0 || t.group >= a.groups;
  const int p0 = t.p * G::kP, pn = a.k - p0;
  const Operand<T> P = {wg + (none ? 0 : t.group) * a.w_group + p0, a.w_stride, pn, nullptr, true, elements_between(wg, wu)};
  const Operand<T> Q = {dgate + t.row * a.gate_stride, a.gate_stride, t.rows, nullptr, true, elements_between(dgate, dup)};
  by_rows(t.rows, [&](auto parts) {
    constexpr int NQ = parts;
    f32x4 acc[8][NQ] = {};
    if (!none) G::run(P, Q, a.n, lds, acc, [] {});
    const int64_t to = t.row * a.x_stride + p0;
    if (a.f32) G::store(acc, (float*)dx + to, a.x_stride, pn, t.rows);
    else G::store(acc, (T*)dx + to, a.x_stride, pn, t.rows);
  });
}

struct Kernels {
  template <typename T, typename G>
  static int narrow(int64_t tiles, const GatedArgs& a, const GatedTensors& v, hipStream_t s) {
    return launch_rows_of_tiles<k_gated_dx<T, G>, G>("gated", tiles, s, a, (const T*)v.in, (const T*)v.in2, (const T*)v.w,
                                                     (const T*)v.w2, v.out);
  }
  template <typename T, typename G>
  static int wide(int64_t tiles, const GatedArgs& a, const GatedTensors& v, hipStream_t s) {
    return launch_rows_of_tiles<k_gated_dx_wide<T, G>, G>("gated", tiles, s, a, (const T*)v.in, (const T*)v.in2, (const T*)v.w,
                                                          (const T*)v.w2, v.out);
  }
};


}  // namespace

int gated_input(const GatedArgs& a, const GatedTensors& v, int type, hipStream_t s) {
  return launch_gated<kInput, Kernels>(a, v, type, s);
}

}  // namespace moe
