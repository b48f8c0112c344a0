// The gated feed-forward's gradients of gate and up (moe_gated.h).
//
// The sums are half of the forward pass's, and every output takes two loads and three stores beside them, at the same time
// in all workgroups: 16384 rows of 32 groups of 2048 x 4096 in 354 us, about 41 of each round of tiles without a product, and
// 632 tiles, 2.47 rounds of the 256 CUs that take 3.
#include "moe_gated.h"

namespace moe {
namespace {

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
  const int64_t first = t.row * a.gate_stride + p0;
  struct Kept {
    typename G::template Quad<T>::type g, u;
  };
  auto row = [&](int q) { return q < t.rows ? q : -1; };
  Kept kept[G::NP][G::NQ];
  typename G::Acc acc = {};
  G::run(P, Q, none ? 0 : a.k, lds, acc, [&] {
    G::load_quads(kept, pn, row, [&](int64_t q, int p, int n) -> Kept {
      const int64_t at = first + q * a.gate_stride + p;
      return {G::load_quad(gate + at, n), G::load_quad(up + at, n)};
    });
  });
  G::use_quads(acc, kept, pn, row, [&](int64_t q, int p, int n, f32x4 dh, const Kept& k) {
    f32x4 dg = {}, du = {}, v = {};
    if (!none) {   // rows of no group have no gradients, whatever is kept there
      const f32x4 g = __builtin_convertvector(k.g, f32x4), u = __builtin_convertvector(k.u, f32x4);
      if (a.gate.act == MOE_ACT_SILU) v = gated_back_all<MOE_ACT_SILU>(g, u, dh, a.gate.limit, dg, du);
      else v = gated_back_all<MOE_ACT_GELU>(g, u, dh, a.gate.limit, dg, du);
    }
    const int64_t at = first + q * a.gate_stride + p;
    G::store_quad(dgate + at, dg, n);
    G::store_quad(dup + at, du, n);
    if (h) G::store_quad(h + (t.row + q) * a.h_stride + p0 + p, v, n);
  });
}

// (All registers are taken: 2 values a lane in bf16 and 5 in fp16 go to scratch memory before the loop over the sum and come back
// where the outputs are made. No wait for a tile's loads stands between.)
template <typename T, typename G, int ACT>
__global__ __launch_bounds__(256, 1) void k_gated_dh_wide(GatedArgs a, const T* __restrict__ dy, const T* __restrict__ wd,
                                                         const T* gate, const T* up, T* dgate, T* dup, T* __restrict__ h) {
  extern __shared__ __align__(16) uint8_t lds[];
  report(a);
  const Tile t = my_tile<G>(a, a.n);
  if (t.rows <= 0) return;
  const bool none = t.group < 0 || t.group >= a.groups;
  const int p0 = t.p * G::kP, pn = a.n - p0;
  const Operand<T> P = {wd + (none ? 0 : t.group) * a.down_group + p0, a.down_stride, pn, nullptr, true};
  const Operand<T> Q = {dy + t.row * a.y_stride, a.y_stride, t.rows, nullptr, true};
  const int p = G::first_out();
  const int64_t first = t.row * a.gate_stride + p0 + p, first_h = t.row * a.h_stride + p0 + p;
  if (none) {   // rows of no group have no gradients, whatever is kept there
    for (int j = 0; j < 8; ++j)
      for (int i = 0; i < 4; ++i) {
        const int q = G::row_of(j);
        if (q >= t.rows || p + 32 * i >= pn) continue;
        store_oct(dgate + first + q * a.gate_stride + 32 * i, f32x8{}, 8);
        store_oct(dup + first + q * a.gate_stride + 32 * i, f32x8{}, 8);
        if (h) store_oct(h + first_h + q * a.h_stride + 32 * i, f32x8{}, 8);
      }
    return;
  }
  by_rows(t.rows, [&](auto parts) {
    constexpr int NQ = parts;
    struct Kept {
      oct<T> g[4], u[4];
    };
    // gate and up of the wave's j-th 16 rows; those of the next are asked for before this one's are used (and before its
    // stores, which a wait for a later load would be for too). Past the tile's rows and outputs its last ones.
    auto load = [&](int j, Kept& k) {
      const int64_t at = first + min(G::row_of(j), t.rows - 1) * a.gate_stride;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t from = at + min(32 * i, pn - 8 - p);   // (widths are multiples of 8)
        __builtin_memcpy(&k.g[i], gate + from, 16);
        __builtin_memcpy(&k.u[i], up + from, 16);
      }
    };
    Kept kept[2];
    f32x4 acc[8][NQ] = {};
    G::run(P, Q, a.k, lds, acc, [&] { load(0, kept[0]); });
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      __builtin_amdgcn_sched_barrier(0);   // (the rows one after another: all at once do not fit the registers)
      if (j + 1 < NQ) load(j + 1, kept[(j + 1) % 2]);
      f32x8 dh[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) dh[i] = G::neighbours(acc[2 * i][j], acc[2 * i + 1][j]);
      if (G::row_of(j) >= t.rows) continue;
      const int64_t at = first + G::row_of(j) * a.gate_stride, at_h = first_h + G::row_of(j) * a.h_stride;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (p + 32 * i >= pn) continue;
        f32x8 dg, du;
        const f32x8 v = gated_back_all<ACT>(unpacked(kept[j % 2].g[i]), unpacked(kept[j % 2].u[i]), dh[i], a.gate.limit, dg, du);
        store_oct(dgate + at + 32 * i, dg, 8);
        store_oct(dup + at + 32 * i, du, 8);
        if (h) store_oct(h + at_h + 32 * i, v, 8);
      }
    }
  });
}

struct Kernels {
  template <typename T, typename G>
  static int narrow(int64_t tiles, const GatedArgs& a, const GatedTensors& v, hipStream_t s) {
    return launch_rows_of_tiles<k_gated_dh<T, G>, G>("gated", tiles, s, a, (const T*)v.in, (const T*)v.w, (const T*)v.gate,
                                                     (const T*)v.up, (T*)v.out, (T*)v.out2, (T*)v.h);
  }
  template <typename T, typename G>
  static int wide(int64_t tiles, const GatedArgs& a, const GatedTensors& v, hipStream_t s) {
    return a.gate.act == MOE_ACT_SILU ? wide_with<T, G, MOE_ACT_SILU>(tiles, a, v, s) : wide_with<T, G, MOE_ACT_GELU>(tiles, a, v, s);
  }
  template <typename T, typename G, int ACT>
  static int wide_with(int64_t tiles, const GatedArgs& a, const GatedTensors& v, hipStream_t s) {
    return launch_rows_of_tiles<k_gated_dh_wide<T, G, ACT>, G>("gated", tiles, s, a, (const T*)v.in, (const T*)v.w,
                                                               (const T*)v.gate, (const T*)v.up, (T*)v.out, (T*)v.out2,
                                                               (T*)v.h);
  }
};


}  // namespace

int gated_hidden(const GatedArgs& a, const GatedTensors& v, int type, hipStream_t s) {
  return launch_gated<kHidden, Kernels>(a, v, type, s);
}

}  // namespace moe
