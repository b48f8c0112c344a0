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
//
// The three calls are compiled apart (moe_gated.hip, moe_gated_hidden.hip, moe_gated_input.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "moe_activation.h"
#include "moe_gemm.h"
#include "moe_groups.h"
#include "moe_wide.h"

namespace moe {

struct GatedArgs : Groups {
  int n, k;
  int f32;   // dx in f32
  Gate gate;
  int64_t x_stride, h_stride, gate_stride, y_stride, w_stride, w_group, down_stride, down_group;
};

enum GatedWay { kForward, kHidden, kInput };

// What a call was given, in the order of its entry point.
struct GatedTensors {
  const void *in, *in2;   // x; dy; dgate and dup
  const void *w, *w2;     // w_gate and w_up; w_down
  const void *gate, *up;  // kept by the forward pass
  void *out, *out2, *h;   // h (gate and up kept as out and out2); dgate and dup, h; dx
};

// One call's kernels (type: MOE_TYPE_BF16 or MOE_TYPE_FP16).
int gated_forward(const GatedArgs& a, const GatedTensors& v, int type, hipStream_t s);
int gated_hidden(const GatedArgs& a, const GatedTensors& v, int type, hipStream_t s);
int gated_input(const GatedArgs& a, const GatedTensors& v, int type, hipStream_t s);

// The tiles of a way. K: its kernels, narrow<T, G>(tiles, ...) in tiles of moe_gemm.h and wide<T, G>(tiles, ...) of moe_wide.h.
template <GatedWay W, typename K, typename T, bool DMA, int BP, int BQ, int WP, int WQ, int ST>
int launch_gated_tile(const GatedArgs& a, const GatedTensors& v, hipStream_t s) {
  typedef Gemm<T, W != kForward, false, BP, BQ, WP, WQ, ST, DMA, false,
               W == kForward ? kRowPairs : W == kInput ? kTwoSums : kSingle> G;
  const int width = W == kInput ? a.k : a.n;
  return K::template narrow<T, G>(row_tiles(a, G::kQ) * ((width + G::kP - 1) / G::kP), a, v, s);
}

template <GatedWay W, typename K, typename T, bool DMA>
int launch_gated_rows(const GatedArgs& a, const GatedTensors& v, hipStream_t s) {
  const int64_t mean = a.rows / a.groups;
  const int width = W == kInput ? a.k : a.n, wide = W == kForward ? 2 * width : width;   // columns of P
  if (mean < 16 || row_tiles(a, 64) * ((wide + 127) / 128) < 96)
    return launch_gated_tile<W, K, T, DMA, 128, 16, 4, 1, 4>(a, v, s);
  if (mean < 64 || row_tiles(a, 128) * ((wide + 127) / 128) < 300)
    return launch_gated_tile<W, K, T, DMA, 128, 64, 2, 2, 3>(a, v, s);
  if constexpr (DMA) {
    const int red = W == kInput ? a.n : a.k;
    if (row_tiles(a, 128) * ((wide + 255) / 256) >= 768 && red >= 1024) {
      typedef WideGemm<T, W != kForward, W == kForward ? kRowPairs : W == kInput ? kTwoSums : kSingle> G;
      if (red % kStep == 0) return K::template wide<T, G>(row_tiles(a, G::kQ) * ((width + G::kP - 1) / G::kP), a, v, s);
      return launch_gated_tile<W, K, T, DMA, 256, 128, 4, 2, 3>(a, v, s);
    }
  }
  return launch_gated_tile<W, K, T, DMA, 128, 128, 2, 2, 2>(a, v, s);
}

template <GatedWay W, typename K, typename T>
int launch_gated_type(const GatedArgs& a, const GatedTensors& v, hipStream_t s) {
  bool aligned;
  if (W == kForward)
    aligned = rows16(v.in, a.x_stride) && rows16(v.w, a.w_stride) && rows16(v.w2, a.w_stride) && a.w_group % 8 == 0;
  else if (W == kHidden)
    aligned = rows16(v.in, a.y_stride) && rows16(v.w, a.down_stride) && a.down_group % 8 == 0 && a.n % 8 == 0;
  else
    aligned = rows16(v.in, a.gate_stride) && rows16(v.in2, a.gate_stride) && rows16(v.w, a.w_stride) &&
              rows16(v.w2, a.w_stride) && a.w_group % 8 == 0 && a.k % 8 == 0;
  return aligned ? launch_gated_rows<W, K, T, true>(a, v, s) : launch_gated_rows<W, K, T, false>(a, v, s);
}

template <GatedWay W, typename K>
int launch_gated(const GatedArgs& a, const GatedTensors& v, int type, hipStream_t s) {
  return type == MOE_TYPE_BF16 ? launch_gated_type<W, K, bf16_t>(a, v, s) : launch_gated_type<W, K, fp16_t>(a, v, s);
}

}  // namespace moe
