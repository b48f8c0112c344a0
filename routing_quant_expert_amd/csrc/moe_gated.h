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

// Which tiles. The times are of bf16 at n = 2048, k = 4096, rows as `rows of groups` (a power law of 0.4), in us.
// The counts of tiles and rows below are points among the sizes that were timed, a little off the chip's own 256 and 512 where
// the times cross there; the crossings differ by way and width, and no single point has the faster side at all of them.
// Few tiles (480 of 64 columns, about two for a CU): the smallest, for more workgroups. 1 of 1: forward 12.3 against 15.1 in
// tiles of 128 columns, hidden 12.8 (16.7), input 12.6 (16.8); past it those read the rows less often: hidden of 100 of 8 37.4
// (28.8). Around it: 100 of 8, n = 1024, k = 2048, forward (384 tiles) 12.3 (13.3), input (480) 17.5 (14.5); hidden of 128 of 1
// (320) 13.9 (18.1), 224 of 1 (512) 20.2 (19.9); but 192 of 1 forward (512) still 19.4 (27.0), hidden (448) already 23.1 (18.8).
// Unaligned rows wait longer for each load: up to 768. bf16, 257 and 515 wide: hidden of 1000 of 13 (380) 12.5 (15.6), input (684)
// 13.7 (16.8), of 1600 (1026) 15.9 (19.3), of 2400 (1476) 20.9 (17.2, 64 rows); 515 and 1001 wide, input of 1500 of 32 (2000) 38.3 (34.5).
// Tall tiles for few rows: under 6 a group forward of 64 of 32 171.7 against 171.7 with 64 rows, 192 of 32 174.2 (175.2), 256 of 32
// 190.5 (176.5); and where tiles of 64 rows would be few, up to 160: hidden of 256 of 1 (96) 19.7 (29.9), input of 128 of 1 (128)
// 17.7 (25.4), but hidden of 512 of 1 (160) 33.5 (30.2), 640 of 1 (192) 42.8 (30.7).
// Tiles of 64 rows for middling groups (under 64 rows) and up to 300 tiles of 128 rows: hidden of 1024 of 1 (160) 32.5 against 51.1
// with 128 rows, 2048 of 1 (288) 52.6 (54.8), 2304 of 1 (320) 71.3 (66.5); input of 1024 of 1 (320) 44.7 (43.6); forward of 400 of 8,
// n = 1024, k = 2048, 15.8 (26.0), but 1536 of 32 204.9 (198.1).
// Wide tiles (moe_wide.h): a round of 256 of them takes about three halves of one of 512 tiles of 128 x 128, so where 3 times
// its rounds are less than twice theirs. Forward of 16384 of 32 530 (597), of k = 512 134 (161), 2048 of 4 87 (123), but 2048
// of 1 88 (67). Where both are equal a round has just begun, and the larger tiles are the better ones for the hidden rows and
// long sums: 4096 of 4 171 (182), hidden 8192 of 32 236 (263), but 8000 of 8 with n = 1024, k = 2048 106 (95). From 768
// tiles on, what counts is the weights' reading, which they do in longer rows: 12288 of 96 723 (774), input 644 (776). The
// backward pass, whose weights' rows lie across the sum, gains by that with few rows too, if most of the CUs have a
// tile: input of 64 of 32 165 (181), 32 of 8 60 (50). The forward pass does not under 24 rows: 4000 of 384 2198 (2194).
// At 4 steps they are still ahead: forward of 16384 of 32, n = 4096, k = 256, 211 (238); shorter sums are not tried.
template <GatedWay W, typename K, typename T, bool DMA>
int launch_gated_rows(const GatedArgs& a, const GatedTensors& v, hipStream_t s) {
  const int64_t mean = a.rows / a.groups;
  const int width = W == kInput ? a.k : a.n, wide = W == kForward ? 2 * width : width;   // columns of P
  auto columns = [&](int p) { return (wide + p - 1) / p; };
  constexpr int kFewRows = W == kForward ? 32 : 16;   // (of 16 rows a wave would have no row of both projections)
  if (row_tiles(a, kFewRows) * columns(64) < (DMA ? 480 : 768)) {
    if constexpr (W == kForward) return launch_gated_tile<W, K, T, DMA, 64, 32, 2, 2, 4>(a, v, s);
    else return launch_gated_tile<W, K, T, DMA, 64, 16, 4, 1, 4>(a, v, s);
  }
  if constexpr (DMA) {
    const int red = W == kInput ? a.n : a.k;
    const int64_t tiles = likely_row_tiles(a, 256) * columns(256), small = likely_row_tiles(a, 128) * columns(128);
    const int64_t ours = 3 * rounds(a, tiles, 256), theirs = 2 * rounds(a, small, 512);
    const bool close = W == kHidden || (W == kInput ? 2 : 1) * (int64_t)red >= 4096;
    const bool pays = mean < 64 ? W != kForward ? tiles >= 128 : mean >= 24 && tiles >= 768
                                : tiles >= 768 || ours < theirs || (ours == theirs && close);
    if (pays && red >= 4 * kStep && red % kStep == 0) {
      typedef WideGemm<T, W != kForward, W == kForward ? kRowPairs : W == kInput ? kTwoSums : kSingle> G;
      return K::template wide<T, G>(row_tiles(a, G::kQ) * ((width + G::kP - 1) / G::kP), a, v, s);
    }
  }
  if (mean < 6 || row_tiles(a, 64) * columns(128) <= 160) return launch_gated_tile<W, K, T, DMA, 128, 16, 4, 1, 4>(a, v, s);
  if (mean < 64 || row_tiles(a, 128) * columns(128) < 300) return launch_gated_tile<W, K, T, DMA, 128, 64, 2, 2, 3>(a, v, s);
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
