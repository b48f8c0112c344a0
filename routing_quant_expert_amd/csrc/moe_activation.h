// The gated activation of the operators beside the layer, in f32:
//   h = act(min(g, L)) * clamp(u, -L, L),  act(z) = z s(z),
// s the logistic function of z (silu) or of 2 sqrt(2/pi) (z + 0.044715 z^3)
// (gelu in its tanh form), and its gradient.
//
// In wide tiles it is the work of one wave a SIMD for up to 256 outputs a lane,
// about 28 instructions each in the backward pass; there the tile's loads and
// stores take longer (two instructions fewer: the same time).
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/moe.h"

namespace moe {

struct Gate {
  int act;       // MOE_ACT_SILU or MOE_ACT_GELU
  float limit;   // infinity: none
};

// act(z) and, with SLOPE, its derivative s + act(z) (1 - s) inner'(z). s is 1 / (1 + 2^t): t's rounding moves it by
// |t| s (1 - s) 2^-24, which stays below 2^-25. At -infinity act and derivative are 0 (s is 0 below -104); at +infinity the
// derivative is NaN (infinity times 0), and so is everything of NaN. Gelu's inner'(z) is taken of z held to +-104, past which
// 1 - s is 0: the square of a finite z may leave f32, and infinity times 0 is no slope of 1.
template <int ACT, bool SLOPE>
__device__ __forceinline__ float activation(float z, float& slope) {
  constexpr float kLog2e = 1.4426950408889634f, kInner = 1.5957691216057308f, kCubic = 0.044715f;   // 2 sqrt(2/pi)
  float t;
  if (ACT == MOE_ACT_GELU) t = z * __builtin_fmaf(z * z, -kInner * kCubic * kLog2e, -kInner * kLog2e);
  else t = z * -kLog2e;
  const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
  const float y = __builtin_amdgcn_fmed3f(z, -104.0f, INFINITY);   // (NaN is in s)
  const float v = y * s;
  if (SLOPE) {
    float by = 1.0f - s;
    if (ACT == MOE_ACT_GELU) {
      const float w = __builtin_amdgcn_fmed3f(z, -104.0f, 104.0f);
      by *= __builtin_fmaf(w * w, 3.0f * kCubic * kInner, kInner);
    }
    slope = __builtin_fmaf(v, by, s);
  }
  return v;
}

// (Comparisons, not minima: NaN stays.)
__device__ __forceinline__ float held(float v, bool over, float limit) { return over ? __builtin_copysignf(limit, v) : v; }

template <int ACT>
__device__ __forceinline__ float gated(float g, float u, float limit) {
  float unused;
  return activation<ACT, false>(held(g, g > limit, limit), unused) * held(u, __builtin_fabsf(u) > limit, limit);
}
// h again, and the gradients of g and u for that of h (the clamps' ends pass it).
template <int ACT>
__device__ __forceinline__ float gated_back(float g, float u, float dh, float limit, float& dg, float& du) {
  const bool g_over = g > limit, u_over = __builtin_fabsf(u) > limit;
  float slope;
  const float v = activation<ACT, true>(held(g, g_over, limit), slope), uc = held(u, u_over, limit);
  dg = g_over ? 0.0f : dh * uc * slope;
  du = u_over ? 0.0f : dh * v;
  return v * uc;
}

// The same for N neighbouring outputs (vectors of f32), the activation chosen once.
template <typename V>
__device__ __forceinline__ V gated_all(const Gate& a, V g, V u) {
  constexpr int N = sizeof(V) / 4;
  V h;
  if (a.act == MOE_ACT_SILU) {
#pragma unroll
    for (int e = 0; e < N; ++e) h[e] = gated<MOE_ACT_SILU>(g[e], u[e], a.limit);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) h[e] = gated<MOE_ACT_GELU>(g[e], u[e], a.limit);
  }
  return h;
}
template <int ACT, typename V>
__device__ __forceinline__ V gated_back_all(V g, V u, V dh, float limit, V& dg, V& du) {
  constexpr int N = sizeof(V) / 4;
  V h;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    float x, y;
    h[e] = gated_back<ACT>(g[e], u[e], dh[e], limit, x, y);
    dg[e] = x;
    du[e] = y;
  }
  return h;
}

}  // namespace moe
