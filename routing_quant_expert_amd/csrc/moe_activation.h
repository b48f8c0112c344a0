// The gated activation of the operators beside the layer, in f32:
//   h = act(min(g, L)) * clamp(u, -L, L),  act(z) = z s(z),
// s the logistic function of z (silu) or of 2 sqrt(2/pi) (z + 0.044715 z^3)
// (gelu in its tanh form), and its gradient.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/moe.h"

namespace moe {

struct Gate {
  int act;       // MOE_ACT_SILU or MOE_ACT_GELU
  float limit;   // infinity: none
};

// e^x for x <= 0: 2^t with t = x log2(e) rounded, and what the rounding left
// to first order: about two steps of f32 off down to e^-87, then 0.
__device__ __forceinline__ float exp_f32(float x) {
  const float t = x * 0x1.715476p+0f;
  const float left = __builtin_fmaf(x, 0x1.4ae0cp-26f, __builtin_fmaf(x, 0x1.715476p+0f, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, left * 0x1.62e43p-1f, e);
}

// act(z) and, with SLOPE, its derivative s + z s (1 - s) inner'. Past +-104 both
// are their limits to f32 (which also keeps infinities from meeting zeros); NaN stays.
template <bool SLOPE>
__device__ __forceinline__ float activation(const Gate& a, float z, float& slope) {
  z = z < -104.0f ? -104.0f : z;
  const float y = z > 104.0f ? 104.0f : z;
  float inner = y, by = 1.0f;
  if (a.act == MOE_ACT_GELU) {
    constexpr float c = 1.5957691216057308f;   // 2 sqrt(2/pi)
    inner = c * __builtin_fmaf(0.044715f * y * y, y, y);
    by = c * __builtin_fmaf(0.134145f * y, y, 1.0f);
  }
  const float e = exp_f32(-__builtin_fabsf(inner)), high = __builtin_amdgcn_rcpf(1.0f + e), low = e * high;
  const float s = inner < 0.0f ? low : high;
  if (SLOPE) slope = __builtin_fmaf(y * s, (inner < 0.0f ? high : low) * by, s);
  return z * s;
}

__device__ __forceinline__ float at_most(float v, float limit) { return v > limit ? limit : v; }
__device__ __forceinline__ float clamped(float v, float limit) { return v > limit ? limit : v < -limit ? -limit : v; }

__device__ __forceinline__ float gated(const Gate& a, float g, float u) {
  float unused;
  return activation<false>(a, at_most(g, a.limit), unused) * clamped(u, a.limit);
}
// h again, and the gradients of g and u for that of h (the clamps' ends pass it).
__device__ __forceinline__ float gated_back(const Gate& a, float g, float u, float dh, float& dg, float& du) {
  float slope;
  const float v = activation<true>(a, at_most(g, a.limit), slope), uc = clamped(u, a.limit);
  dg = g > a.limit ? 0.0f : dh * uc * slope;
  du = u > a.limit || u < -a.limit ? 0.0f : dh * v;
  return v * uc;
}

}  // namespace moe
