// The 16-bit and f32 element types of the operators beside the layer: their
// conversions, and loads and stores of up to 8 consecutive elements at any
// element alignment (global accesses of gfx950 need no more).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

typedef __bf16 bf16_t;
typedef _Float16 fp16_t;

inline size_t elem_bytes(int type) { return type == MOE_TYPE_F32 ? 4 : 2; }

typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef bf16_t bf16x8_t __attribute__((ext_vector_type(8)));
typedef fp16_t fp16x8_t __attribute__((ext_vector_type(8)));

// 8 consecutive elements in registers, as they are in memory.
template <typename T>
struct oct_of;
template <>
struct oct_of<bf16_t> { typedef bf16x8_t type; };
template <>
struct oct_of<fp16_t> { typedef fp16x8_t type; };
template <>
struct oct_of<float> { typedef f32x8 type; };
template <typename T>
using oct = typename oct_of<T>::type;

template <typename V>
__device__ __forceinline__ f32x8 to_f32(V v) { return __builtin_convertvector(v, f32x8); }

// The same of bf16 by the bits: an instruction an element.
__device__ __forceinline__ f32x8 unpacked(bf16x8_t v) {
  uint32_t w[4];
  __builtin_memcpy(w, &v, sizeof(w));
  f32x8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __builtin_bit_cast(float, w[i] << 16);
    f[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
  }
  return f;
}
__device__ __forceinline__ f32x8 unpacked(fp16x8_t v) { return to_f32(v); }

// Elements p[0..7] of which the first n are there (n >= 8: all) are loaded in
// two steps: raw_oct asks for them, and placed_oct, where they are used, moves
// them to their places and fills up with zeros. A load with a branch on its own
// data would make the wave wait for each load in turn.
// `room` (the same in every lane): p lies in a row of at least 8 elements that
// ends at p + n if n < 8; the row's last 8 elements are loaded then. A shorter row is loaded one by one.
template <typename T>
__device__ __forceinline__ oct<T> raw_oct(const T* p, int n, bool room) {
  oct<T> o = {};
  if (room) {
    if (n > 0) __builtin_memcpy(&o, p + min(n - 8, 0), 8 * sizeof(T));
  } else if (n > 0) {
#pragma unroll 1
    for (int i = 0; i < min(n, 8); ++i) {
      const T v = p[i];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = e == i ? v : o[e];
    }
  }
  return o;
}
template <typename T>
__device__ __forceinline__ oct<T> placed_oct(oct<T> o, int n, bool room) {
  if (!room) return o;
  constexpr int W = 2 * sizeof(T);   // words
  uint32_t w[W];
  const int by = min(max(8 - n, 0), 8);
  __builtin_memcpy(w, &o, sizeof(w));
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = by & 8 ? 0 : w[i];
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = by & 4 ? (i + 2 < W ? w[i + 2] : 0) : w[i];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = by & 2 ? (i + 1 < W ? w[i + 1] : 0) : w[i];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = by & 1 ? (i + 1 < W ? w[i + 1] << 16 : 0) | w[i] >> 16 : w[i];
  } else {
#pragma unroll
    for (int s = 4; s > 0; s /= 2)
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = by & s ? (i + s < W ? w[i + s] : 0) : w[i];
  }
  __builtin_memcpy(&o, w, sizeof(w));
  return o;
}
template <typename T>
__device__ __forceinline__ oct<T> load_oct(const T* p, int n, bool room) {
  return placed_oct<T>(raw_oct(p, n, room), n, room);
}

// The first n of f rounded to nearest even in T (infinities and NaN kept).
template <typename T>
__device__ __forceinline__ void store_oct(T* p, f32x8 f, int n) {
  const oct<T> o = __builtin_convertvector(f, oct<T>);
  if (n >= 8) {
    __builtin_memcpy(p, &o, 8 * sizeof(T));
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = o[i];
  }
}

}  // namespace moe
