// Joining a block to the residual stream (moe_join_forward, moe_join_backward):
// the norm after a block, its gate and residual scale, the residual add and
// the norm before the next block as one pass over the rows, and its gradients.
//
//   z = b rb w_post, x' = x + s g z, y = x' rx w_pre,  r? = rsqrt(mean(.^2) + eps)
// and backwards, with n = x' rx, dn = dy w_pre, nb = b rb, dz = s g dx:
//   dx = dx_out + rx (dn - n mean(dn n)),  db = rb (dz w_post - nb mean(dz w_post nb)),
//   dw_pre = sum dy n, dw_post = sum dz nb, dgate = s dx z.
//
// Bound by HBM: every operand is read once and every result written once, the
// row stays in registers in between (8192 rows of 4096, f32 stream: forward 75
// us, 5.4 TB/s, gradients 120 us, 5.0 TB/s; a copy reaches 5.1). 4096 rows in
// 16 bits, gradients: 51 us, 3.9 TB/s, of which the column sums take 4. One
// row of 4096: 3.8 us in the kernel, 4.6 with the call. Gradients of rows wider
// than 8192 are read twice and do not fit the registers (k_join_back): 1500
// rows of 16384 take 223 us, 1.3 TB/s, where the forward pass takes 46. A row belongs to TPR threads (one wave,
// or a workgroup), thread t holding the chunks t, t + TPR, ... of 8 elements
// (the last one short where the row is no multiple of 8).
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "moe_element.h"
#include "moe_host.h"
#include "moe_wave.h"

namespace moe {
namespace {

constexpr int kJoinThreads = 256;
constexpr int64_t kJoinMaxRows = (int64_t)1 << 22;   // rows * 1024 threads stay below a launch's 2^32 threads

struct JoinArgs {
  int dim;
  int gate_rows;
  float scale, eps;
  int64_t m;
  int64_t x_stride, x_out_stride, b_stride, gate_stride, y_stride;
};

// Sums of N values over the TPR threads of a row, in every one of them. TPR =
// 64: the wave's butterfly; more: the waves' sums meet in LDS (`buf` is used
// by one call of the row; the next call takes the other buffer, so one barrier a call is enough).
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* buf) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum_xor(v[i]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[i * W + wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += buf[i * W + w];
      v[i] = s;
    }
  }
}

__device__ __forceinline__ float sum_of_squares(f32x8 f) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(f[i], f[i], s);
  return s;
}

__device__ __forceinline__ f32x8 fma8(f32x8 a, f32x8 b, f32x8 c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = fmaf(a[i], b[i], c[i]);
  return c;
}
__device__ __forceinline__ f32x8 fma8(f32x8 a, float b, f32x8 c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = fmaf(a[i], b, c[i]);
  return c;
}

__device__ __forceinline__ float dot8(f32x8 a, f32x8 b) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
  return s;
}

// How rows end (chosen by the launch: a branch at every load costs 10 to 30%):
// whole chunks, a short one at the end, or a row of less than one chunk.
enum Rows { kWhole, kRagged, kTiny };
template <int ROWS, typename T>
__device__ __forceinline__ oct<T> raw_chunk(const T* p, int n) {
  if constexpr (ROWS != kWhole) return raw_oct(p, n, ROWS == kRagged);
  oct<T> o = {};
  if (n > 0) __builtin_memcpy(&o, p, sizeof(o));
  return o;
}
template <int ROWS, typename T>
__device__ __forceinline__ oct<T> placed_chunk(oct<T> o, int n) {
  return ROWS == kRagged ? placed_oct<T>(o, n, true) : o;
}

// (x_out may be x and y may be b: each thread has read what it overwrites.)
template <typename T, typename RT, int TPR, int NC, int ROWS>
__global__ __launch_bounds__(TPR < kJoinThreads ? kJoinThreads : TPR) void k_join(
    JoinArgs a, const RT* x, const T* b, const T* __restrict__ w_post, const T* __restrict__ gate,
    const T* __restrict__ w_pre, RT* x_out, T* y) {
  constexpr int kRows = TPR < kJoinThreads ? kJoinThreads / TPR : 1;
  __shared__ float buf[2][TPR / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  if (row >= a.m) return;   // whole waves; with TPR > 64 the whole workgroup
  // Everything is asked for at once, the vectors too (from the caches): a call of few rows waits for memory once.
  f32x8 xv[NC];
  const float inv_dim = 1.0f / (float)a.dim;
  oct<RT> xr[NC];
  oct<T> br[NC] = {}, po[NC] = {}, ga[NC] = {}, pr[NC] = {};
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = 8 * (t + TPR * i), left = a.dim - c;
    xr[i] = raw_chunk<ROWS>(x + row * a.x_stride + c, left);
    if (b) br[i] = raw_chunk<ROWS>(b + row * a.b_stride + c, left);
    if (w_post) po[i] = raw_chunk<ROWS>(w_post + c, left);
    if (gate) ga[i] = raw_chunk<ROWS>(gate + (a.gate_rows ? row * a.gate_stride : 0) + c, left);
    if (w_pre) pr[i] = raw_chunk<ROWS>(w_pre + c, left);
  }
  if (ROWS != kWhole) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int left = a.dim - 8 * (t + TPR * i);
      xr[i] = placed_chunk<ROWS, RT>(xr[i], left);
      br[i] = placed_chunk<ROWS, T>(br[i], left);
      po[i] = placed_chunk<ROWS, T>(po[i], left);
      ga[i] = placed_chunk<ROWS, T>(ga[i], left);
      pr[i] = placed_chunk<ROWS, T>(pr[i], left);
    }
  }
  if (b) {
    float rb = 1.0f;
    if (w_post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NC; ++i) s[0] += sum_of_squares(to_f32(br[i]));
      row_sums<TPR>(s, buf[0]);
      rb = 1.0f / sqrtf(s[0] * inv_dim + a.eps);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      f32x8 z = to_f32(br[i]);
      if (w_post) z = z * rb * to_f32(po[i]);
      if (gate) z = z * to_f32(ga[i]);
      xv[i] = to_f32(xr[i]) + a.scale * z;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NC; ++i) xv[i] = to_f32(xr[i]);
  }
  if (x_out) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = 8 * (t + TPR * i);
      store_oct(x_out + row * a.x_out_stride + c, xv[i], a.dim - c);
    }
  }
  if (!w_pre) return;
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NC; ++i) s[0] += sum_of_squares(xv[i]);
  row_sums<TPR>(s, buf[1]);
  const float rx = 1.0f / sqrtf(s[0] * inv_dim + a.eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = 8 * (t + TPR * i);
    store_oct(y + row * a.y_stride + c, xv[i] * rx * to_f32(pr[i]), a.dim - c);
  }
}

// The gradients: workgroup p takes the rows p, p + P, ... (P workgroups), so
// that its threads keep the sums over rows of their columns in registers; they
// are written as f32 partial sums [P][3][dim] that k_join_sums adds up.
// The vectors and the row stay in registers in workgroups of up to 512 threads
// (dim <= 8192), and the next two rows are on their way while one is worked on
// where NC is 1 (dim <= 4096). Wider rows are read again where they are used,
// from the caches: 1024 threads have 128 registers each, of which the sums of
// two chunks take 48, and the compiler still keeps 132 to 155 of a thread's
// values in scratch memory, as it does 64 of f32 streams of odd widths from
// 4097 to 8191 (1500 rows: 82 us of 8191, 52 of 8192).
//
// One reduction a row: with d = dy w_pre and h = gate w_post b, the sum that
// db needs, of dz w_post nb, is s rb (sum h dx_out + rx (sum h d - c1 sum h x')),
// so its three parts are summed together with those of x'^2, d x' and b^2.
template <typename T, typename RT>
struct JoinChunk {
  oct<RT> dxo, xo;
  oct<T> dy, b, gate;
};

template <typename T, typename RT, int TPR, int NC, int ROWS>
__global__ __launch_bounds__(TPR) void k_join_back(JoinArgs a, const T* __restrict__ dy, const RT* dxo,
                                                   const RT* __restrict__ xo, const T* b,
                                                   const T* __restrict__ w_post, const T* __restrict__ gate,
                                                   const T* __restrict__ w_pre, RT* dx, T* db,
                                                   T* __restrict__ dgate_rows,
                                                   float* __restrict__ part, int sums) {
  constexpr bool kKeep = TPR <= 512, kAhead = kKeep && NC == 1;
  typedef JoinChunk<T, RT> Chunk;
  // (in f32 where they fit: at 16 bits the kernel's time is its vector instructions as much as HBM's)
  typedef std::conditional_t<kAhead, f32x8, oct<T>> Vector;
  struct Vectors {
    Vector pre, post, gate;
  };
  __shared__ float buf[2][6 * (TPR / 64)];
  const int t = threadIdx.x;
  const float inv_dim = 1.0f / (float)a.dim;
  const bool through = db && w_post;   // db goes through the norm
  auto vectors_at = [&](int c) {
    Vectors v = {};
    auto get = [&](const T* p) {
      const oct<T> o = placed_chunk<ROWS, T>(raw_chunk<ROWS>(p + c, a.dim - c), a.dim - c);
      return __builtin_convertvector(o, Vector);
    };
    if (dy) v.pre = get(w_pre);
    if (w_post) v.post = get(w_post);
    if (gate && !a.gate_rows) v.gate = get(gate);
    return v;
  };
  auto chunk_at = [&](int64_t row, int c) {
    Chunk r = {};
    const int left = a.dim - c;
    if (dxo) r.dxo = raw_chunk<ROWS>(dxo + row * a.x_out_stride + c, left);
    if (dy) {
      r.xo = raw_chunk<ROWS>(xo + row * a.x_out_stride + c, left);
      r.dy = raw_chunk<ROWS>(dy + row * a.y_stride + c, left);
    }
    if (b) r.b = raw_chunk<ROWS>(b + row * a.b_stride + c, left);
    if (gate && a.gate_rows) r.gate = raw_chunk<ROWS>(gate + row * a.gate_stride + c, left);
    return r;
  };
  // Rows of no multiple of 8 elements: the chunks put in place, where they are used.
  auto place_chunk = [&](Chunk& r, int c) {
    r.dxo = placed_chunk<ROWS, RT>(r.dxo, a.dim - c);
    r.xo = placed_chunk<ROWS, RT>(r.xo, a.dim - c);
    r.dy = placed_chunk<ROWS, T>(r.dy, a.dim - c);
    r.b = placed_chunk<ROWS, T>(r.b, a.dim - c);
    r.gate = placed_chunk<ROWS, T>(r.gate, a.dim - c);
  };
  auto gate_of = [&](const Chunk& r, const Vectors& v) { return a.gate_rows ? to_f32(r.gate) : to_f32(v.gate); };
  f32x8 s_pre[NC] = {}, s_post[NC] = {}, s_gate[NC] = {};
  Vectors vec[NC];
  Chunk cur[NC], next[NC], then[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (kKeep) vec[i] = vectors_at(8 * (t + TPR * i));
    if (kAhead) {
      next[i] = chunk_at(blockIdx.x, 8 * (t + TPR * i));
      if (blockIdx.x + gridDim.x < a.m) then[i] = chunk_at(blockIdx.x + gridDim.x, 8 * (t + TPR * i));
    }
  }
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x, turn ^= 1) {
    if (kAhead) {
      // (dx may be dx_out and db may be b: only this workgroup writes its rows, each after it was read)
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        cur[i] = next[i];
        next[i] = then[i];
        if (row + 2 * (int64_t)gridDim.x < a.m) then[i] = chunk_at(row + 2 * (int64_t)gridDim.x, 8 * (t + TPR * i));
      }
    }
    float s[6] = {};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = 8 * (t + TPR * i);
      if (!kAhead) cur[i] = chunk_at(row, c);
      if (!kKeep) vec[i] = vectors_at(c);
      place_chunk(cur[i], c);
      const Chunk& r = cur[i];
      const Vectors& v = vec[i];
      const f32x8 bv = to_f32(r.b), xv = to_f32(r.xo), d = to_f32(r.dy) * to_f32(v.pre);
      s[0] += sum_of_squares(xv);
      s[1] += dot8(d, xv);
      if (w_post) s[2] += sum_of_squares(bv);
      if (through) {
        f32x8 h = bv * to_f32(v.post);
        if (gate) h = h * gate_of(r, v);
        s[3] += dot8(h, to_f32(r.dxo));
        s[4] += dot8(h, d);
        s[5] += dot8(h, xv);
      }
    }
    row_sums<TPR>(s, buf[turn]);   // (the next row takes the other buffer: one barrier a row is enough)
    const float rx = 1.0f / sqrtf(s[0] * inv_dim + a.eps);
    const float c1 = s[1] * rx * rx * inv_dim;   // mean(dn n) rx: n mean(dn n) = x' c1
    const float rb = w_post ? 1.0f / sqrtf(s[2] * inv_dim + a.eps) : 1.0f;
    // rb mean(dz w_post nb)
    const float c2 = through ? rb * rb * a.scale * inv_dim * (dy ? s[3] + rx * (s[4] - c1 * s[5]) : s[3]) : 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = 8 * (t + TPR * i), left = a.dim - c;
      if (!kKeep) {
        cur[i] = chunk_at(row, c);
        vec[i] = vectors_at(c);
        place_chunk(cur[i], c);
      }
      const Chunk& r = cur[i];
      const Vectors& v = vec[i];
      f32x8 g = to_f32(r.dxo);
      if (dy) {
        const f32x8 xv = to_f32(r.xo), dn = to_f32(r.dy);
        s_pre[i] = fma8(dn, xv * rx, s_pre[i]);
        g = fma8(fma8(xv, -c1, dn * to_f32(v.pre)), rx, g);
      }
      store_oct(dx + row * a.x_stride + c, g, left);
      if (!b) continue;
      const f32x8 bv = to_f32(r.b), nb = bv * rb;
      f32x8 dz = g * a.scale;
      f32x8 z = nb;
      if (w_post) z = z * to_f32(v.post);
      if (gate) {
        if (!a.gate_rows) s_gate[i] = fma8(dz, z, s_gate[i]);
        else if (dgate_rows) store_oct(dgate_rows + row * a.gate_stride + c, dz * z, left);
        dz = dz * gate_of(r, v);
      }
      if (w_post) {
        s_post[i] = fma8(dz, nb, s_post[i]);
        dz = fma8(bv, -c2, dz * to_f32(v.post)) * rb;
      }
      if (db) store_oct(db + row * a.b_stride + c, dz, left);
    }
  }
  if (!sums) return;
  float* out = part + (int64_t)blockIdx.x * 3 * a.dim;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = 8 * (t + TPR * i), left = a.dim - c;
    if (left <= 0) break;
    store_oct(out + c, s_pre[i], left);
    store_oct(out + a.dim + c, s_post[i], left);
    store_oct(out + 2 * (int64_t)a.dim + c, s_gate[i], left);
  }
}

// Column sums of the partial sums [parts][3 * dim], in a fixed order: 64
// columns a workgroup, wave w adding the rows w, w + 16, ...
__global__ __launch_bounds__(1024) void k_join_sums(const float* __restrict__ part, int parts, int dim,
                                                    float* __restrict__ dw_pre, float* __restrict__ dw_post,
                                                    float* __restrict__ dgate) {
  __shared__ float buf[16][64];
  const int which = blockIdx.y;
  float* out = which == 0 ? dw_pre : which == 1 ? dw_post : dgate;
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  const float* from = part + (int64_t)which * dim + min(col, dim - 1);
  float s = 0.0f;
#pragma unroll 8
  for (int p = wave; p < parts; p += 16) s += from[(int64_t)p * 3 * dim];
  buf[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < dim) {
#pragma unroll
    for (int w = 1; w < 16; ++w) s += buf[w][lane];
    out[col] = s;
  }
}

// Workgroups of the gradient kernel for m rows: as many as run at once (its
// registers leave 8 waves a CU), but at least 4 rows each where that still gives one a CU: a workgroup's
// partial sums cost as much traffic as a row. 8192 rows of 512: 24 us with 1024
// workgroups, 31 with 512, 48 with 256; of 2048: 50 with 512, 60 with 256; 4096
// rows of 4096: 59 with 512, 52 with 256.
int join_parts(int dim, int64_t m) {
  const int64_t at_once = dim <= 1024 ? 1024 : dim <= 2048 ? 512 : 256;
  const int64_t fed = m / 4 > 256 ? m / 4 : 256;
  const int64_t parts = at_once < fed ? at_once : fed;
  return (int)(m < parts ? (m < 1 ? 1 : m) : parts);
}

int check_join(const moe_join* j, int64_t m) {
  if (!j) return fail(MOE_EINVAL, "join is NULL%s%lld");
  if (j->type != MOE_TYPE_BF16 && j->type != MOE_TYPE_FP16)
    return fail(MOE_EINVAL, "join: type must be MOE_TYPE_BF16 or MOE_TYPE_FP16%s (%lld)", "", j->type);
  if (j->residual_type != j->type && j->residual_type != MOE_TYPE_F32)
    return fail(MOE_EINVAL, "join: residual_type must be type or MOE_TYPE_F32%s (%lld)", "", j->residual_type);
  if (j->gate_rows != 0 && j->gate_rows != 1)
    return fail(MOE_EINVAL, "join: gate_rows must be 0 or 1%s (%lld)", "", j->gate_rows);
  if (!std::isfinite(j->scale) || !(j->eps > 0.0f) || !std::isfinite(j->eps))
    return fail(MOE_EINVAL, "join: scale must be finite and eps finite and > 0%s%lld");
  if (j->dim < 1) return fail(MOE_EINVAL, "join: dim must be >= 1%s (%lld)", "", j->dim);
  if (j->dim > MOE_JOIN_MAX_DIM) return fail(MOE_EUNSUPPORTED, "join: dim above MOE_JOIN_MAX_DIM%s (%lld)", "", j->dim);
  if (j->x_stride < j->dim || j->x_out_stride < j->dim || j->b_stride < j->dim || j->y_stride < j->dim ||
      (j->gate_rows && j->gate_stride < j->dim))
    return fail(MOE_EINVAL, "join: a row stride is below dim%s (%lld)", "", j->dim);
  if (m < 1) return fail(MOE_EINVAL, "m must be >= 1%s (m %lld)", "", m);
  if (m >= kJoinMaxRows) return fail(MOE_EUNSUPPORTED, "join: too many rows%s (m %lld)", "", m);
  return MOE_OK;
}

// In place (`out` is `in`): rows of one stride. With two strides a row would be
// written where another one, still to be read by another workgroup, lies.
bool other_rows(const void* in, int64_t in_stride, const void* out, int64_t out_stride, int64_t m) {
  return out && in == out && in_stride != out_stride && m > 1;
}

// An element pointer is aligned to its element.
bool off_element(const void* p, int type) { return (uintptr_t)p % elem_bytes(type) != 0; }

JoinArgs join_args(const moe_join& j, int64_t m) {
  return {j.dim, j.gate_rows, j.scale, j.eps, m, j.x_stride, j.x_out_stride, j.b_stride, j.gate_stride, j.y_stride};
}

template <typename T, typename RT, int TPR, int NC, int ROWS>
void launch_join_as(const JoinArgs& a, const void* x, const void* b, const void* w_post, const void* gate,
                    const void* w_pre, void* x_out, void* y, hipStream_t s) {
  constexpr int kRows = TPR < kJoinThreads ? kJoinThreads / TPR : 1;
  k_join<T, RT, TPR, NC, ROWS><<<dim3((unsigned)((a.m + kRows - 1) / kRows)), dim3(kRows * TPR), 0, s>>>(
      a, (const RT*)x, (const T*)b, (const T*)w_post, (const T*)gate, (const T*)w_pre, (RT*)x_out, (T*)y);
}

template <typename T, typename RT, int ROWS, typename... A>
void launch_join_rows(const JoinArgs& a, A... args) {
  if (a.dim <= 512) launch_join_as<T, RT, 64, 1, ROWS>(a, args...);
  else if (a.dim <= 1024) launch_join_as<T, RT, 64, 2, ROWS>(a, args...);
  else if (a.dim <= 2048) launch_join_as<T, RT, 256, 1, ROWS>(a, args...);
  else if (a.dim <= 4096) launch_join_as<T, RT, 256, 2, ROWS>(a, args...);
  else if (a.dim <= 8192) launch_join_as<T, RT, 512, 2, ROWS>(a, args...);
  else launch_join_as<T, RT, 1024, 2, ROWS>(a, args...);
}

template <typename T, typename RT, typename... A>
void launch_join(const JoinArgs& a, A... args) {
  if (a.dim < 8) launch_join_as<T, RT, 64, 1, kTiny>(a, args...);
  else if (a.dim % 8) launch_join_rows<T, RT, kRagged>(a, args...);
  else launch_join_rows<T, RT, kWhole>(a, args...);
}

template <typename T, typename RT, int TPR, int NC, int ROWS>
void launch_back_as(const JoinArgs& a, const void* dy, const void* dxo, const void* xo, const void* b,
                    const void* w_post, const void* gate, const void* w_pre, void* dx, void* db, void* dgate_rows,
                    float* part, int sums, hipStream_t s) {
  k_join_back<T, RT, TPR, NC, ROWS><<<dim3(join_parts(a.dim, a.m)), dim3(TPR), 0, s>>>(
      a, (const T*)dy, (const RT*)dxo, (const RT*)xo, (const T*)b, (const T*)w_post, (const T*)gate, (const T*)w_pre,
      (RT*)dx, (T*)db, (T*)dgate_rows, part, sums);
}

template <typename T, typename RT, int ROWS, typename... A>
void launch_back_rows(const JoinArgs& a, A... args) {
  if (a.dim <= 512) launch_back_as<T, RT, 64, 1, ROWS>(a, args...);
  else if (a.dim <= 1024) launch_back_as<T, RT, 128, 1, ROWS>(a, args...);
  else if (a.dim <= 2048) launch_back_as<T, RT, 256, 1, ROWS>(a, args...);
  else if (a.dim <= 4096) launch_back_as<T, RT, 512, 1, ROWS>(a, args...);
  else if (a.dim <= 8192) launch_back_as<T, RT, 512, 2, ROWS>(a, args...);
  else launch_back_as<T, RT, 1024, 2, ROWS>(a, args...);
}

template <typename T, typename RT, typename... A>
void launch_back(const JoinArgs& a, A... args) {
  if (a.dim < 8) launch_back_as<T, RT, 64, 1, kTiny>(a, args...);
  else if (a.dim % 8) launch_back_rows<T, RT, kRagged>(a, args...);
  else launch_back_rows<T, RT, kWhole>(a, args...);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_join_forward(const moe_join* j, const void* x, const void* b, const void* w_post, const void* gate,
                     const void* w_pre, int64_t m, void* x_out, void* y, void* stream) {
  if (int r = check_join(j, m)) return r;
  if (!x) return fail(MOE_EINVAL, "join: x must be non-NULL%s%lld");
  if (b && !x_out) return fail(MOE_EINVAL, "join: x_out must be non-NULL where there is a block output%s%lld");
  if (!b && (w_post || gate)) return fail(MOE_EINVAL, "join: w_post and gate need a block output%s%lld");
  if (!w_pre != !y) return fail(MOE_EINVAL, "join: w_pre and y go together%s%lld");
  if (!x_out && !y) return fail(MOE_EINVAL, "join: nothing to write%s%lld");
  for (const void* p : {b, w_post, gate, w_pre, (const void*)y})
    if (off_element(p, j->type)) return fail(MOE_EINVAL, "join: a pointer is not aligned to its elements%s%lld");
  for (const void* p : {x, (const void*)x_out})
    if (off_element(p, j->residual_type)) return fail(MOE_EINVAL, "join: a pointer is not aligned to its elements%s%lld");
  if (other_rows(x, j->x_stride, x_out, j->x_out_stride, m) || other_rows(b, j->b_stride, y, j->y_stride, m))
    return fail(MOE_EINVAL, "join: in place with two row strides%s%lld");
  const JoinArgs a = join_args(*j, m);
  const hipStream_t s = (hipStream_t)stream;
  const bool f32 = j->residual_type == MOE_TYPE_F32;
  if (j->type == MOE_TYPE_BF16)
    f32 ? launch_join<bf16_t, float>(a, x, b, w_post, gate, w_pre, x_out, y, s)
        : launch_join<bf16_t, bf16_t>(a, x, b, w_post, gate, w_pre, x_out, y, s);
  else
    f32 ? launch_join<fp16_t, float>(a, x, b, w_post, gate, w_pre, x_out, y, s)
        : launch_join<fp16_t, fp16_t>(a, x, b, w_post, gate, w_pre, x_out, y, s);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MOE_OK : hip_fail(e, "join");
}

size_t moe_join_workspace_bytes(const moe_join* j, int64_t max_m) {
  if (check_join(j, max_m)) return 0;
  return ((size_t)join_parts(j->dim, max_m) * 3 * j->dim * sizeof(float) + 255) & ~(size_t)255;
}

int moe_join_backward(const moe_join* j, const void* dy, const void* dx_out, const void* x_out, const void* b,
                      const void* w_post, const void* gate, const void* w_pre, int64_t m, void* dx, void* db,
                      float* dw_post, void* dgate, float* dw_pre, void* ws, size_t ws_bytes, void* stream) {
  if (int r = check_join(j, m)) return r;
  if (!dy && !dx_out) return fail(MOE_EINVAL, "join: dy or dx_out must be non-NULL%s%lld");
  if (!dx) return fail(MOE_EINVAL, "join: dx must be non-NULL%s%lld");
  if (dy && (!x_out || !w_pre)) return fail(MOE_EINVAL, "join: dy needs x_out and w_pre%s%lld");
  if (!b && (w_post || gate || db)) return fail(MOE_EINVAL, "join: w_post, gate and db need a block output%s%lld");
  if ((dw_pre && !dy) || (dw_post && !w_post) || (dgate && !gate))
    return fail(MOE_EINVAL, "join: a gradient is asked for whose input is NULL%s%lld");
  for (const void* p : {dy, b, w_post, gate, w_pre, (const void*)db})
    if (off_element(p, j->type)) return fail(MOE_EINVAL, "join: a pointer is not aligned to its elements%s%lld");
  for (const void* p : {dx_out, x_out, (const void*)dx})
    if (off_element(p, j->residual_type)) return fail(MOE_EINVAL, "join: a pointer is not aligned to its elements%s%lld");
  if (off_element(dgate, j->gate_rows ? j->type : MOE_TYPE_F32) || off_element(dw_post, MOE_TYPE_F32) ||
      off_element(dw_pre, MOE_TYPE_F32))
    return fail(MOE_EINVAL, "join: a pointer is not aligned to its elements%s%lld");
  if (other_rows(dx_out, j->x_out_stride, dx, j->x_stride, m))
    return fail(MOE_EINVAL, "join: in place with two row strides%s%lld");
  float* dgate_sum = j->gate_rows ? nullptr : (float*)dgate;
  const int sums = dw_pre || dw_post || dgate_sum;
  if (sums) {
    if (!ws) return fail(MOE_EINVAL, "workspace is NULL%s%lld");
    if ((uintptr_t)ws & 255) return fail(MOE_EINVAL, "workspace must be 256-byte aligned%s%lld");
    const size_t need = moe_join_workspace_bytes(j, m);
    if (ws_bytes < need) return fail(MOE_EWORKSPACE, "workspace too small%s: need %lld bytes", "", (long long)need);
  }
  const JoinArgs a = join_args(*j, m);
  const hipStream_t s = (hipStream_t)stream;
  const bool f32 = j->residual_type == MOE_TYPE_F32;
  void* dgate_rows = j->gate_rows ? dgate : nullptr;
  float* part = (float*)ws;
  if (j->type == MOE_TYPE_BF16)
    f32 ? launch_back<bf16_t, float>(a, dy, dx_out, x_out, b, w_post, gate, w_pre, dx, db, dgate_rows, part, sums, s)
        : launch_back<bf16_t, bf16_t>(a, dy, dx_out, x_out, b, w_post, gate, w_pre, dx, db, dgate_rows, part, sums, s);
  else
    f32 ? launch_back<fp16_t, float>(a, dy, dx_out, x_out, b, w_post, gate, w_pre, dx, db, dgate_rows, part, sums, s)
        : launch_back<fp16_t, fp16_t>(a, dy, dx_out, x_out, b, w_post, gate, w_pre, dx, db, dgate_rows, part, sums, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_fail(e, "join_back");
  if (sums) {
    k_join_sums<<<dim3((j->dim + 63) / 64, 3), dim3(1024), 0, s>>>(part, join_parts(j->dim, m), j->dim, dw_pre, dw_post,
                                                                  dgate_sum);
    e = hipGetLastError();
    if (e != hipSuccess) return hip_fail(e, "join_sums");
  }
  return MOE_OK;
}

}  // extern "C"
