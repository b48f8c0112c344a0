// The matrix core of the operators beside the layer: one workgroup's tile
//   C[q][p] = sum over r of Q(q, r) P(p, r),   q < BQ, p < BP,
// on v_mfma_f32_16x16x32 (bf16 or fp16, f32 sums), operands staged in LDS.
//
// An operand is stored either in rows (its reduction axis r is contiguous) or
// in columns (its own axis is contiguous, r strides): weights are read as they
// lie for a product and for its input gradient, activations as they lie for a
// weight gradient. A step is 64 r. Its tiles sit in LDS as they came from
// memory, in 16-byte chunks whose place within the row is XORed with a few
// bits of the row, so that the lanes of an operand read spread over the banks.
// A row tile is read with plain 16-byte reads (lane l: row l%16, eight r from
// 8 * (l/16)); a column tile with the transposing 8-byte reads of gfx950,
// which hand lane l of 16 the four r of column l from four rows of 16 columns.
//
// P is the output's contiguous axis and the MFMA's row operand: a lane then
// holds four neighbouring outputs of one row.
#pragma once

#include <type_traits>

#include "moe_element.h"
#include "moe_internal.h"
#include "moe_kquant.h"

namespace moe {

constexpr int kStep = 64;   // r per step

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4g __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_tr_t;

__device__ __forceinline__ f32x4 mfma16(bf16x8_t a, bf16x8_t b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(fp16x8_t a, fp16x8_t b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// An operand of one tile: `base` at its first row (column) and r = 0, `count`
// rows (columns) there, `ld` elements from one row to the next (COL: from one
// r to the next). Gathered rows: row i of the tile is row rows[i] of base (below 0: any row, its outputs are not stored).
template <typename T>
struct Operand {
  const T* base;
  int64_t ld;
  int count;
  const int32_t* rows;
};

template <typename T, bool COL, int R, int NT, bool GATHER = false>
struct TileOf {
  typedef std::conditional_t<GATHER, int64_t, uint32_t> Off;   // a tile's elements stay within 2^32 of its base
  static constexpr int kBytes = R * kStep * 2;
  static constexpr int kChunks = R * kStep / 8;
  static constexpr int kPer = kChunks >= NT ? kChunks / NT : 1;   // chunks a thread brings in
  static constexpr int kRowChunks = COL ? R / 8 : kStep / 8;      // chunks of a stored row
  static_assert(kChunks % NT == 0 || NT % kChunks == 0, "chunks over threads");
  static_assert(!COL || R >= 64, "the swizzle of a column tile needs 8 chunks a row");

  __device__ static __forceinline__ int swizzle(int row) { return COL ? 2 * (row & 3) : row & 7; }

  // Chunk position i of the tile: r (within the step) and own index of its first element.
  __device__ static __forceinline__ void place(int i, int& r, int& own) {
    const int row = i / kRowChunks, c = 8 * ((i % kRowChunks) ^ swizzle(row));
    r = COL ? row : c;
    own = COL ? c : row;
  }
  // The thread's k-th chunk position (threads beyond the chunks repeat others').
  __device__ static __forceinline__ int position(int k) {
    return kChunks < NT ? threadIdx.x % kChunks : threadIdx.x + NT * k;
  }

  // Element offsets of the thread's chunks of a full step from the operand's
  // base. Rows past the operand's (and for DMA columns) repeat its last: they
  // make outputs that are not stored.
  template <bool DMA>
  __device__ static __forceinline__ void offsets(const Operand<T>& o, Off (&off)[kPer]) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      int r, own;
      place(position(k), r, own);
      if (COL) {
        if (DMA) own = min(own, o.count - 8);
        off[k] = (Off)r * (Off)o.ld + own;
      } else {
        own = min(own, o.count - 1);
        if constexpr (GATHER) own = max(o.rows[own], 0);
        off[k] = (Off)own * (Off)o.ld + r;
      }
    }
  }
  __device__ static __forceinline__ int64_t step_stride(const Operand<T>& o) { return COL ? kStep * o.ld : kStep; }

  __device__ static __forceinline__ void dma(const T* at, const Off (&off)[kPer], uint8_t* tile) {
    uint8_t* first = tile + 16 * 64 * __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % (kChunks < NT ? kChunks / 64 : NT / 64));
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(at + off[k]),
                                       (__attribute__((address_space(3))) void*)(first + 16 * NT * k), 16, 0, 0);
  }

  // The same through registers, at any alignment: r past `left` and columns
  // past the operand's are zero.
  __device__ static __forceinline__ void load(const Operand<T>& o, const T* at, const Off (&off)[kPer], int left,
                                              oct<T> (&v)[kPer]) {
    if (left >= kStep && (!COL || o.count >= R)) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) __builtin_memcpy(&v[k], at + off[k], 16);
      return;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      int r, own;
      place(position(k), r, own);
      v[k] = load_oct(at + off[k], COL ? (r < left ? o.count - own : 0) : left - r);
    }
  }
  __device__ static __forceinline__ void store(const oct<T> (&v)[kPer], uint8_t* tile) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) *reinterpret_cast<oct<T>*>(tile + 16 * position(k)) = v[k];
  }

  // The MFMA operand of the 16 rows (columns) from `own`, r = 32 kk + 8 * (lane / 16) + 0..7.
  __device__ static __forceinline__ oct<T> operand(const uint8_t* tile, int own, int kk, int lane) {
    if constexpr (!COL) {
      const int row = own + (lane & 15);
      return *reinterpret_cast<const oct<T>*>(tile + 16 * (row * kRowChunks + ((4 * kk + (lane >> 4)) ^ (row & 7))));
    } else {
      const int r = 32 * kk + 8 * (lane >> 4) + ((lane & 15) >> 2), col = own + 4 * (lane & 3);
      const uint8_t* p = tile + 16 * (r * kRowChunks + ((col >> 3) ^ swizzle(r))) + 2 * (col & 7);
      // r and r + 4 have the same swizzle
      struct { s16x4 lo, hi; } v;
      v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_tr_t)p);
      v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_tr_t)(p + 4 * 16 * kRowChunks));
      return __builtin_bit_cast(oct<T>, v);
    }
  }
};

// Every wave is past its reads of LDS, and its writes are there.
__device__ __forceinline__ void lds_barrier() {
  wait_lgkm0();
  block_sync_lds();
}

// Waits until at most N * `steps` of this wave's loads are in flight (steps <= MAX).
template <int N, int MAX>
__device__ __forceinline__ void wait_steps(int steps) {
  if constexpr (MAX > 0) {
    if (steps < MAX) return wait_steps<N, MAX - 1>(steps);
  }
  wait_vmcnt<N * MAX>();
}

// WP x WQ waves of BP/WP x BQ/WQ outputs each; ST slots of one step in LDS.
// DMA: 16-byte aligned rows, brought into LDS directly; otherwise through registers, any alignment.
template <typename T, bool PCOL, bool QCOL, int BP, int BQ, int WP, int WQ, int ST, bool DMA, bool GATHER = false>
struct Gemm {
  static constexpr int NT = 64 * WP * WQ;
  typedef TileOf<T, PCOL, BP, NT> PT;
  typedef TileOf<T, QCOL, BQ, NT, GATHER> QT;
  static constexpr int kSlots = DMA ? ST : 2;
  static constexpr int kSlot = PT::kBytes + QT::kBytes;
  static constexpr int kLds = kSlots * kSlot;
  static constexpr int kP = BP, kQ = BQ;
  static constexpr int NP = BP / WP / 16, NQ = BQ / WQ / 16;
  typedef f32x4 Acc[NP][NQ];

  __device__ static __forceinline__ int wave_p() { return (threadIdx.x >> 6) % WP * (BP / WP); }
  __device__ static __forceinline__ int wave_q() { return (threadIdx.x >> 6) / WP * (BQ / WQ); }

  __device__ static __forceinline__ void compute(const uint8_t* slot, Acc& acc) {
    const int lane = threadIdx.x & 63, p0 = wave_p(), q0 = wave_q();
#pragma unroll
    for (int kk = 0; kk < kStep / 32; ++kk) {
      oct<T> pv[NP], qv[NQ];
#pragma unroll
      for (int j = 0; j < NQ; ++j) qv[j] = QT::operand(slot + PT::kBytes, q0 + 16 * j, kk, lane);
#pragma unroll
      for (int i = 0; i < NP; ++i) pv[i] = PT::operand(slot, p0 + 16 * i, kk, lane);
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < NQ; ++j) acc[i][j] = mfma16(pv[i], qv[j], acc[i][j]);
    }
  }

  // One step of the products of tile rows q whose bit is set in `some` (bit j: the j-th 16 rows of the tile).
  __device__ static __forceinline__ void compute_some(const uint8_t* ptile, const uint8_t* qtile, uint32_t some, Acc& acc) {
    const int lane = threadIdx.x & 63, p0 = wave_p(), q0 = wave_q();
    some >>= __builtin_amdgcn_readfirstlane(q0 / 16);
#pragma unroll
    for (int kk = 0; kk < kStep / 32; ++kk) {
      oct<T> pv[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) pv[i] = PT::operand(ptile, p0 + 16 * i, kk, lane);
#pragma unroll
      for (int j = 0; j < NQ; ++j) {
        if (!(some >> j & 1)) continue;
        const oct<T> qv = QT::operand(qtile, q0 + 16 * j, kk, lane);
#pragma unroll
        for (int i = 0; i < NP; ++i) acc[i][j] = mfma16(pv[i], qv, acc[i][j]);
      }
    }
  }

  // Adds the sum over r < red. LDS is free for other use after a barrier.
  __device__ static __forceinline__ void run(const Operand<T>& p, const Operand<T>& q, int red, uint8_t* lds,
                                             Acc& acc) {
    const int64_t ps = PT::step_stride(p), qs = QT::step_stride(q);
    typename PT::Off po[PT::kPer];
    typename QT::Off qo[QT::kPer];
    PT::template offsets<DMA>(p, po);
    QT::template offsets<DMA>(q, qo);
    if constexpr (DMA) {
      const int nk = red / kStep, tail = red % kStep;
      constexpr int kPer = PT::kPer + QT::kPer;
      const T *pat = p.base, *qat = q.base;
      auto issue = [&](uint8_t* slot) {
        PT::dma(pat, po, slot);
        QT::dma(qat, qo, slot + PT::kBytes);
        pat += ps;
        qat += qs;
      };
      uint8_t* const end = lds + kLds;
#pragma unroll
      for (int s = 0; s < ST - 1; ++s)
        if (s < nk) issue(lds + s * kSlot);
      uint8_t *get = lds, *put = end - kSlot;
      if (tail) {   // the last, partial step first, in the slot that the ring needs last
        oct<T> pv[PT::kPer], qv[QT::kPer];
        PT::load(p, p.base + nk * ps, po, tail, pv);
        QT::load(q, q.base + nk * qs, qo, tail, qv);
        PT::store(pv, put);
        QT::store(qv, put + PT::kBytes);
        lds_barrier();
        compute(put, acc);
      }
#pragma unroll 1
      for (int s = 0; s < nk; ++s) {
        wait_steps<kPer, ST - 2>(nk - 1 - s);   // step s is in; later ones may be in flight
        lds_barrier();                          // for every wave; and all are done with step s - 1
        if (s + ST - 1 < nk) issue(put);
        compute(get, acc);
        get = get + kSlot == end ? lds : get + kSlot;
        put = put + kSlot == end ? lds : put + kSlot;
      }
    } else {
      const int nk = (red + kStep - 1) / kStep;
      oct<T> pv[PT::kPer], qv[QT::kPer];
      const T *pat = p.base, *qat = q.base;
      auto load = [&](int s) {
        PT::load(p, pat, po, red - s * kStep, pv);
        QT::load(q, qat, qo, red - s * kStep, qv);
        pat += ps;
        qat += qs;
      };
      auto store = [&](int s) {
        uint8_t* slot = lds + (s & 1) * kSlot;
        PT::store(pv, slot);
        QT::store(qv, slot + PT::kBytes);
      };
      if (nk > 0) {
        load(0);
        store(0);
      }
#pragma unroll 1
      for (int s = 0; s < nk; ++s) {
        lds_barrier();   // step s is there, and all are done with step s - 1
        if (s + 1 < nk) load(s + 1);
        compute(lds + (s & 1) * kSlot, acc);
        if (s + 1 < nk) store(s + 1);
      }
    }
  }

  // Writes the tile's first `pn` outputs of each row at `out` (type f32 or T),
  // rows `ld` apart; row(q) is the place of tile row q (below 0: not stored).
  template <typename Row>
  __device__ static __forceinline__ void store(const Acc& acc, void* out, bool f32, int64_t ld, int pn, Row&& row) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      const int64_t q = row(wave_q() + 16 * j + (lane & 15));
      if (q < 0) continue;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int p = wave_p() + 16 * i + 4 * (lane >> 4);
        if (f32) store_quad((float*)out + q * ld + p, acc[i][j], pn - p);
        else store_quad((T*)out + q * ld + p, acc[i][j], pn - p);
      }
    }
  }

  // The first n of four outputs, rounded to nearest even in U.
  template <typename U>
  __device__ static __forceinline__ void store_quad(U* at, f32x4 f, int n) {
    typedef U quad __attribute__((ext_vector_type(4)));
    const quad v = __builtin_convertvector(f, quad);
    if (n >= 4) {
      __builtin_memcpy(at, &v, sizeof(v));
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) at[i] = v[i];
    }
  }
};

// Workgroup b of n -> a place in an order in which neighbours share operands:
// consecutive workgroups go to consecutive XCDs, so each XCD takes a contiguous
// eighth of the order and finds the shared operands in its own L2.
__device__ __forceinline__ int64_t xcd_order(int64_t b, int64_t n) {
  const int64_t per = (n + 7) / 8;
  return b / 8 < per ? (b % 8) * per + b / 8 : n;
}

// Place l of an order over n_rt row tiles x np column tiles: 8 row tiles that
// share a column tile after one another, then the next column tile.
__device__ __forceinline__ void tile_at(int64_t l, int n_rt, int np, int& rt, int& pt) {
  constexpr int kSuper = 8;
  const int sup = (int)(l / (kSuper * np)), in = (int)(l - (int64_t)sup * kSuper * np);
  const int wide = max(min(kSuper, n_rt - kSuper * sup), 1);
  rt = kSuper * sup + in % wide;
  pt = in / wide;
}

// The wave's inclusive prefix sums.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    const int o = __shfl_up(v, s);
    if (lane >= s) v += o;
  }
  return v;
}

// Rows that can be brought into LDS 16 bytes at a time.
inline bool rows16(const void* p, int64_t stride) { return ((uintptr_t)p & 15) == 0 && stride % 8 == 0; }

// `blocks` workgroups of Kernel with `lds` bytes of dynamic LDS.
template <auto Kernel, typename... A>
int launch_tiles(const char* what, dim3 blocks, int threads, int lds, hipStream_t s, A... args) {
  static const hipError_t attr = hipFuncSetAttribute((const void*)Kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (attr != hipSuccess) return hip_fail(attr, what);
  Kernel<<<blocks, dim3(threads), lds, s>>>(args...);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MOE_OK : hip_fail(e, what);
}

// Workgroups for `tiles` tiles placed by xcd_order (whole rounds of the XCDs), or 0 where one launch cannot have them.
inline int64_t tile_blocks(int64_t tiles, int threads) {
  const int64_t blocks = (tiles + 7) / 8 * 8;
  return blocks * threads < (int64_t)1 << 32 ? blocks : 0;
}

}  // namespace moe
