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
//
// What keeps the matrix instructions fed: loads into LDS that no compiler wait
// stands behind, one barrier a step, and the operands of one half step read
// while the products of the half before run (in place of a wait for all loads
// in every step: 128 x 128 tiles went from 648 to 830 TFLOP/s on 16384 rows
// over 32 groups of 4096 x 2048). No LDS bank conflicts by the counters.
#pragma once

#include <type_traits>

#include "moe_element.h"
#include "moe_internal.h"
#include "moe_kquant.h"
#include "moe_once.h"
#include "moe_wave.h"

namespace moe {

constexpr int kStep = 64;   // r per step

typedef float f32x4 __attribute__((ext_vector_type(4)));
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
// r to the next). `room`: the stored rows that this tile is part of (COL: the
// tile's r lie along several) have 8 elements or more. Gathered rows: row i of the tile is row rows[i] of base (below 0: any row, its outputs are not stored).
template <typename T>
struct Operand {
  const T* base;
  int64_t ld;
  int count;
  const int32_t* rows;
  bool room;
};

template <typename T, bool COL, int R, int NT, bool GATHER = false>
struct TileOf {
  typedef std::conditional_t<GATHER, int64_t, uint32_t> Off;   // a tile's elements stay within 2^31 of its base
  static constexpr int kBytes = R * kStep * 2;
  static constexpr int kChunks = R * kStep / 8;
  static constexpr int kPer = kChunks >= NT ? kChunks / NT : 1;   // chunks a thread brings in
  static constexpr int kRowChunks = COL ? R / 8 : kStep / 8;      // chunks of a stored row
  static_assert(kChunks % NT == 0 || NT % kChunks == 0, "chunks over threads");
  static_assert(!COL || R >= 64, "the swizzle of a column tile needs 8 chunks a row");

  // A transposing read takes four rows of 32 bytes for each quarter of the wave, the quarters 8 rows apart.
  // Rows of 256 bytes and more all start at LDS bank 0: 8 swizzles keep the 8 rows of half a wave apart (4 where a row has 8 chunks only).
  __device__ static __forceinline__ int swizzle(int row) {
    return !COL ? row & 7 : kRowChunks >= 16 ? 2 * ((row & 3) | (row >> 1 & 4)) : 2 * (row & 3);
  }

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

  // `at` is the same in every lane. The compiler does not see these writes of
  // LDS: it would wait for all of them before any later LDS read. The waits
  // are the caller's. (m0 is declared as changed; nothing else in these kernels holds a value there.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  __device__ static __forceinline__ void dma(const T* at, const Off (&off)[kPer], uint32_t tile) {
    const uint32_t first = tile + 16 * 64 * __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % (kChunks < NT ? kChunks / 64 : NT / 64));
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if constexpr (GATHER)
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                     : : "v"(at + off[k]), "s"(first + 16 * NT * k) : "memory", "m0");
      else
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                     : : "v"(2 * off[k]), "s"(at), "s"(first + 16 * NT * k) : "memory", "m0");
    }
  }

#pragma clang diagnostic pop

  // COL: a last step of `left` r: the rows past it repeat the last one, until clear() zeroes them in LDS.
  __device__ static __forceinline__ void dma_part(const Operand<T>& o, const T* at, int left, uint32_t tile) {
    static_assert(COL, "a partial step of a column tile is whole rows");
    Off off[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      int r, own;
      place(position(k), r, own);
      off[k] = (Off)min(r, left - 1) * (Off)o.ld + min(own, o.count - 8);
    }
    dma(at, off, tile);
  }
  __device__ static __forceinline__ void clear(int left, uint8_t* tile) {
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (position(k) / kRowChunks >= left) *reinterpret_cast<oct<T>*>(tile + 16 * position(k)) = oct<T>{};
  }

  // The same through registers, at any alignment: r past `left` and columns
  // past the operand's are zero.
  __device__ static __forceinline__ bool whole(const Operand<T>& o, int left) {
    return left >= kStep && (!COL || o.count >= R);
  }
  __device__ static __forceinline__ int there(const Operand<T>& o, int k, int left) {   // of the thread's k-th chunk
    int r, own;
    place(position(k), r, own);
    return COL ? (r < left ? o.count - own : 0) : left - r;
  }
  __device__ static __forceinline__ void load(const Operand<T>& o, const T* at, const Off (&off)[kPer], int left,
                                              oct<T> (&v)[kPer]) {
    if (whole(o, left)) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) __builtin_memcpy(&v[k], at + off[k], 16);
    } else if (o.room) {
      // Every lane loads, where its chunk is not there the row's last elements (or the last row's): without a
      // branch the loads need not be waited for one by one. store() puts them in place.
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        int r, own;
        place(position(k), r, own);
        const int64_t e = COL ? min(r, left - 1) * o.ld + min(own, o.count - 8) : (int64_t)off[k] - r + min(r, left - 8);
        __builtin_memcpy(&v[k], at + e, 16);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[k] = raw_oct(at + off[k], there(o, k, left), false);
    }
  }
  __device__ static __forceinline__ void store(const Operand<T>& o, int left, const oct<T> (&v)[kPer], uint8_t* tile) {
    if (whole(o, left)) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) *reinterpret_cast<oct<T>*>(tile + 16 * position(k)) = v[k];
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        *reinterpret_cast<oct<T>*>(tile + 16 * position(k)) = placed_oct<T>(v[k], there(o, k, left), o.room);
    }
  }

  // The MFMA operand of the 16 rows (columns) from `own`, r = 32 kk + 8 * (lane / 16) + 0..7.
  __device__ static __forceinline__ oct<T> operand(const uint8_t* tile, int own, int kk, int lane) {
    if constexpr (!COL) {
      const int row = own + (lane & 15);
      return *reinterpret_cast<const oct<T>*>(tile + 16 * (row * kRowChunks + ((4 * kk + (lane >> 4)) ^ swizzle(row))));
    } else {
      const int r = 32 * kk + 8 * (lane >> 4) + ((lane & 15) >> 2), col = own + 4 * (lane & 3);
      const uint8_t* p = tile + 16 * (r * kRowChunks + ((col >> 3) ^ swizzle(r))) + 2 * (col & 7);
      // (r and r + 4 have the same swizzle)
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

// The same pointer in every lane, as a scalar.
template <typename T>
__device__ __forceinline__ const T* uniform(const T* p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (const T*)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ uint32_t lds_offset(const uint8_t* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)p;
}

// Waits until at most N * `steps` (steps <= MAX) + MORE of this wave's loads and stores are in flight.
template <int N, int MAX, int MORE = 0>
__device__ __forceinline__ void wait_steps(int steps) {
  if constexpr (MAX > 0) {
    if (steps < MAX) return wait_steps<N, MAX - 1, MORE>(steps);
  }
  wait_vmcnt<N * MAX + MORE>();
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
  static constexpr int kStores = NP * NQ;   // store instructions of a wave's whole part of a tile

  __device__ static __forceinline__ int wave_p() { return (threadIdx.x >> 6) % WP * (BP / WP); }
  __device__ static __forceinline__ int wave_q() { return (threadIdx.x >> 6) / WP * (BQ / WQ); }

  // The MFMA operands of 32 r, and their products.
  struct Half {
    oct<T> p[NP], q[NQ];
  };
  __device__ static __forceinline__ void read(const uint8_t* slot, int kk, Half& h) {
    const int lane = threadIdx.x & 63, p0 = wave_p(), q0 = wave_q();
#pragma unroll
    for (int j = 0; j < NQ; ++j) h.q[j] = QT::operand(slot + PT::kBytes, q0 + 16 * j, kk, lane);
#pragma unroll
    for (int i = 0; i < NP; ++i) h.p[i] = PT::operand(slot, p0 + 16 * i, kk, lane);
  }
  __device__ static __forceinline__ void multiply(const Half& h, Acc& acc) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int j = 0; j < NQ; ++j) acc[i][j] = mfma16(h.p[i], h.q[j], acc[i][j]);
  }
  // Places the reads of one half step evenly among the first products of the half before.
  __device__ static __forceinline__ void interleave() {
    constexpr int kReads = NP * (PCOL ? 2 : 1) + NQ * (QCOL ? 2 : 1), kProducts = NP * NQ;
    constexpr int kEach = (2 * kReads + kProducts - 1) / kProducts;
#pragma unroll
    for (int i = 0; i < kProducts; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, kEach, 0);   // LDS reads
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);       // a product
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  __device__ static __forceinline__ void compute(const uint8_t* slot, Acc& acc) {
    Half h;
#pragma unroll
    for (int kk = 0; kk < kStep / 32; ++kk) {
      read(slot, kk, h);
      multiply(h, acc);
    }
  }

  // One step of the products of the wave's j-th 16 tile rows q, whose operand is the sum of `PIECES` tiles.
  template <int PIECES>
  __device__ static __forceinline__ void multiply_row(const uint8_t* ptile, const uint8_t* qtiles, int j, f32x4 (&acc)[NP]) {
    const int lane = threadIdx.x & 63, p0 = wave_p(), q0 = wave_q();
#pragma unroll
    for (int kk = 0; kk < kStep / 32; ++kk) {
      oct<T> pv[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) pv[i] = PT::operand(ptile, p0 + 16 * i, kk, lane);
#pragma unroll
      for (int n = 0; n < PIECES; ++n) {
        const oct<T> qv = QT::operand(qtiles + n * QT::kBytes, q0 + 16 * j, kk, lane);
#pragma unroll
        for (int i = 0; i < NP; ++i) acc[i] = mfma16(pv[i], qv, acc[i]);
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
      const T *pat = uniform(p.base), *qat = uniform(q.base);
      auto issue = [&](const uint8_t* slot) {
        const uint32_t at = lds_offset(slot);
        PT::dma(pat, po, at);
        QT::dma(qat, qo, at + PT::kBytes);
        pat += ps;
        qat += qs;
      };
      uint8_t* const end = lds + kLds;
#pragma unroll
      for (int s = 0; s < ST - 1; ++s)
        if (s < nk) issue(lds + s * kSlot);
      if (tail) {   // the last, partial step first, in the slot that the ring needs last
        uint8_t* const put = end - kSlot;
        oct<T> pv[PT::kPer], qv[QT::kPer];
        PT::load(p, p.base + nk * ps, po, tail, pv);
        QT::load(q, q.base + nk * qs, qo, tail, qv);
        PT::store(p, tail, pv, put);
        QT::store(q, tail, qv, put + PT::kBytes);
        lds_barrier();
        compute(put, acc);
        lds_barrier();
      }
      if (nk == 0) return;
      if (ST - 1 < nk) issue(end - kSlot);
      // The operands of one half step are read while the products of the half
      // before run; a slot is free, and filled with the step ST later, as soon as every wave has read its second half.
      Half h0, h1;
      wait_steps<kPer, ST - 1>(nk - 1);
      lds_barrier();
      read(lds, 0, h0);
      const uint8_t* get = lds;
      int s = 0;
#pragma unroll 1
      for (; s < nk - ST; ++s) {
        read(get, 1, h1);
        multiply(h0, acc);
        interleave();
        wait_vmcnt<kPer * (ST - 2)>();   // step s + 1 is in; later ones may be in flight
        lds_barrier();                   // for every wave; and all have read step s
        issue(get);
        get = get + kSlot == end ? lds : get + kSlot;
        read(get, 0, h0);
        multiply(h1, acc);
        interleave();
      }
#pragma unroll 1
      for (; s < nk - 1; ++s) {
        read(get, 1, h1);
        multiply(h0, acc);
        interleave();
        wait_steps<kPer, ST - 2>(nk - 2 - s);
        lds_barrier();
        get = get + kSlot == end ? lds : get + kSlot;
        read(get, 0, h0);
        multiply(h1, acc);
        interleave();
      }
      read(get, 1, h1);
      multiply(h0, acc);
      multiply(h1, acc);
    } else {
      const int nk = (red + kStep - 1) / kStep;
      struct Stage {
        oct<T> p[PT::kPer], q[QT::kPer];
      };
      const T *pat = p.base, *qat = q.base;
      auto load = [&](int s, Stage& g) {
        PT::load(p, pat, po, red - s * kStep, g.p);
        QT::load(q, qat, qo, red - s * kStep, g.q);
        pat += ps;
        qat += qs;
      };
      auto store = [&](int s, const Stage& g) {
        uint8_t* slot = lds + (s & 1) * kSlot;
        PT::store(p, red - s * kStep, g.p, slot);
        QT::store(q, red - s * kStep, g.q, slot + PT::kBytes);
      };
      if (nk == 0) return;
      if constexpr (PT::kPer + QT::kPer <= 6) {   // two steps on their way, where the registers hold them
        Stage g0, g1;
        load(0, g0);
        if (nk > 1) load(1, g1);
        store(0, g0);
#pragma unroll 1
        for (int s = 0;; s += 2) {
          lds_barrier();   // step s is there, and all are done with step s - 1
          if (s + 2 < nk) load(s + 2, g0);
          compute(lds, acc);
          if (s + 1 == nk) break;
          store(s + 1, g1);
          lds_barrier();
          if (s + 3 < nk) load(s + 3, g1);
          compute(lds + kSlot, acc);
          if (s + 2 == nk) break;
          store(s + 2, g0);
        }
      } else {
        Stage g;
        load(0, g);
        store(0, g);
#pragma unroll 1
        for (int s = 0; s < nk; ++s) {
          lds_barrier();   // step s is there, and all are done with step s - 1
          if (s + 1 < nk) load(s + 1, g);
          compute(lds + (s & 1) * kSlot, acc);
          if (s + 1 < nk) store(s + 1, g);
        }
      }
    }
  }

  // The same as a stream of tiles without a pause between them (DMA, both
  // operands in columns): the slots that a tile's last steps leave take the next
  // tile's first ones, so that they arrive while the tile is finished and stored.
  struct Ring {
    uint8_t* lds;
    Operand<T> p, q;   // the tile whose steps are asked for
    int red, issued;   // its sum's length, and its steps asked for so far
    int get, put;      // slots of the next step to use and of the next one asked for
    int arrived;       // 1: its first step has been waited for
    int stores;        // store instructions of the tile before, issued after this tile's first steps
    typename PT::Off po[PT::kPer];
    typename QT::Off qo[QT::kPer];

    __device__ __forceinline__ explicit Ring(uint8_t* lds) : lds(lds), get(0), put(0), stores(0) {}
    __device__ __forceinline__ void start(const Operand<T>& p_, const Operand<T>& q_, int red_) {
      p = p_;
      q = q_;
      p.base = uniform(p.base);
      q.base = uniform(q.base);
      red = red_;
      issued = 0;
      arrived = 0;
      PT::template offsets<true>(p, po);
      QT::template offsets<true>(q, qo);
    }
    __device__ __forceinline__ int steps() const { return (red + kStep - 1) / kStep; }
    __device__ __forceinline__ void issue() {
      const uint32_t at = lds_offset(lds) + put * kSlot;
      const int left = red - kStep * issued;
      const T *pat = p.base + issued * PT::step_stride(p), *qat = q.base + issued * QT::step_stride(q);
      if (left >= kStep) {
        PT::dma(pat, po, at);
        QT::dma(qat, qo, at + PT::kBytes);
      } else {
        PT::dma_part(p, pat, left, at);
        QT::dma_part(q, qat, left, at + PT::kBytes);
      }
      ++issued;
      put = put + 1 == ST ? 0 : put + 1;
    }
    __device__ __forceinline__ void fill() {
      while (issued < ST && issued < steps()) issue();
    }
  };
  // Adds the sums of the ring's tile; next() starts the ring on the tile after
  // it and says whether there is one. Every wave is past its reads of LDS at the end.
  template <typename Next>
  __device__ static __forceinline__ int run_on(Ring& ring, Acc& acc, Next&& next) {
    constexpr int kPer = PT::kPer + QT::kPer;
    const int red = ring.red, nk = ring.steps(), tail = red % kStep;
    int over = 0, more = 0;
    auto advance = [&] {
      ring.get = ring.get + 1 == ST ? 0 : ring.get + 1;
    };
    auto slot = [&] { return ring.lds + ring.get * kSlot; };
    auto clear = [&](int s) {   // the partial last step
      if (s + 1 < nk || !tail) return;
      PT::clear(tail, slot());
      QT::clear(tail, slot() + PT::kBytes);
      lds_barrier();
    };
    // Loads and stores complete in the order of their issue. The steps that were
    // asked for before the last tile's stores do not wait for them; later ones do.
    const int before = ring.stores ? ring.issued : 0;
    ring.fill();
    if (nk > 0) {
      Half h0, h1;
      if (!ring.arrived) wait_steps<kPer, ST - 1>(ring.issued - 1);
      lds_barrier();
      clear(0);
      read(slot(), 0, h0);
      int s = 0;
      const T *pat = ring.p.base + ring.issued * PT::step_stride(ring.p);
      const T *qat = ring.q.base + ring.issued * QT::step_stride(ring.q);
#pragma unroll 1
      for (; ring.issued < red / kStep; ++s) {   // whole steps to ask for
        read(slot(), 1, h1);
        multiply(h0, acc);
        interleave();
        if (s + 1 < before) wait_vmcnt<kPer * (ST - 2) + kStores>();   // step s + 1 is in
        else wait_vmcnt<kPer * (ST - 2)>();
        lds_barrier();                                                 // for every wave; and all have read step s
        const uint32_t at = lds_offset(slot());   // (ST steps are on their way: the one asked for next takes this slot)
        PT::dma(pat, ring.po, at);
        QT::dma(qat, ring.qo, at + PT::kBytes);
        pat += PT::step_stride(ring.p);
        qat += QT::step_stride(ring.q);
        ++ring.issued;
        advance();
        read(slot(), 0, h0);
        multiply(h1, acc);
        interleave();
      }
      ring.put = (ring.get + ring.issued - s) % ST;
#pragma unroll 1
      for (; s < nk - 1; ++s) {
        read(slot(), 1, h1);
        multiply(h0, acc);
        interleave();
        const int flying = !over ? ring.issued - 2 - s : nk - 2 - s + (more ? ring.issued : 0);
        if (s + 1 < before) wait_steps<kPer, ST - 2, kStores>(flying);   // step s + 1 is in
        else wait_steps<kPer, ST - 2>(flying);
        lds_barrier();   // for every wave; and all have read step s
        if (!over && ring.issued == nk) {
          over = 1;
          more = next();
        }
        if (over ? more && ring.issued < ring.steps() : true) ring.issue();
        advance();
        clear(s + 1);
        read(slot(), 0, h0);
        multiply(h1, acc);
        interleave();
      }
      read(slot(), 1, h1);
      multiply(h0, acc);
      multiply(h1, acc);
      advance();
      lds_barrier();
    }
    if (!over) more = next();
    if (more) {
      ring.fill();
      if (ring.issued > 0) {   // before the stores, which would be waited for too
        wait_steps<kPer, ST - 1>(ring.issued - 1);
        ring.arrived = 1;
      }
    }
    return more;
  }

  // Writes the tile's first `pn` outputs of each row at `out` (type f32 or T),
  // rows `ld` apart; row(q) is the place of tile row q (below 0: not stored).
  template <typename Row>
  __device__ static __forceinline__ void store(const Acc& acc, void* out, bool f32, int64_t ld, int pn, Row&& row) {
    if (f32) store_to(acc, (float*)out, ld, pn, row);
    else store_to(acc, (T*)out, ld, pn, row);
  }
  template <typename U, typename Row>
  __device__ static __forceinline__ void store_to(const Acc& acc, U* out, int64_t ld, int pn, Row& row) {
    if constexpr (NP % 2 == 0) {
      if (pn >= BP) return store_whole(acc, out, ld, row);
    }
    store_part(acc, out, ld, pn, row);
  }
  template <typename U, typename Row>
  __device__ static __forceinline__ void store_part(const Acc& acc, U* out, int64_t ld, int pn, Row& row) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      const int64_t q = row(wave_q() + 16 * j + (lane & 15));
      if (q < 0) continue;
      const int p = wave_p() + 4 * (lane >> 4);
#pragma unroll
      for (int i = 0; i < NP; ++i) store_quad(out + q * ld + p + 16 * i, acc[i][j], pn - p - 16 * i);
    }
  }
  // Lanes q and q + 8 of 16 exchange a quad, so that a store writes 32
  // neighbouring outputs of 8 rows instead of 16 of 16 rows.
  template <typename U, typename Row>
  __device__ static __forceinline__ void store_whole(const Acc& acc, U* out, int64_t ld, Row& row) {
    const int lane = threadIdx.x & 63, upper = lane >> 3 & 1;
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      const int64_t qa = row(wave_q() + 16 * j + (lane & 7)), qb = row(wave_q() + 16 * j + 8 + (lane & 7));
      U* const at = out + wave_p() + 16 * upper + 4 * (lane >> 4);
#pragma unroll
      for (int i = 0; i < NP; i += 2) {
        f32x4 a = acc[i][j], b = acc[i + 1][j], x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = dpp_f32<kDppRor8>(upper ? a[e] : b[e]);
          a[e] = upper ? x[e] : a[e];
          b[e] = upper ? b[e] : x[e];
        }
        if (qa >= 0) store_quad(at + qa * ld + 16 * i, a, 4);
        if (qb >= 0) store_quad(at + qb * ld + 16 * i, b, 4);
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

// The wave's inclusive prefix sums: within 16 lanes by shifts, then the last
// lane of each 16 (and of the lower 32) to those above. All lanes take part.
__device__ __forceinline__ int wave_scan(int v, int lane) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);   // row_shr:8
  const int a = __builtin_amdgcn_readlane(v, 15), b = __builtin_amdgcn_readlane(v, 31), c = __builtin_amdgcn_readlane(v, 47);
  return v + (lane < 16 ? 0 : lane < 32 ? a : lane < 48 ? a + b : a + b + c);
}

// Rows that can be brought into LDS 16 bytes at a time.
inline bool rows16(const void* p, int64_t stride) { return ((uintptr_t)p & 15) == 0 && stride % 8 == 0; }

// `blocks` workgroups of Kernel with `lds` bytes of dynamic LDS.
template <auto Kernel, typename... A>
int launch_tiles(const char* what, dim3 blocks, int threads, int lds, hipStream_t s, A... args) {
  static OncePerDevice attr;   // (a kernel's dynamic LDS is the same in every call)
  int device = 0;
  hipError_t e = hipGetDevice(&device);
  if (e == hipSuccess)
    e = attr(device, [&] { return hipFuncSetAttribute((const void*)Kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds); });
  if (e != hipSuccess) return hip_fail(e, what);
  Kernel<<<blocks, dim3(threads), lds, s>>>(args...);
  e = hipGetLastError();
  return e == hipSuccess ? MOE_OK : hip_fail(e, what);
}

// Workgroups for `tiles` tiles placed by xcd_order (whole rounds of the XCDs), or 0 where one launch cannot have them.
inline int64_t tile_blocks(int64_t tiles, int threads) {
  const int64_t blocks = (tiles + 7) / 8 * 8;
  return blocks * threads < (int64_t)1 << 32 ? blocks : 0;
}

}  // namespace moe
