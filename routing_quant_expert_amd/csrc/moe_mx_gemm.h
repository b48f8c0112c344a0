// The tile product of moe_gemm.h for operands in microscaled 4-bit floats, on
// v_mfma_scale_f32_16x16x128_f8f6f4 (e2m1 elements, one e8m0 scale for 32 of a
// row, f32 sums).
//
// A step is 256 elements: 128 bytes of a row, staged in LDS in the same
// 16-byte chunks and with the same swizzle as 64 16-bit elements, so that both
// kinds of product ask the same of memory and LDS while this one multiplies
// four times as much. A chunk is one block of 32 elements. The sum does not
// depend on the order of the blocks: lane group q of 4 takes blocks 2 q and
// 2 q + 1 of the step in its two products, whose scales then lie next to each
// other (one 16-bit read; the instruction selects the byte).
#pragma once

#include "moe_gemm.h"

namespace moe {

constexpr int kMxStep = 256;   // elements of a step
constexpr int kMxBlock = 32;   // elements of a scale

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// C += A B of the lane's 32 elements each; byte KK of the scales.
template <int KK>
__device__ __forceinline__ f32x4 mfma_mx(i32x4 a, i32x4 b, f32x4 c, int sa, int sb) {
  constexpr int kFp4 = 4;
  const i32x8 a8 = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 b8 = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, kFp4, kFp4, KK, sa, KK, sb);
}

// The rows of a tile: `count` of them, codes `ld` and scales `scale_ld` bytes apart. Of a pair of matrices (as kRowPairs)
// the second one's codes and scales are `then` and `scales_then` bytes further.
struct MxOperand {
  const uint8_t *codes, *scales;
  int64_t ld, scale_ld;
  int count;
  int64_t then = 0, scales_then = 0;
};

// The first n (at most 16; below 1: none) of 16 bytes at p, the others 0. room: 16 bytes end at p + n.
__device__ __forceinline__ i32x4 bytes16(const uint8_t* p, int n, bool room) {
  unsigned __int128 v = 0;
  if (n >= 16) {
    __builtin_memcpy(&v, p, 16);
  } else if (n > 0) {
    if (room) {
      __builtin_memcpy(&v, p + n - 16, 16);
      v >>= 8 * (16 - n);
    } else {
#pragma unroll 1
      for (int i = 0; i < n; ++i) v |= (unsigned __int128)p[i] << (8 * i);
    }
  }
  return __builtin_bit_cast(i32x4, v);
}

template <int R, int NT, bool PAIRS>
struct MxTile {
  static constexpr int kCodes = R * 128;
  static constexpr int kChunks = R * 8;
  static constexpr int kPer = kChunks >= NT ? kChunks / NT : 1;   // chunks a thread brings in
  static constexpr int kWords = R * 2;                            // of 4 scales
  static constexpr int kWordsThere = kWords < 64 ? 64 : kWords;   // (a wave brings in 64; those past the rows' repeat the last row's)
  static constexpr int kBytes = kCodes + 4 * kWordsThere;
  static_assert(kChunks % NT == 0 || NT % kChunks == 0, "chunks over threads");
  static_assert(kWordsThere <= NT && NT % kWordsThere == 0, "one word of scales a thread");
  static_assert(!PAIRS || (NT % 256 == 0 && kChunks >= NT && kWords == NT), "a thread's chunks, and a wave's scales, are all of one matrix");

  __device__ static __forceinline__ int position(int k) { return kChunks < NT ? threadIdx.x % kChunks : threadIdx.x + NT * k; }
  __device__ static __forceinline__ int chunk(int i) { return i % 8 ^ (i / 8 & 7); }
  // The row of its matrix that tile row `row` is (the tile's last one for those past it).
  __device__ static __forceinline__ int own(const MxOperand& o, int row) {
    return min(PAIRS ? row / 32 * 16 + row % 16 : row, o.count - 1);
  }
  // Scales of a pair lie apart by matrix: those of the first in the first half.
  __device__ static __forceinline__ int scale_row(int row) { return PAIRS ? (row / 16 % 2) * (R / 2) + row / 32 * 16 + row % 16 : row; }
  __device__ static __forceinline__ int word() { return threadIdx.x % kWordsThere; }
  __device__ static __forceinline__ int word_row(const MxOperand& o) {
    const int row = min(word() / 2, R - 1);
    return min(PAIRS ? row % (R / 2) : row, o.count - 1);
  }

  __device__ static __forceinline__ const uint8_t* codes(const MxOperand& o) {
    return o.codes + (PAIRS && (threadIdx.x >> 7 & 1) ? o.then : 0);
  }
  __device__ static __forceinline__ const uint8_t* scales(const MxOperand& o) {
    return o.scales + (PAIRS && word() >= kWords / 2 ? o.scales_then : 0);
  }
  struct Offsets {
    uint32_t codes[kPer], scales;
  };
  __device__ static __forceinline__ void offsets(const MxOperand& o, Offsets& off) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) off.codes[k] = (uint32_t)own(o, position(k) / 8) * (uint32_t)o.ld + 16 * chunk(position(k));
    off.scales = (uint32_t)word_row(o) * (uint32_t)o.scale_ld + 4 * (word() & 1);
  }

  // (As TileOf::dma; `codes` and `scales` are the same in every lane.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  __device__ static __forceinline__ void dma(const uint8_t* codes, const uint8_t* scales, const Offsets& off, uint32_t tile) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t first = tile + 16 * 64 * (wave % (kChunks < NT ? kChunks / 64 : NT / 64));
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                   : : "v"(off.codes[k]), "s"(codes), "s"(first + 16 * NT * k) : "memory", "m0");
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
                 : : "v"(off.scales), "s"(scales), "s"(tile + kCodes + 4 * 64 * (wave % (kWordsThere / 64))) : "memory", "m0");
  }
#pragma clang diagnostic pop

  // The same through registers at any alignment; `left` elements of each row are there (fewer than a step: zeros follow),
  // `row_bytes` and `row_blocks` in a whole row.
  struct Stage {
    i32x4 codes[kPer];
    uint32_t scales;
  };
  __device__ static __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, const Offsets& off, int left,
                                              bool room, Stage& g) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int at = 16 * chunk(position(k));
      g.codes[k] = bytes16(codes + off.codes[k], (left + 1) / 2 - at, room);
      if (left & 1) {   // the half of the last byte past an odd row
        const int last = left / 2 - at;
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (last >= 4 * w && last < 4 * w + 4) g.codes[k][w] &= (16u << (8 * (last - 4 * w))) - 1;
      }
    }
    const int n = (left + kMxBlock - 1) / kMxBlock - 4 * (word() & 1);   // scales there
    uint32_t v = 0;
    if (n >= 4) {
      __builtin_memcpy(&v, scales + off.scales, 4);
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) v |= (uint32_t)scales[off.scales + i] << (8 * i);
    }
    g.scales = v;
  }
  __device__ static __forceinline__ void store(const Stage& g, uint8_t* tile) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) *reinterpret_cast<i32x4*>(tile + 16 * position(k)) = g.codes[k];
    *reinterpret_cast<uint32_t*>(tile + kCodes + 4 * word()) = g.scales;
  }

  // The lane's block and its two scales: row `own` + lane % 16, blocks 2 (lane / 16) + kk.
  __device__ static __forceinline__ i32x4 operand(const uint8_t* tile, int own, int kk, int lane) {
    const int row = own + (lane & 15);
    return *reinterpret_cast<const i32x4*>(tile + 128 * row + 16 * ((2 * (lane >> 4) + kk) ^ (row & 7)));
  }
  __device__ static __forceinline__ int scale(const uint8_t* tile, int own, int lane) {
    return *reinterpret_cast<const uint16_t*>(tile + kCodes + 8 * scale_row(own + (lane & 15)) + 2 * (lane >> 4));
  }
};

// DMA: codes 16-byte and scales 4-byte aligned, brought into LDS directly; otherwise through registers, any alignment.
template <int BP, int BQ, int WP, int WQ, int ST, bool DMA, bool PAIRS>
struct MxGemm : TileOut<BP, BQ, WP, WQ, PAIRS> {
  typedef TileOut<BP, BQ, WP, WQ, PAIRS> Out;
  using Out::NT, Out::NP, Out::NQ, Out::wave_p, Out::wave_q;
  typedef typename Out::Acc Acc;
  typedef MxTile<BP, NT, PAIRS> PT;
  typedef MxTile<BQ, NT, false> QT;
  static constexpr int kSlots = DMA ? ST : 2;
  static constexpr int kSlot = PT::kBytes + QT::kBytes;
  static constexpr int kLds = kSlots * kSlot;

  struct Half {
    i32x4 p[NP], q[NQ];
    int ps[NP], qs[NQ];
  };
  // kk = 0: with the step's scales, which the second half takes from `first`.
  template <int KK>
  __device__ static __forceinline__ void read(const uint8_t* slot, Half& h, const Half* first = nullptr) {
    const int lane = threadIdx.x & 63, p0 = wave_p(), q0 = wave_q();
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      h.q[j] = QT::operand(slot + PT::kBytes, q0 + 16 * j, KK, lane);
      h.qs[j] = KK ? first->qs[j] : QT::scale(slot + PT::kBytes, q0 + 16 * j, lane);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      h.p[i] = PT::operand(slot, p0 + 16 * i, KK, lane);
      h.ps[i] = KK ? first->ps[i] : PT::scale(slot, p0 + 16 * i, lane);
    }
  }
  template <int KK>
  __device__ static __forceinline__ void multiply(const Half& h, Acc& acc) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int j = 0; j < NQ; ++j) acc[i][j] = mfma_mx<KK>(h.p[i], h.q[j], acc[i][j], h.ps[i], h.qs[j]);
  }
  // Places `reads` LDS reads evenly among the first products of the half before.
  template <int READS>
  __device__ static __forceinline__ void interleave() {
    constexpr int kProducts = NP * NQ, kEach = (2 * READS + kProducts - 1) / kProducts;
#pragma unroll
    for (int i = 0; i < kProducts; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, kEach, 0);   // LDS reads
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);       // a product
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  __device__ static __forceinline__ void compute(const uint8_t* slot, Acc& acc) {
    Half h0, h1;
    read<0>(slot, h0);
    read<1>(slot, h1, &h0);
    multiply<0>(h0, acc);
    multiply<1>(h1, acc);
  }

  // Adds the sum over the k elements of the rows. LDS is free for other use after a barrier.
  __device__ static __forceinline__ void run(const MxOperand& p, const MxOperand& q, int k, uint8_t* lds, Acc& acc) {
    typename PT::Offsets po;
    typename QT::Offsets qo;
    PT::offsets(p, po);
    QT::offsets(q, qo);
    const bool room = k >= 32;
    struct Stage {
      typename PT::Stage p;
      typename QT::Stage q;
    };
    auto load = [&](int s, Stage& g) {
      PT::load(PT::codes(p) + 128 * (int64_t)s, PT::scales(p) + 8 * (int64_t)s, po, k - s * kMxStep, room, g.p);
      QT::load(QT::codes(q) + 128 * (int64_t)s, QT::scales(q) + 8 * (int64_t)s, qo, k - s * kMxStep, room, g.q);
    };
    auto store = [&](uint8_t* slot, const Stage& g) {
      PT::store(g.p, slot);
      QT::store(g.q, slot + PT::kBytes);
    };
    if constexpr (DMA) {
      const int nk = k / kMxStep;
      constexpr int kPer = PT::kPer + QT::kPer + 2;
      const uint8_t *pc = uniform(PT::codes(p)), *ps = uniform(PT::scales(p)), *qc = uniform(q.codes), *qs = uniform(q.scales);
      auto issue = [&](const uint8_t* slot) {
        const uint32_t at = lds_offset(slot);
        PT::dma(pc, ps, po, at);
        QT::dma(qc, qs, qo, at + PT::kBytes);
        pc += 128;
        qc += 128;
        ps += 8;
        qs += 8;
      };
      uint8_t* const end = lds + kLds;
#pragma unroll
      for (int s = 0; s < ST - 1; ++s)
        if (s < nk) issue(lds + s * kSlot);
      if (k % kMxStep) {   // the last, partial step first, in the slot that the ring needs last
        Stage g;
        load(nk, g);
        store(end - kSlot, g);
        lds_barrier();
        compute(end - kSlot, acc);
        lds_barrier();
      }
      if (nk == 0) return;
      if (ST - 1 < nk) issue(end - kSlot);
      // (as Gemm::run)
      Half h0, h1;
      wait_steps<kPer, ST - 1>(nk - 1);
      lds_barrier();
      read<0>(lds, h0);
      const uint8_t* get = lds;
      int s = 0;
#pragma unroll 1
      for (; s < nk - ST; ++s) {
        read<1>(get, h1, &h0);
        multiply<0>(h0, acc);
        interleave<NP + NQ>();
        wait_vmcnt<kPer * (ST - 2)>();   // step s + 1 is in; later ones may be in flight
        lds_barrier();                   // for every wave; and all have read step s
        issue(get);
        get = get + kSlot == end ? lds : get + kSlot;
        read<0>(get, h0);
        multiply<1>(h1, acc);
        interleave<2 * (NP + NQ)>();
      }
#pragma unroll 1
      for (; s < nk - 1; ++s) {
        read<1>(get, h1, &h0);
        multiply<0>(h0, acc);
        interleave<NP + NQ>();
        wait_steps<kPer, ST - 2>(nk - 2 - s);
        lds_barrier();
        get = get + kSlot == end ? lds : get + kSlot;
        read<0>(get, h0);
        multiply<1>(h1, acc);
        interleave<2 * (NP + NQ)>();
      }
      read<1>(get, h1, &h0);
      multiply<0>(h0, acc);
      multiply<1>(h1, acc);
    } else {
      const int nk = (k + kMxStep - 1) / kMxStep;
      if (nk == 0) return;
      Stage g;
      load(0, g);
      store(lds, g);
#pragma unroll 1
      for (int s = 0; s < nk; ++s) {
        lds_barrier();   // step s is there, and all are done with step s - 1
        if (s + 1 < nk) load(s + 1, g);
        compute(lds + (s & 1) * kSlot, acc);
        if (s + 1 < nk) store(lds + (s + 1 & 1) * kSlot, g);
      }
    }
  }
};

}  // namespace moe
