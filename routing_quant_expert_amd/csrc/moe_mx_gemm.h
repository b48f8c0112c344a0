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
//
// A step's scales are 8 bytes of every row, each in a cache line of its own: brought in step by step they cost as many
// lines as the codes (12288 rows over 384 groups of 2048 x 4096, gated: 787 us, 643 without them). So they come for G
// steps at once, into buffers of their own (685 with four).
#pragma once

#include "moe_wide.h"

namespace moe {

constexpr int kMxStep = 256;   // elements of a step
constexpr int kMxBlock = 32;   // elements of a scale

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// C += A B of the lane's 32 elements each; bytes SA and SB of the scales.
template <int SA, int SB>
__device__ __forceinline__ f32x4 mfma_mx(i32x4 a, i32x4 b, f32x4 c, int sa, int sb) {
  constexpr int kFp4 = 4;
  const i32x8 a8 = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 b8 = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, kFp4, kFp4, SA, sa, SB, sb);
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

// R rows of NT threads' tile; scales for G steps at once.
template <int R, int NT, bool PAIRS, int G>
struct MxTile {
  static constexpr int kCodes = R * 128;
  static constexpr int kChunks = R * 8;
  static constexpr int kPer = kChunks >= NT ? kChunks / NT : 1;   // chunks a thread brings in
  static constexpr int kRowWords = 2 * G;                         // of 4 scales
  static constexpr int kWords = R * kRowWords;
  static constexpr int kPerScales = kWords >= NT ? kWords / NT : 1;
  static constexpr int kScales = 4 * kWords;
  static_assert(kChunks % NT == 0 || NT % kChunks == 0, "chunks over threads");
  static_assert((kWords % NT == 0 || NT % kWords == 0) && kWords % 64 == 0, "words of scales over threads");
  static_assert(!PAIRS || (NT % (64 * G) == 0 && NT % 256 == 0 && kChunks >= NT && kWords >= NT), "what a thread brings in is all of one matrix");

  __device__ static __forceinline__ int position(int k) { return kChunks < NT ? threadIdx.x % kChunks : threadIdx.x + NT * k; }
  __device__ static __forceinline__ int chunk(int i) { return i % 8 ^ (i / 8 & 7); }
  // The row of its matrix that tile row `row` is (the tile's last one for those past it).
  __device__ static __forceinline__ int own(const MxOperand& o, int row) {
    return min(PAIRS ? row / 32 * 16 + row % 16 : row, o.count - 1);
  }
  // Word w of a row lies at word w ^ turned(row): 16 rows then spread over the banks.
  __device__ static __forceinline__ int turned(int row) { return G == 4 ? row >> 1 & 4 : 0; }
  __device__ static __forceinline__ int word(int k) { return kWords < NT ? threadIdx.x % kWords : threadIdx.x + NT * k; }

  // Where a thread's rows start, the same in every lane of its wave (8 rows of chunks, 32 / G rows of scales to a wave).
  __device__ static __forceinline__ const uint8_t* codes(const MxOperand& o) {
    return o.codes + (PAIRS && (threadIdx.x >> 7 & 1) ? o.then : 0);
  }
  __device__ static __forceinline__ const uint8_t* scales(const MxOperand& o) {
    return o.scales + (PAIRS && (threadIdx.x / (32 * G) & 1) ? o.scales_then : 0);
  }
  struct Offsets {
    uint32_t codes[kPer], scales[kPerScales];
  };
  // Of scales: the first `words` of a row; those past them repeat the last one.
  __device__ static __forceinline__ void scale_offsets(const MxOperand& o, int words, uint32_t (&off)[kPerScales]) {
#pragma unroll
    for (int k = 0; k < kPerScales; ++k) {
      const int row = word(k) / kRowWords, w = word(k) % kRowWords ^ turned(row);
      off[k] = (uint32_t)own(o, row) * (uint32_t)o.scale_ld + 4 * min(w, words - 1);
    }
  }
  __device__ static __forceinline__ void offsets(const MxOperand& o, Offsets& off) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) off.codes[k] = (uint32_t)own(o, position(k) / 8) * (uint32_t)o.ld + 16 * chunk(position(k));
    scale_offsets(o, kRowWords, off.scales);
  }

  // (As TileOf::dma; `at` is the same in every lane of a wave.) ONCE: nothing else reads these codes, and they are the first
  // to leave the caches: a line of scales, which is read in pieces of 4 steps, then stays until its last piece.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  template <bool ONCE>
  __device__ static __forceinline__ void dma_codes(const uint8_t* at, const uint32_t (&off)[kPer], uint32_t tile) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t first = tile + 16 * 64 * (wave % (kChunks < NT ? kChunks / 64 : NT / 64));
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if constexpr (ONCE)
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt"
                     : : "v"(off[k]), "s"(at), "s"(first + 16 * NT * k) : "memory", "m0");
      else
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                     : : "v"(off[k]), "s"(at), "s"(first + 16 * NT * k) : "memory", "m0");
    }
  }
  __device__ static __forceinline__ void dma_scales(const uint8_t* at, const uint32_t (&off)[kPerScales], uint32_t buffer) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t first = buffer + 4 * 64 * (wave % (kWords < NT ? kWords / 64 : NT / 64));
#pragma unroll
    for (int k = 0; k < kPerScales; ++k)
      asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
                   : : "v"(off[k]), "s"(at), "s"(first + 4 * NT * k) : "memory", "m0");
  }
  // The thread's k-th word of scales, for any k.
  __device__ static __forceinline__ uint32_t word_offset(const MxOperand& o, int k) {
    static_assert(G == 4 && NT == 256);   // 32 rows to k
    const int row = threadIdx.x / 8, first = PAIRS ? row % 16 : row;
    return (uint32_t)min(first + (PAIRS ? 16 : 32) * k, o.count - 1) * (uint32_t)o.scale_ld + 4 * (threadIdx.x % 8 ^ turned(row));
  }
  // One chunk, and one word of scales, alone.
  __device__ static __forceinline__ void dma_code(const uint8_t* at, uint32_t off, uint32_t tile, int k) {
    const uint32_t first = tile + 16 * 64 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 : : "v"(off), "s"(at), "s"(first + 16 * NT * k) : "memory", "m0");
  }
  __device__ static __forceinline__ void dma_scale(const uint8_t* at, uint32_t off, uint32_t buffer, int k) {
    const uint32_t first = buffer + 4 * 64 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
                 : : "v"(off), "s"(at), "s"(first + 4 * NT * k) : "memory", "m0");
  }
#pragma clang diagnostic pop

  // One step through registers at any alignment; `left` elements of each row are there (fewer than a step: zeros follow),
  // room: the rows have 16 bytes of codes or more. Its scales take the words of a buffer's first step.
  static constexpr int kStepWords = 2 * R;
  static constexpr int kPerStep = kStepWords >= NT ? kStepWords / NT : 1;
  struct Stage {
    i32x4 codes[kPer];
    uint32_t scales[kPerStep];
  };
  __device__ static __forceinline__ int step_word(int k) { return kStepWords < NT ? threadIdx.x % kStepWords : threadIdx.x + NT * k; }
  __device__ static __forceinline__ void load(const MxOperand& o, const uint32_t (&off)[kPer], int s, int left, bool room, Stage& g) {
    const uint8_t* const from = codes(o) + 128 * (int64_t)s;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int at = 16 * chunk(position(k));
      g.codes[k] = bytes16(from + off[k], (left + 1) / 2 - at, room);
      if (left & 1) {   // the half of the last byte past an odd row
        const int last = left / 2 - at;
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (last >= 4 * w && last < 4 * w + 4) g.codes[k][w] &= (16u << (8 * (last - 4 * w))) - 1;
      }
    }
#pragma unroll
    for (int k = 0; k < kPerStep; ++k) {
      const int row = step_word(k) / 2, w = step_word(k) % 2;
      const uint8_t* const p = o.scales + (PAIRS && (row / 16 & 1) ? o.scales_then : 0) + 8 * (int64_t)s +
                               (uint32_t)own(o, row) * (uint32_t)o.scale_ld + 4 * w;
      const int n = (left + kMxBlock - 1) / kMxBlock - 4 * w;   // scales there
      uint32_t v = 0;
      if (n >= 4) {
        __builtin_memcpy(&v, p, 4);
      } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (i < n) v |= (uint32_t)p[i] << (8 * i);
      }
      g.scales[k] = v;
    }
  }
  __device__ static __forceinline__ void store(const Stage& g, uint8_t* tile, uint8_t* buffer) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) *reinterpret_cast<i32x4*>(tile + 16 * position(k)) = g.codes[k];
#pragma unroll
    for (int k = 0; k < kPerStep; ++k) {
      const int row = step_word(k) / 2, w = step_word(k) % 2;
      *reinterpret_cast<uint32_t*>(buffer + 4 * (kRowWords * row + (w ^ turned(row)))) = g.scales[k];
    }
  }

  // The lane's block and its two scales: row `own` + lane % 16, blocks 2 (lane / 16) + kk of the step, which is step `in` of
  // its buffer.
  __device__ static __forceinline__ i32x4 operand(const uint8_t* tile, int own, int kk, int lane) {
    const int row = own + (lane & 15);
    return *reinterpret_cast<const i32x4*>(tile + 128 * row + 16 * ((2 * (lane >> 4) + kk) ^ (row & 7)));
  }
  __device__ static __forceinline__ int scale(const uint8_t* buffer, int own, int in, int lane) {
    const int row = own + (lane & 15);
    return *reinterpret_cast<const uint16_t*>(buffer + 4 * (kRowWords * row + ((2 * in + (lane >> 5)) ^ turned(row))) + 2 * (lane >> 4 & 1));
  }
};

// DMA: codes 16-byte and scales 4-byte aligned, brought into LDS directly; otherwise through registers, any alignment.
// ONCE: hardly any group has rows for a second tile, which would read its weights again.
template <int BP, int BQ, int WP, int WQ, int ST, int G, bool DMA, bool PAIRS, bool ONCE = false>
struct MxGemm : TileOut<BP, BQ, WP, WQ, PAIRS> {
  typedef TileOut<BP, BQ, WP, WQ, PAIRS> Out;
  using Out::NT, Out::NP, Out::NQ, Out::wave_p, Out::wave_q;
  typedef typename Out::Acc Acc;
  typedef MxTile<BP, NT, PAIRS, G> PT;
  typedef MxTile<BQ, NT, false, G> QT;
  static constexpr int kSlots = DMA ? ST : 2;
  static constexpr int kSlot = PT::kCodes + QT::kCodes;
  // A buffer takes the next G steps' scales together with the first of these steps' codes, when all waves are past the
  // step ST before it: the buffer's last steps are then no later than that.
  static constexpr int kBuffers = DMA ? (ST + G - 2) / G + 1 : 2;
  static constexpr int kBuffer = PT::kScales + QT::kScales;
  static constexpr int kLds = kSlots * kSlot + kBuffers * kBuffer;

  struct Half {
    i32x4 p[NP], q[NQ];
    int ps[NP], qs[NQ];
  };
  // KK = 0: with the step's scales, step `in` of `buffer`; the second half takes them from `first`.
  template <int KK>
  __device__ static __forceinline__ void read(const uint8_t* slot, const uint8_t* buffer, int in, Half& h, const Half* first = nullptr) {
    const int lane = threadIdx.x & 63, p0 = wave_p(), q0 = wave_q();
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      h.q[j] = QT::operand(slot + PT::kCodes, q0 + 16 * j, KK, lane);
      h.qs[j] = KK ? first->qs[j] : QT::scale(buffer + PT::kScales, q0 + 16 * j, in, lane);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      h.p[i] = PT::operand(slot, p0 + 16 * i, KK, lane);
      h.ps[i] = KK ? first->ps[i] : PT::scale(buffer, p0 + 16 * i, in, lane);
    }
  }
  template <int KK>
  __device__ static __forceinline__ void multiply(const Half& h, Acc& acc) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int j = 0; j < NQ; ++j) acc[i][j] = mfma_mx<KK, KK>(h.p[i], h.q[j], acc[i][j], h.ps[i], h.qs[j]);
  }
  // Places `READS` LDS reads evenly among the first products of the half before.
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
  __device__ static __forceinline__ void compute(const uint8_t* slot, const uint8_t* buffer, Acc& acc) {
    Half h0, h1;
    read<0>(slot, buffer, 0, h0);
    read<1>(slot, buffer, 0, h1, &h0);
    multiply<0>(h0, acc);
    multiply<1>(h1, acc);
  }

  // Waits until nothing older than what steps first .. last (fewer than ST) brought in is in flight.
  __device__ static __forceinline__ void wait_before(int first, int last) {
    constexpr int kCodes = PT::kPer + QT::kPer, kScales = PT::kPerScales + QT::kPerScales;
    if (last >= first && last / G * G >= first) wait_steps<kCodes, ST - 1, kScales>(last - first + 1);
    else wait_steps<kCodes, ST - 1>(max(last - first + 1, 0));
  }

  // Adds the sum over the k elements of the rows. LDS is free for other use after a barrier.
  __device__ static __forceinline__ void run(const MxOperand& p, const MxOperand& q, int k, uint8_t* lds, Acc& acc) {
    typename PT::Offsets po;
    typename QT::Offsets qo;
    PT::offsets(p, po);
    QT::offsets(q, qo);
    const bool room = k >= 32;
    uint8_t *const end = lds + kSlots * kSlot, *const buffers = end, *const last = buffers + (kBuffers - 1) * kBuffer;
    struct Stage {
      typename PT::Stage p;
      typename QT::Stage q;
    };
    auto load = [&](int s, Stage& g) {
      PT::load(p, po.codes, s, k - s * kMxStep, room, g.p);
      QT::load(q, qo.codes, s, k - s * kMxStep, room, g.q);
    };
    auto store = [&](const Stage& g, uint8_t* slot, uint8_t* buffer) {
      PT::store(g.p, slot, buffer);
      QT::store(g.q, slot + PT::kCodes, buffer + PT::kScales);
    };
    if constexpr (DMA) {
      const int nk = k / kMxStep;
      const uint8_t *pc = uniform(PT::codes(p)), *ps = uniform(PT::scales(p)), *qc = uniform(q.codes), *qs = uniform(q.scales);
      uint32_t put = lds_offset(buffers);   // the buffer of the next scales asked for
      auto issue = [&](int s, const uint8_t* slot) {
        if (s % G == 0) {
          if (nk - s >= G) {
            PT::dma_scales(ps, po.scales, put);
            QT::dma_scales(qs, qo.scales, put + PT::kScales);
          } else {
            uint32_t pw[PT::kPerScales], qw[QT::kPerScales];
            PT::scale_offsets(p, 2 * (nk - s), pw);
            QT::scale_offsets(q, 2 * (nk - s), qw);
            PT::dma_scales(ps, pw, put);
            QT::dma_scales(qs, qw, put + PT::kScales);
          }
          ps += 8 * G;
          qs += 8 * G;
          put = put == lds_offset(last) ? lds_offset(buffers) : put + kBuffer;
        }
        const uint32_t at = lds_offset(slot);
        PT::template dma_codes<ONCE>(pc, po.codes, at);
        QT::template dma_codes<false>(qc, qo.codes, at + PT::kCodes);
        pc += 128;
        qc += 128;
      };
#pragma unroll
      for (int s = 0; s < ST - 1; ++s)
        if (s < nk) issue(s, lds + s * kSlot);
      if (k % kMxStep) {   // the last, partial step first, in the slot and the buffer that the ring needs last
        Stage g;
        load(nk, g);
        store(g, end - kSlot, last);
        lds_barrier();
        compute(end - kSlot, last, acc);
        lds_barrier();
      }
      if (nk == 0) return;
      if (ST - 1 < nk) issue(ST - 1, end - kSlot);
      // (as Gemm::run)
      Half h0, h1;
      wait_before(1, min(nk, ST) - 1);
      lds_barrier();
      const uint8_t *get = lds, *scales = buffers;
      read<0>(get, scales, 0, h0);
      int s = 0;
      auto next = [&] {   // to step s + 1
        get = get + kSlot == end ? lds : get + kSlot;
        if ((s + 1) % G == 0) scales = scales == last ? buffers : scales + kBuffer;
      };
#pragma unroll 1
      for (; s < nk - ST; ++s) {
        read<1>(get, scales, s % G, h1, &h0);
        multiply<0>(h0, acc);
        interleave<NP + NQ>();
        if constexpr (ST == 2) wait_vmcnt<0>();
        else wait_before(s + 2, s + ST - 1);   // step s + 1 is in; later ones may be in flight
        lds_barrier();                         // for every wave; and all have read step s
        issue(s + ST, get);
        next();
        read<0>(get, scales, (s + 1) % G, h0);
        multiply<1>(h1, acc);
        interleave<2 * (NP + NQ)>();
      }
#pragma unroll 1
      for (; s < nk - 1; ++s) {
        read<1>(get, scales, s % G, h1, &h0);
        multiply<0>(h0, acc);
        interleave<NP + NQ>();
        wait_before(s + 2, min(nk, s + ST) - 1);
        lds_barrier();
        next();
        read<0>(get, scales, (s + 1) % G, h0);
        multiply<1>(h1, acc);
        interleave<2 * (NP + NQ)>();
      }
      read<1>(get, scales, s % G, h1, &h0);
      multiply<0>(h0, acc);
      multiply<1>(h1, acc);
    } else {
      const int nk = (k + kMxStep - 1) / kMxStep;
      if (nk == 0) return;
      Stage g;
      load(0, g);
      store(g, lds, buffers);
#pragma unroll 1
      for (int s = 0; s < nk; ++s) {
        lds_barrier();   // step s is there, and all are done with step s - 1
        if (s + 1 < nk) load(s + 1, g);
        compute(lds + (s & 1) * kSlot, buffers + (s & 1) * kBuffer, acc);
        if (s + 1 < nk) store(g, lds + (s + 1 & 1) * kSlot, buffers + (s + 1 & 1) * kBuffer);
      }
    }
  }
};

// The same in wide tiles (moe_wide.h): rows of whole groups of four steps (k a multiple of 1024), 16-byte aligned codes and
// 4-byte aligned scales. The scales of four steps come in quarters, one beside the codes of each step, during the four
// steps that end one before they are needed: a buffer's last step has then been read by all.
template <bool PAIRS>
struct WideMx : WideOut<PAIRS> {
  typedef MxTile<256, 256, PAIRS, 4> PT;
  typedef MxTile<256, 256, false, 4> QT;
  typedef WideOut<PAIRS> Out;
  static constexpr int kSlot = PT::kCodes + QT::kCodes;
  static constexpr int kBuffer = PT::kScales + QT::kScales;
  static constexpr int kLds = 2 * kSlot + 2 * kBuffer;   // all of a CU's
  static constexpr int kGroup = 4 * kMxStep;

  // Two operands' scales of a step share a register: bytes 2 (i % 2) + kk.
  template <int NQ>
  struct Half {
    i32x4 p[8], q[NQ];
    u16x2 ps[4], qs[NQ / 2];
  };
  // Where a lane's operands lie in a slot and its scales in a buffer: the rows' n-th 4096 n bytes (scales: 1024 n) after `q`,
  // P's i-th 2048 i (512 i) after `p`; the scales of the buffer's step `in` are at the place with 8 in XORed to it.
  struct Places {
    uint32_t p[2], q[2], ps, qs;
    __device__ __forceinline__ Places() {
      const int lane = threadIdx.x & 63, row = lane & 15;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const uint32_t at = 128 * row + 16 * ((2 * (lane >> 4) + kk) ^ (row & 7));
        q[kk] = PT::kCodes + 128 * 16 * (Out::wave() / 2) + at;
        p[kk] = 128 * Out::wave_p() + at;
      }
      const uint32_t at = 32 * row + 4 * (lane >> 5 ^ PT::turned(row)) + 2 * (lane >> 4 & 1);
      qs = PT::kScales + 32 * 16 * (Out::wave() / 2) + at;
      ps = 32 * Out::wave_p() + at;
    }
  };
  // Read number n of half step KK of a slot: the rows' operands, then P's; in the first half with their scales, which the
  // second half takes from `first`.
  template <int KK, int NQ>
  __device__ static __forceinline__ void read(uint32_t slot, uint32_t ps, uint32_t qs, const Places& places, int n, Half<NQ>& h,
                                              const Half<NQ>* first) {
    typedef unsigned short u16;
    if (n < NQ) {
      h.q[n] = lds_at<i32x4>(slot + places.q[KK] + 4096 * n);
      if (!KK) h.qs[n / 2][n % 2] = lds_at<u16>(qs + 1024 * n);
      else if (n % 2) h.qs[n / 2] = first->qs[n / 2];
    } else {
      const int i = n - NQ;
      h.p[i] = lds_at<i32x4>(slot + places.p[KK] + 2048 * i);
      if (!KK) h.ps[i / 2][i % 2] = lds_at<u16>(ps + 512 * i);
      else if (i % 2) h.ps[i / 2] = first->ps[i / 2];
    }
  }
  template <int KK, int NQ>
  __device__ static __forceinline__ void multiply(const Half<NQ>& h, int n, f32x4 (&acc)[8][NQ]) {
    const int i = n / NQ, j = n % NQ, a = __builtin_bit_cast(int, h.ps[i / 2]), b = __builtin_bit_cast(int, h.qs[j / 2]);
    f32x4& c = acc[i][j];
    if (i % 2) c = j % 2 ? mfma_mx<2 + KK, 2 + KK>(h.p[i], h.q[j], c, a, b) : mfma_mx<2 + KK, KK>(h.p[i], h.q[j], c, a, b);
    else c = j % 2 ? mfma_mx<KK, 2 + KK>(h.p[i], h.q[j], c, a, b) : mfma_mx<KK, KK>(h.p[i], h.q[j], c, a, b);
  }

  template <int NQ>
  __device__ static __forceinline__ void run(const MxOperand& p, const MxOperand& q, int k, uint8_t* lds, f32x4 (&acc)[8][NQ]) {
    // a step's loads: 8 + NQ of codes, and of a quarter of scales two of P's and NQ / 4 of the rows' (NQ = 6: two, NQ = 2: one,
    // of which some repeat the last)
    constexpr int kScaleQ = (NQ + 3) / 4, kLoads = 8 + NQ + 2 + kScaleQ;
    typedef WideOrder<NQ, kLoads> O;
    const int nk = k / kMxStep, groups = nk / 4;
    typename PT::Offsets po;
    typename QT::Offsets qo;
    PT::offsets(p, po);
    QT::offsets(q, qo);
    const uint8_t *pc = uniform(PT::codes(p)), *qc = uniform(q.codes), *ps = uniform(PT::scales(p)), *qs = uniform(q.scales);
    uint8_t* const buffers = lds + 2 * kSlot;
    // Number n of a step's loads, codes into `at`; the scales are quarter `part` of a buffer at `to`.
    auto load = [&](int n, uint32_t at, uint32_t to, int part) {
      if (n < 8) {
        PT::dma_code(pc, po.codes[n], at, n);
      } else if (n < 8 + NQ) {
        QT::dma_code(qc, qo.codes[n - 8], at + PT::kCodes, n - 8);
      } else if (n < 8 + NQ + 2) {
        const int w = 2 * part + n - 8 - NQ;
        PT::dma_scale(ps, PT::word_offset(p, w), to, w);
      } else {
        const int w = min(kScaleQ * part + n - 8 - NQ - 2, NQ - 1);
        QT::dma_scale(qs, QT::word_offset(q, w), to + PT::kScales, w);
      }
    };
    auto loaded = [&] {
      pc += 128;
      qc += 128;
    };
    // group 0's scales, then the codes of steps 0 and 1 with the first quarter of group 1's scales
#pragma unroll
    for (int n = 0; n < 8; ++n) PT::dma_scale(ps, PT::word_offset(p, n), lds_offset(buffers), n);
#pragma unroll
    for (int n = 0; n < NQ; ++n) QT::dma_scale(qs, QT::word_offset(q, n), lds_offset(buffers) + PT::kScales, n);
    if (groups > 1) {
      ps += 32;
      qs += 32;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int n = 0; n < 8 + NQ; ++n) load(n, lds_offset(lds) + s * kSlot, 0, 0);
      loaded();
    }
#pragma unroll
    for (int n = 8 + NQ; n < kLoads; ++n) load(n, 0, lds_offset(buffers) + kBuffer, 0);
    Half<NQ> h0, h1;
    wait_vmcnt<kLoads>();
    lds_barrier();
    uint32_t get = lds_offset(lds), then = get + kSlot, scales = lds_offset(buffers);
    const Places places;
#pragma unroll
    for (int n = 0; n < O::kReads; ++n) read<0>(get, scales + places.ps, scales + places.qs, places, n, h0, (const Half<NQ>*)nullptr);
    // Step s; with LOAD the codes of step s + 2, and the scales that step s + 1's quarter stands for, are asked for.
    auto step = [&](int s, auto LOAD, auto NEXT) {
      const uint32_t at = get;
      const int part = (s + 1) & 3;
      if (LOAD && part == 0) {   // the next group's, or the last one's again
        const bool more = (s + 1) / 4 + 1 < groups;
        ps += more ? 32 : 0;
        qs += more ? 32 : 0;
      }
      const uint32_t to = lds_offset(buffers) + ((((s + 1) >> 2) + 1) & 1) * kBuffer;
#pragma unroll
      for (int g = 0; g < O::kGroups; ++g) {
#pragma unroll
        for (int n = O::kEach * g; n < O::kEach * (g + 1); ++n)
          if (n < O::kReads) read<1>(get, 0, 0, places, n, h1, &h0);
        if (LOAD && g == O::kFree) lds_barrier();   // all have read the step
        multiply<0>(h0, 2 * g, acc);
        multiply<0>(h0, 2 * g + 1, acc);
        if (LOAD) {
#pragma unroll
          for (int n = 0; n < kLoads; ++n)
            if (O::at(n) == g) load(n, at, to, part);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (NEXT) {   // the next step is there, for every wave
        wait_vmcnt<LOAD ? O::first() : 0>();
        lds_barrier();
        if (part == 0) scales = scales == lds_offset(buffers) ? scales + kBuffer : lds_offset(buffers);
      }
      const uint32_t ps_at = scales + (places.ps ^ 8 * part), qs_at = scales + (places.qs ^ 8 * part);
#pragma unroll
      for (int g = 0; g < O::kGroups; ++g) {
        if (NEXT) {
#pragma unroll
          for (int n = O::kEach * g; n < O::kEach * (g + 1); ++n)
            if (n < O::kReads) read<0>(then, ps_at, qs_at, places, n, h0, (const Half<NQ>*)nullptr);
        }
        multiply<1>(h1, 2 * g, acc);
        multiply<1>(h1, 2 * g + 1, acc);
        if (LOAD) {
#pragma unroll
          for (int n = 0; n < kLoads; ++n)
            if (O::at(n) == O::kGroups + g) load(n, at, to, part);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (LOAD) loaded();
      const uint32_t was = get;
      get = then;
      then = was;
    };
    own_registers(acc);
#pragma unroll 1
    for (int s = 0; s < nk - 2; ++s) step(s, std::true_type(), std::true_type());
    step(nk - 2, std::false_type(), std::true_type());
    step(nk - 1, std::false_type(), std::false_type());
  }
};

}  // namespace moe
