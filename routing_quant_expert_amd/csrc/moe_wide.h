// The tile product of moe_gemm.h for aligned rows and sums of whole steps (four
// and more): 256 x (up to) 256 outputs, one workgroup of four waves a CU. For
// many rows, and where weights are read across the sum for few rows of many
// groups too, in longer pieces of a row (launch_gated_rows, launch_mx).
//
// A wave holds 128 x 128 sums in accumulation registers, so that an LDS read
// feeds eight products where 64 x 64 sums make it four: 64 x 64 take the LDS
// port for 1400 cycles in every 1024 of the matrix instructions, 128 x 128 for
// 750. There is no second wave on the SIMD to fill a pause; what a wave waits
// for is arranged instead. The products of a half step run between the reads of
// the next half's operands and the loads of the step after next, one of them at
// a time: 16 loads in a row take the memory pipeline 1024 cycles, in which the
// wave that issues them cannot go on (435 us with loads among the products, 489
// without, 16384 rows over 4 groups of 2048 x 4096, gated).
//
//   step s    first half:  products | reads of the second half | barrier: all have read step s | loads of step s + 2 ...
//             second half: wait for step s + 1, barrier | products | reads of its first half | ... loads of step s + 2
//
// The rows of a tile are dealt to the two waves across it 16 at a time, so that
// a tile with fewer rows takes fewer products of every wave (NQ = 8, 6, 4 or 2
// for 32 rows each).
#pragma once

#include "moe_gemm.h"

namespace moe {

// How the loads and reads of a step lie among its products, in groups of two products (32 cycles, in which LDS gives each
// wave one operand). Evenly spread: 16384 rows over 4 groups of 2048 x 4096, gated, 430 us with two reads a group and the
// loads in half of the step, 411 with one and the loads in two thirds of it.
template <int NQ, int LOADS>
struct WideOrder {
  static constexpr int kGroups = 4 * NQ;                                            // of a half step
  static constexpr int kReads = 8 + NQ;                                             // operands of a half step
  static constexpr int kEach = kReads > kGroups / 2 + 2 ? 2 : 1;                    // reads in a group
  static constexpr int kFree = kReads + 2 < kGroups ? kReads + 2 : kGroups - 1;     // the step's reads are back: the barrier
  static constexpr int kWindow = 2 * kGroups - kFree - kGroups / 5;                 // groups of the loads
  static constexpr int at(int load) { return kFree + load * kWindow / LOADS; }
  static constexpr int first() {                                                    // loads in the first half step
    int n = 0;
    while (n < LOADS && at(n) < kGroups) ++n;
    return n;
  }
};

// The sums of a wide tile: wave w has outputs 128 (w % 2) on, and of every 32 rows the 16 from 16 (w / 2).
// PAIRS: of two matrices, 64 outputs each.
template <bool PAIRS>
struct WideOut {
  static constexpr int NT = 256, kP = PAIRS ? 128 : 256, kQ = 256;
  __device__ static __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
  __device__ static __forceinline__ int wave_p() { return wave() % 2 * 128; }
  __device__ static __forceinline__ int row_of(int j) { return 32 * j + 16 * (wave() / 2) + (threadIdx.x & 15); }
  // The first of the 8 outputs that a lane has of tiles 0 and 1 after neighbours() (of tiles i and i + 1: 16 i on).
  __device__ static __forceinline__ int first_out() {
    const int g = threadIdx.x >> 4 & 3;
    return (PAIRS ? wave_p() / 2 : wave_p()) + 16 * (g % 2) + 8 * (g / 2);
  }
  // Four sums of tile a and of tile b, 16 outputs apart -> eight neighbouring ones of one of them: 16 lanes with their neighbours.
  __device__ static __forceinline__ f32x8 neighbours(f32x4 a, f32x4 b) {
    f32x8 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = a[e], y = b[e];
      const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y), false, false);
      const uint32_t s0 = s[0], s1 = s[1];   // (as moe_wave.h)
      v[e] = __builtin_bit_cast(float, s0);
      v[e + 4] = __builtin_bit_cast(float, s1);
    }
    return v;
  }
  // Writes N tiles of sums at `out`, rows `ld` apart, `pn` outputs and `rows` rows.
  template <int N, int NQ, typename U>
  __device__ static __forceinline__ void store(const f32x4 (&v)[N][NQ], U* out, int64_t ld, int pn, int rows) {
    const int p = first_out();
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      f32x8 sums[N / 2];
#pragma unroll
      for (int i = 0; i < N; i += 2) sums[i / 2] = neighbours(v[i][j], v[i + 1][j]);
      if (row_of(j) >= rows) continue;
      U* const to = out + row_of(j) * ld + p;
#pragma unroll
      for (int i = 0; i < N; i += 2)
        if (p + 16 * i < pn) store_oct(to + 16 * i, sums[i / 2], pn - p - 16 * i);
    }
  }
};

// Every sum in registers of its own before the loop: zeroed ones would share theirs, and be moved apart in every step.
template <int NQ>
__device__ __forceinline__ void own_registers(f32x4 (&acc)[8][NQ]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < NQ; ++j) asm volatile("" : "+a"(acc[i][j]));
}

template <typename V>
__device__ __forceinline__ V lds_at(uint32_t offset) {
  return *(const __attribute__((address_space(3))) V*)offset;
}

// Whole steps of rows that start 16-byte aligned (columns: widths that are multiples of 8). DMA only.
template <typename T, bool PCOL, Two TWO>
struct WideGemm : WideOut<TWO == kRowPairs> {
  typedef TileOf<T, PCOL, 256, 256, false, TWO == kRowPairs> PT;
  typedef TileOf<T, false, 256, 256> QT;
  static constexpr int kSlot = PT::kBytes + QT::kBytes;
  static constexpr int kLds = 2 * kSlot;
  typedef WideOut<TWO == kRowPairs> Out;

  __device__ static __forceinline__ bool second_rows() { return threadIdx.x >> 7 & 1; }

  template <int NQ>
  struct Half {
    oct<T> p[8], q[NQ];
  };
  // Where a lane's operands lie in a slot (TileOf::operand): the rows' n-th 4096 n bytes after `q` of its half step, P's i-th
  // 2048 i after `p` of its half step, or of columns 16384 kk after its own `p`. A wave issues one instruction in 4 cycles,
  // 512 in a step's products, so an address for every read costs (16384 rows over 4 groups, gated: 411 us, 402 so).
  struct Places {
    uint32_t p[PCOL ? 8 : 2], q[2];
    __device__ __forceinline__ Places() {
      const int lane = threadIdx.x & 63, row = lane & 15, chunk = lane >> 4;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const uint32_t at = 128 * row + 16 * ((4 * kk + chunk) ^ QT::swizzle(row));
        q[kk] = PT::kBytes + 128 * 16 * (Out::wave() / 2) + at;
        if (!PCOL) p[kk] = 128 * Out::wave_p() + at;
      }
      if constexpr (PCOL) {
        const int r = 8 * chunk + (row >> 2), col = Out::wave_p() + 4 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int own = col + 16 * i;
          p[i] = 16 * (r * PT::kRowChunks + ((own >> 3) ^ PT::swizzle(r))) + 2 * (own & 7);
        }
      }
    }
  };
  // Read number n of half step kk of a slot: the rows' operands, then P's.
  template <int NQ>
  __device__ static __forceinline__ void read(uint32_t slot, const Places& places, int kk, int n, Half<NQ>& h) {
    if (n < NQ) {
      h.q[n] = lds_at<oct<T>>(slot + places.q[kk] + 4096 * n);
    } else if constexpr (!PCOL) {
      h.p[n - NQ] = lds_at<oct<T>>(slot + places.p[kk] + 2048 * (n - NQ));
    } else {
      const uint32_t at = slot + places.p[n - NQ] + 32 * 16 * PT::kRowChunks * kk;
      struct { s16x4 lo, hi; } v;
      v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_tr_t)at);
      v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_tr_t)(at + 4 * 16 * PT::kRowChunks));
      h.p[n - NQ] = __builtin_bit_cast(oct<T>, v);
    }
  }
  template <int NQ>
  __device__ static __forceinline__ void multiply(const Half<NQ>& h, int n, f32x4 (&acc)[8][NQ]) {
    const int i = n / NQ, j = n % NQ;
    acc[i][j] = mfma16(h.p[i], h.q[j], acc[i][j]);
  }

  // Adds the sum over r < red, whole steps, at least two (kTwoSums: both sums, each over r < red). last() is called before the last half step.
  template <int NQ, typename Last>
  __device__ static __forceinline__ void run(const Operand<T>& p, const Operand<T>& q, int red, uint8_t* lds,
                                             f32x4 (&acc)[8][NQ], Last&& last) {
    typedef WideOrder<NQ, 8 + NQ> O;
    const int each = red / kStep, nk = TWO == kTwoSums ? 2 * each : each;
    const int64_t ps = PT::step_stride(p), qs = QT::step_stride(q);
    typename PT::Off po[8];
    typename QT::Off qo[8];
    PT::template offsets<true>(p, po);
    QT::template offsets<true>(q, qo);
    const T *pat = uniform(p.base), *qat = uniform(q.base);
    int left = each;
    auto load = [&](int n, uint32_t at) {   // number n of the next step's
      if (n < 8) PT::dma_one(pat, po[n], at, n);
      else QT::dma_one(qat, qo[n - 8], at + PT::kBytes, n - 8);
    };
    auto loaded = [&] {
      pat += ps;
      qat += qs;
      if constexpr (TWO == kTwoSums) {
        if (--left == 0) {
          pat += p.then - each * ps;
          qat += q.then - each * qs;
        }
      }
    };
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int n = 0; n < 8 + NQ; ++n) load(n, lds_offset(lds) + s * kSlot);
      loaded();
    }
    Half<NQ> h0, h1;
    wait_vmcnt<8 + NQ>();
    lds_barrier();
    uint32_t get = lds_offset(lds), then = get + kSlot;
    const Places places;
#pragma unroll
    for (int n = 0; n < O::kReads; ++n) read(get, places, 0, n, h0);
    // The two half steps of a step. LOAD: the step after next follows; NEXT: the next one does.
    auto step = [&](auto LOAD, auto NEXT) {
      const uint32_t at = get;
#pragma unroll
      for (int g = 0; g < O::kGroups; ++g) {
#pragma unroll
        for (int n = O::kEach * g; n < O::kEach * (g + 1); ++n)
          if (n < O::kReads) read(get, places, 1, n, h1);
        if (LOAD && g == O::kFree) lds_barrier();   // all have read the step
        multiply(h0, 2 * g, acc);
        multiply(h0, 2 * g + 1, acc);
        if (LOAD) {
#pragma unroll
          for (int n = 0; n < 8 + NQ; ++n)
            if (O::at(n) == g) load(n, at);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (NEXT) {   // the next step is there, for every wave
        wait_vmcnt<LOAD ? O::first() : 0>();
        lds_barrier();
      } else {
        last();
      }
#pragma unroll
      for (int g = 0; g < O::kGroups; ++g) {
        if (NEXT) {
#pragma unroll
          for (int n = O::kEach * g; n < O::kEach * (g + 1); ++n)
            if (n < O::kReads) read(then, places, 0, n, h0);
        }
        multiply(h1, 2 * g, acc);
        multiply(h1, 2 * g + 1, acc);
        if (LOAD) {
#pragma unroll
          for (int n = 0; n < 8 + NQ; ++n)
            if (O::at(n) == O::kGroups + g) load(n, at);
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
    for (int s = 0; s < nk - 2; ++s) step(std::true_type(), std::true_type());
    step(std::false_type(), std::true_type());
    step(std::false_type(), std::false_type());
  }
};

// body(NQ) is called with the 32-row parts that the tile's rows need.
template <typename Body>
__device__ __forceinline__ void by_rows(int rows, Body&& body) {
  if (rows > 192) body(std::integral_constant<int, 8>());
  else if (rows > 128) body(std::integral_constant<int, 6>());
  else if (rows > 64) body(std::integral_constant<int, 4>());
  else body(std::integral_constant<int, 2>());
}

}  // namespace moe
