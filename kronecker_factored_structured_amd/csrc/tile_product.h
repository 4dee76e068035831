// The tiled matrix product shared by the vocabulary head (vocab_ce.hip) and the orthogonalised update (muon.hip):
//   C[m][n] = sum_k A[m][k] B[n][k]
// on the 16-bit matrix instruction with fp32 sums, and an epilogue that takes the sums where they are.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kron_internal.h"

namespace kron {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));

// A 16-bit matrix whose rows are ld values apart and start at a 16-byte boundary.  With two planes (fp32 values, see
// below) each 32 columns are 64 values, their first parts and then their second ones: a cache line.
struct Operand {
  const uint16_t* p;
  int64_t ld;
  int rows, cols;        // what may be read: cols is a multiple of 8 (two planes: of 32)
  const int* idx = nullptr;      // ROW: where the rows are, if not in order (all within 4 GB)
};

// fp32 values as two parts of fp16: v 2^s = hi + lo, both rounded to nearest, s so that the largest |v| 2^s is below 2^15.
// They leave at most 2^-22 of the value, or 2^-25 (2^-40 of the largest) where lo is subnormal.  Of a product's
// four terms lo lo, at most 2^-22 of it, is left out.

namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef short s4v __attribute__((ext_vector_type(4)));

typedef _Float16 h4 __attribute__((ext_vector_type(4)));

// Values whose small ones count as well (the softmax of unlikely tokens) have their second part 2^11 up, next to where the first
// one ends: 2^-36 where it is subnormal.  The other operand's first part goes 2^-11 down for that product, in registers (its values
// below 2^-3 of 2^15 lose bits then, at most 2^-25 times the second part: 2^-41 of the largest).

// The first part of four values, and what it leaves of them.  They are held as they are: folded into the conversion, the
// product that made one may round to another first part there than in what is left (one value in 2^13, off by 2^-11).
__device__ inline h4 first_part(f4& v) {
  h4 h;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float x = v[e];
    asm("" : "+v"(x));
    h[e] = (_Float16)x;
    v[e] = x - (float)h[e];
  }
  return h;
}

template <bool BF>
__device__ inline f4 mma(u4 a, u4 b, f4 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

typedef __attribute__((address_space(3))) char lds_t;

constexpr int kBK = 64;      // contraction of a step: rows of 128 bytes, whole cache lines

// ROW: the contraction runs along the operand's rows; COL: over its rows (read transposed from LDS).
enum Side { ROW, COL };

// One operand's tile of R rows (ROW) or columns (COL) x kBK, loaded straight into LDS by NW wavefronts, a KB a load: eight
// rows of 128 bytes.  ROW: 64 of the contraction (two planes: 32).  COL: 64 columns (32), the tile is R / 64 (R / 32) such
// blocks of 64 (32) rows.  The 16-byte pieces of a row are permuted, by the address that each lane loads from, so that
// fragment() reads without bank conflicts: a ROW read is served eight lanes (rows) at a time, a COL read 32 lanes: 32 bytes
// of each of eight rows 0..3, 8..11.
template <Side SD, int R, int NW, int NP>
struct TileLoad {
  static constexpr int kLoads = R * 128 / 1024 / NW;      // 1 KB wave loads of each wavefront
  static constexpr int kBlock = 64 / NP;                  // columns, and rows, of a COL block
  static_assert(kLoads * NW * 1024 == R * 128 && (SD == ROW || R % 64 == 0), "");
  const uint16_t* base;
  uint32_t off[kLoads];
  int64_t ld;
  int rows, wave;

  static __device__ int turn(int row) { return ((row >> 1) & 1) | (((row >> 3) & 1) << 1); }
  __device__ void init(const Operand& o, int at, int wave_, int lane) {
    wave = wave_, ld = o.ld, rows = o.rows;
    base = SD == ROW && !o.idx ? o.p + (int64_t)at * o.ld : o.p;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int q = wave * kLoads + i;
      if constexpr (SD == ROW) {
        const int row = q * 8 + lane / 8, chunk = (lane & 7) ^ (row & 7);
        const int r = min(row, rows - 1 - at);
        off[i] = (uint32_t)(o.idx ? o.idx[at + r] : r) * (uint32_t)(ld * 2) + chunk * 16;
      } else {
        const int row = (q % (kBlock / 8)) * 8 + lane / 8, slot = lane & 7, blk = q / (kBlock / 8);
        const int chunk = (((slot >> 1) ^ turn(row)) << 1) | (slot & 1);
        off[i] = NP == 2 ? (uint32_t)min(at / 32 + blk, o.cols / 32 - 1) * 128 + chunk * 16
                         : (uint32_t)min(at + blk * 64 + chunk * 8, o.cols - 8) * 2;
      }
    }
  }
  // Load i of the wavefront's share of the tile at k0.
  __device__ void issue(int i, int k0, lds_t* lds, int lane) const {
    const char* src;
    if constexpr (SD == ROW) {
      src = (const char*)(base + k0 * NP) + off[i];
    } else {
      const int row = min(k0 + ((wave * kLoads + i) % (kBlock / 8)) * 8 + lane / 8, rows - 1);
      src = (const char*)base + (int64_t)row * ld * 2 + off[i];
    }
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                     (__attribute__((address_space(3))) void*)(lds + (wave * kLoads + i) * 1024), 16, 0, 0);
  }
};

// Up to 16 bytes of a row, of which `left` values are there; zeros behind them.
template <bool F32>
__device__ inline u4 row_end(const char* p, int left) {
  constexpr int PER = F32 ? 4 : 8;
  typedef u4 any __attribute__((aligned(2)));
  if (left >= PER) return *(const any*)p;
  u4 o = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < PER; ++e)
    if (e < left) {
      if constexpr (F32) o[e] = ((const uint32_t*)p)[e];
      else o[e / 2] |= (uint32_t)((const uint16_t*)p)[e] << (16 * (e & 1));
    }
  return o;
}

// Operand block i (16 rows) of half kk of a step (32 of its 64 products; two planes: part kk) out of a tile in LDS; `at`:
// the wavefront's first row.
template <Side SD, int NP>
__device__ inline u4 fragment(const lds_t* lds, int at, int i, int kk, int lane) {
  const int g = lane >> 4, c = lane & 15;
  if constexpr (SD == ROW) {
    return *(const __attribute__((address_space(3))) u4*)(lds + (at + 16 * i + c) * 128 + (((kk * 4 + g) ^ (c & 7)) * 16));
  } else {
    // two transposing reads: sixteen lanes give sixteen columns of four rows, lane 4 r + q four columns of row r
    typedef TileLoad<SD, 64, 1, NP> L;
    const int r0 = (NP == 2 ? 0 : kk * 32) + 8 * g + (c >> 2), r1 = r0 + 4, blk = at / 16 + i;
    const int per = L::kBlock / 16, seg = NP == 2 ? kk * 2 + blk % per : blk % per;
    const lds_t* t = lds + (blk / per) * (L::kBlock * 128) + (c & 3) * 8;
    union { s4v h[2]; u4 u; } o;
    o.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4v*)(t + r0 * 128 + (seg ^ L::turn(r0)) * 32));
    o.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4v*)(t + r1 * 128 + (seg ^ L::turn(r1)) * 32));
    return o.u;
  }
}

// WM x WN wavefronts, each TM x TN blocks of 16 x 16; NS steps' tiles in LDS (two, more for small tiles, whose steps are
// shorter than their loads), NP planes.
//
// A step is two halves of 32 products.  While one half's fragments are multiplied the next half's come out of LDS.  Between
// the halves a barrier: behind it the next step's tiles are in LDS, its first fragments are read, and this step's tiles,
// all in registers by then, make room for step t + NS's, whose loads go out between the products (issued together
// they hold the wavefronts up: dW of 768 x 21760 over 8192 rows 303 -> 280 us) and have NS - 1 steps' time.  With two
// planes a step is 32 products in three parts, lo hi, hi hi and hi lo: each part's fragments serve two of them.
//
// KG: as many groups of WM x WN wavefronts share a tile's contraction, each with its own tiles in LDS; the first group has
// the sums in the end.
//
// UP: B's second parts are 2^UP up (two planes).
//
// F32: two "planes" that are fp32 values as they are (ROW, whole rows of 128 bytes), on the fp32 instruction.  The four
// products of a lane's 16 bytes are of every fourth k, of both operands alike.
//
// 256 x 256 tiles of eight wavefronts: 8192 x 8256 x 8192 bf16 runs at 1,370 TFLOP/s.  Registers alone would do 1,660 with
// this instruction and such values (the clock falls to 2.0 GHz with the power they take; 2,090 with zeros), loads alone
// 1,700, reads of LDS alone 4,850.  Measured beside it: 32 x 32 blocks (1,810 out of registers) 1,080-1,150; four
// wavefronts of 128 x 128 each 1,000; steps of 32 with three to five in LDS 960-1,040; raised wave priority 1,265; reads,
// loads and products interleaved by hand 1,350.
template <int WM_, int WN_, int TM_, int TN_, Side SA_, Side SB_, bool BF_, int NP_, int NS_ = 2, bool F32_ = false, int KG_ = 1, int UP = 0>
struct Product {
  static constexpr bool F32 = F32_;
  static constexpr int KG = KG_;
  static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_, NP = NP_, NS = NS_;
  static constexpr int BM = WM * TM * 16, BN = WN * TN * 16, NW = WM * WN, kThreads = 64 * NW * KG;
  static constexpr int kStage = (BM + BN) * 128, kStep = kBK / NP;
  static constexpr int kLdsBytes = KG * NS * kStage;
  typedef TileLoad<SA_, BM, NW, NP> LA;
  typedef TileLoad<SB_, BN, NW, NP> LB;
  static constexpr int kLoads = LA::kLoads + LB::kLoads;
  static constexpr bool kWhole = TM * TN <= 16;      // a step's fragments fit the registers twice
  f4 acc[TM][TN];

  struct FragsA { u4 f[TM]; };
  struct FragsB { u4 f[TN]; };
  __device__ static void read(FragsA& a, const lds_t* st, int kk, int wm, int lane) {
#pragma unroll
    for (int i = 0; i < TM; ++i) a.f[i] = fragment<SA_, NP>(st, wm * TM * 16, i, kk, lane);
  }
  __device__ static void read(FragsB& b, const lds_t* st, int kk, int wn, int lane) {
#pragma unroll
    for (int j = 0; j < TN; ++j) b.f[j] = fragment<SB_, NP>(st + BM * 128, wn * TN * 16, j, kk, lane);
  }
  __device__ void multiply_row(int i, const FragsA& a, const FragsB& b) {
    if constexpr (F32) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.f[i][e]), __uint_as_float(b.f[j][e]), acc[i][j], 0, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mma<BF_>(a.f[i], b.f[j], acc[i][j]);
    }
  }
  // Block row i of A's first part for products with B's second one.
  __device__ static void lower(FragsA& a, int i) {
    if constexpr (UP > 0) a.f[i] = __builtin_bit_cast(u4, __builtin_bit_cast(h8, a.f[i]) * (_Float16)(1.f / (1 << UP)));
  }
  // between(i): what is issued beside block row i's products.
  template <class F>
  __device__ void multiply(const FragsA& a, const FragsB& b, const F& between) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      between(i);
      multiply_row(i, a, b);
    }
  }
  // What this wavefront reads is there, and what it loads but for the last STAGES tiles; and so it is for all of them.
  template <int STAGES>
  __device__ static void in_step() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(STAGES * kLoads) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  // Sums over k from k_begin (a multiple of 64) to k_end.  A ROW operand is read up to the next multiple of 64, where
  // either operand is zero; a COL operand's rows beyond its last are that one again.  Ends with a barrier.
  __device__ void run(const Operand& A, const Operand& B, int m0, int n0, int k_begin, int k_end, lds_t* lds) {
    const int lane = threadIdx.x & 63, group = KG > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / NW : 0;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) - group * NW;
    const int wm = wave % WM, wn = wave / WM;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f4{0, 0, 0, 0};
    const int all_steps = (k_end - k_begin + kStep - 1) / kStep;
    if (all_steps <= 0) return;
    // every group takes part in `most` steps' barriers, and has `total` steps of its own
    const int most = (all_steps + KG - 1) / KG, total = KG == 1 ? all_steps : min(most, all_steps - group * most);
    k_begin += group * most * kStep;
    lds_t* const whole_lds = lds;
    lds += group * NS * kStage;
    LA la;
    LB lb;
    la.init(A, m0, wave, lane);
    lb.init(B, n0, wave, lane);
    int next = 0;      // of the tiles to load
    auto load = [&](int st, int i) {      // load i of the wavefront's for the next tiles
      const int k = k_begin + next * kStep;
      if (i < LA::kLoads) la.issue(i, k, lds + st * kStage, lane);
      else lb.issue(i - LA::kLoads, k, lds + st * kStage + BM * 128, lane);
    };
    auto all = [&](int st) {
      if (next >= total) return;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load(st, i);
      ++next;
    };
#pragma unroll
    for (int i = 0; i < NS; ++i) all(i);
    if (total >= NS) in_step<NS - 1>();
    else in_step<0>();
    int st = 0;
    auto none = [](int) {};
    if constexpr (kWhole) {
      // two sets of a step's fragments: the next step's come in while this one's are multiplied
      FragsA a[2][2];
      FragsB b[2][2];
      auto fetch = [&](int set, int at) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          read(a[set][kk], lds + at * kStage, kk, wm, lane);
          read(b[set][kk], lds + at * kStage, kk, wn, lane);
        }
      };
      fetch(0, 0);
      auto step = [&](auto set, auto more) {
        in_step<more ? NS - 2 : 0>();
        all(st);
        st = st + 1 == NS ? 0 : st + 1;
        fetch(1 - set, st);      // (behind the last step: of no use, and not used)
        if constexpr (NP == 2 && !F32) multiply(a[set][1], b[set][0], none);
        else multiply(a[set][1], b[set][1], none);
        if constexpr (UP > 0) {
          multiply(a[set][0], b[set][0], none);
          multiply(a[set][0], b[set][1], [&](int i) { lower(a[set][0], i); });
        } else {
          if constexpr (NP == 2 && !F32) multiply(a[set][0], b[set][1], none);
          multiply(a[set][0], b[set][0], none);
        }
      };
      std::integral_constant<int, 0> even;
      std::integral_constant<int, 1> odd;
      int t = 0;
      for (; t + 1 < total - NS; t += 2) {
        step(even, std::true_type{});
        step(odd, std::true_type{});
      }
      if constexpr (KG == 1) {
        for (; t + 1 < total; t += 2) {
          step(even, std::false_type{});
          step(odd, std::false_type{});
        }
        if (t < total) step(even, std::false_type{});
        __syncthreads();
      } else {
        for (; t < most; t += 2) {
          if (t < total) step(even, std::false_type{});
          else __builtin_amdgcn_s_barrier();
          if (t + 1 >= most) break;
          if (t + 1 < total) step(odd, std::false_type{});
          else __builtin_amdgcn_s_barrier();
        }
        __syncthreads();
        typedef __attribute__((address_space(3))) f4 lf4;
        static_assert((KG - 1) * NW * TM * TN * 1024 <= kLdsBytes, "");
        if (group > 0)
#pragma unroll
          for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) *(lf4*)(whole_lds + ((((group - 1) * NW + wave) * TM + i) * TN + j) * 1024 + lane * 16) = acc[i][j];
        __syncthreads();
        if (group == 0)
#pragma unroll
          for (int q = 0; q < KG - 1; ++q)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
              for (int j = 0; j < TN; ++j) acc[i][j] += *(const lf4*)(whole_lds + (((q * NW + wave) * TM + i) * TN + j) * 1024 + lane * 16);
      }
      return;
    }
    static_assert((!F32 && KG == 1) || kWhole, "");
    FragsA a0, a1;
    FragsB b0, b1;
    constexpr int first = NP == 2 ? 1 : 0;      // of A's parts
    read(b0, lds, 0, wn, lane);
    read(a0, lds, first, wm, lane);
    auto step = [&](auto more) {
      const lds_t* now = lds + st * kStage;
      auto loads = [&](int i) {
        if (!more) return;
        constexpr int per = (kLoads + TM - 1) / TM;
#pragma unroll
        for (int q = 0; q < per; ++q)
          if (i * per + q < kLoads) load(st, i * per + q);
      };
      const int after = st + 1 == NS ? 0 : st + 1;
      if constexpr (NP == 2) {
        read(a1, now, 0, wm, lane);
        multiply(a0, b0, none);
        read(b1, now, 1, wn, lane);
        multiply(a1, b0, none);
        if constexpr (UP > 0) {
          // (in place, behind the products that need it as it was: with both of them alive tiles of 256 spill, 1.55 -> 1.76 ms
          // of 2050 x 1024 x 32003 with gradients; so 1.56)
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < TM; ++i) lower(a1, i);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        read(b1, now, 1, wn, lane);
        read(a1, now, 1, wm, lane);
        multiply(a0, b0, none);
      }
      in_step<more ? NS - 2 : 0>();
      read(b0, lds + after * kStage, 0, wn, lane);      // (behind the last step: of no use, and not used)
      read(a0, lds + after * kStage, first, wm, lane);
      multiply(a1, b1, loads);
      if (more) ++next;
      st = after;
    };
    int t = 0;
    for (; t < total - NS; ++t) step(std::true_type{});
    for (; t < total; ++t) step(std::false_type{});
    __syncthreads();
  }

  // What is left of rows (ROW, as they are) behind the last whole step, from `at` to K; row_a(m), row_b(n): where they begin.
  template <class RA, class RB>
  __device__ void run_end(const RA& row_a, const RB& row_b, int at, int K) {
    static_assert(NP == 1 || F32, "");
    constexpr int SZ = F32 ? 4 : 2, PER = 16 / SZ;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, c = lane & 15;
    const char *pa[TM], *pb[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) pa[i] = row_a((wave % WM) * TM * 16 + 16 * i + c);
#pragma unroll
    for (int j = 0; j < TN; ++j) pb[j] = row_b((wave / WM) * TN * 16 + 16 * j + c);
#pragma unroll 1
    for (int k = at + g * PER; k - g * PER < K; k += 4 * PER) {
      FragsA a;
      FragsB b;
#pragma unroll
      for (int j = 0; j < TN; ++j) b.f[j] = row_end<F32>(pb[j] + k * SZ, K - k);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        a.f[i] = row_end<F32>(pa[i] + k * SZ, K - k);
        multiply_row(i, a, b);
      }
    }
  }
};

// Workgroup `id` of tm x tn tiles as (mt, nt): each of the eight XCDs takes a run of them, in bands of `width` nt
// tiles (what is read again soon stays in its L2).
__device__ inline void tile_of(int id, int count, int tm, int tn, int& mt, int& nt, int width = 8) {
  const int x = id & 7, q = count / 8, r = count % 8;
  id = x * q + min(x, r) + (id >> 3);
  const int band = id / (width * tm), first = band * width, wide = min(width, tn - first), in = id - band * width * tm;
  nt = first + in % wide, mt = in / wide;
}

// A tile's sums as 16-bit values into rows n of `out` (ld values apart, m contiguous; `rows` of the tile's are written), with
// two planes each 32 of m as their first parts and then their second: through the LDS of the wavefront, so that whole
// lines are written (dz of 8192 x 12288: 195 -> 173 us against eight bytes of each of sixteen rows at a time).
// value(i, j): part after part of the four values of block (i, j).
template <class P, class F>
__device__ __forceinline__ void store_rows(char* smem, uint16_t* out, int64_t ld, int rows, const F& value) {
  constexpr int RB = P::TM * 32 * P::NP, CH = RB / 16, PR = 64 / CH;      // bytes and 16-byte pieces of a row, rows at a time
  static_assert(CH * PR == 64 && P::NW * RB * 16 <= P::kLdsBytes, "");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  const int wm = wave % P::WM, wn = wave / P::WM;
  char* mine = smem + wave * (RB * 16);
#pragma unroll
  for (int j = 0; j < P::TN; ++j) {
#pragma unroll
    for (int i = 0; i < P::TM; ++i)
#pragma unroll
      for (int q = 0; q < P::NP; ++q) {
        const int piece = (P::NP == 2 ? (i >> 1) * 8 + q * 4 + (i & 1) * 2 : 2 * i) + (g >> 1);
        *(uint2*)(mine + c * RB + ((piece ^ (c & (CH - 1))) * 16) + (g & 1) * 8) = value(i, j);
      }
    asm volatile("" ::: "memory");
#pragma unroll
    for (int q = 0; q < 16 / PR; ++q) {
      const int r = q * PR + lane / CH, ch = lane % CH, n = wn * P::TN * 16 + 16 * j + r;
      const u4 v = *(const u4*)(mine + r * RB + ((ch ^ (r & (CH - 1))) * 16));
      if (n < rows) *(u4*)(out + (int64_t)n * ld + wm * P::TM * 16 * P::NP + ch * 8) = v;
    }
    asm volatile("" ::: "memory");
  }
}

// Lets a kernel have all of a CU's LDS, once for each device.
template <auto kernel>
hipError_t allow_lds() {
  static std::atomic<uint64_t> done{0};
  int device = 0;
  hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return e;
  const uint64_t bit = uint64_t(1) << (device & 63);
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace
}  // namespace kron
