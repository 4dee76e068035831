// The tiled matrix product shared by the vocabulary head (vocab_ce.hip) and the orthogonalised update (muon.hip):
//   C[m][n] = sum_k A[m][k] B[n][k]
// on the 16-bit matrix instruction with fp32 sums, and an epilogue that takes the sums where they are.
#pragma once

#include <algorithm>
#include <atomic>

#include "kron_internal.h"

namespace kron {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));

// A 16-bit matrix whose rows are ld elements apart, in one plane or in two (fp32 values, see Planes below).
// Rows start at a 16-byte boundary.
struct Operand {
  const uint16_t* p;
  int64_t ld, plane;
  int rows, cols;        // what may be read: cols is a multiple of 8
};

// fp32 values as two planes of fp16: v 2^s = hi + lo 2^-11, both rounded to nearest.
constexpr float kLo = 2048.f, kLoInv = 1.f / 2048.f;

namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef short s4v __attribute__((ext_vector_type(4)));

template <bool BF>
__device__ inline f4 mma(u4 a, u4 b, f4 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

typedef __attribute__((address_space(3))) char lds_t;

constexpr int kBK = 64;      // contraction of a step

// ROW: the contraction runs along the operand's rows; COL: over its rows (read transposed from LDS).
enum Side { ROW, COL };

// One operand's tile of R rows (ROW) or columns (COL) x kBK, NW wavefronts loading it.
template <Side SD, int R, int NW>
struct TileLoad {
  static constexpr int kLoads = R * kBK * 2 / 1024 / NW;      // 1 KB wave loads of each wavefront
  static_assert(kLoads * NW * 1024 == R * kBK * 2, "");
  static constexpr int kPer = SD == ROW ? 8 : 512 / R;        // rows of one wave load
  const uint16_t* base;
  uint32_t off[kLoads];
  int64_t ld;
  int first, rows, wave;

  __device__ void init(const Operand& o, int at, int wave_, int lane) {
    wave = wave_, ld = o.ld, rows = o.rows;
    base = SD == ROW ? o.p + (int64_t)at * o.ld : o.p;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int q = wave * kLoads + i;
      if constexpr (SD == ROW) {
        const int row = q * 8 + lane / 8, chunk = (lane & 7) ^ (row & 7);
        off[i] = (uint32_t)min(row, rows - 1 - at) * (uint32_t)(ld * 2) + chunk * 16;
      } else {
        constexpr int C = R / 8;
        const int row = q * kPer + lane / C, slot = lane % C;
        const int chunk = (((slot >> 1) ^ (row & 3)) << 1) | (slot & 1);
        off[i] = (uint32_t)min(at + chunk * 8, o.cols - 8) * 2;
      }
    }
  }
  __device__ void issue(int64_t plane, int k0, lds_t* lds, int lane) const {
    const char* b = (const char*)(base + plane + (SD == ROW ? k0 : 0));
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const char* src;
      if constexpr (SD == ROW) {
        src = b + off[i];
      } else {
        const int row = min(k0 + (wave * kLoads + i) * kPer + lane / (R / 8), rows - 1);
        src = b + (int64_t)row * ld * 2 + off[i];
      }
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                       (__attribute__((address_space(3))) void*)(lds + (wave * kLoads + i) * 1024), 16, 0, 0);
    }
  }
};

// Operand block i (16 rows) of k-slice kk (32) out of a tile in LDS; `at`: the wavefront's first row (a multiple of 16).
template <Side SD, int R>
__device__ inline u4 fragment(const lds_t* lds, int at, int i, int kk, int lane) {
  const int g = lane >> 4, c = lane & 15;
  if constexpr (SD == ROW) {
    return *(const __attribute__((address_space(3))) u4*)(lds + (at + 16 * i + c) * 128 + (((kk * 4 + g) ^ (c & 7)) * 16));
  } else {
    const int r4 = c >> 2;
    const lds_t* q = lds + (kk * 32 + 8 * g + r4) * (R * 2) + (((at / 16 + i) ^ r4) * 32) + (c & 3) * 8;
    union { s4v h[2]; u4 u; } o;
    o.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4v*)q);
    o.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4v*)(q + 4 * R * 2));
    return o.u;
  }
}

// WM x WN wavefronts, each TM x TN blocks of 16 x 16.
template <int WM_, int WN_, int TM_, int TN_, Side SA_, Side SB_, bool BF_, int NP_>
struct Product {
  static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_, NP = NP_;
  static constexpr int BM = WM * TM * 16, BN = WN * TN * 16, NW = WM * WN, kThreads = 64 * NW;
  static constexpr int kStage = (BM + BN) * kBK * 2;
  static constexpr int kLdsBytes = 2 * kStage;
  f4 acc[TM][TN];

  __device__ void run(const Operand& A, const Operand& B, int m0, int n0, int k_begin, int k_end, lds_t* lds) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    TileLoad<SA_, BM, NW> la;
    TileLoad<SB_, BN, NW> lb;
    la.init(A, m0, wave, lane);
    lb.init(B, n0, wave, lane);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f4{0, 0, 0, 0};
    const int steps = (k_end - k_begin + kBK - 1) / kBK;
    auto issue = [&](int t, int st) {
      int pair = 0, k = t;
      if constexpr (NP == 2) pair = t / steps, k = t - pair * steps;
      la.issue(NP == 2 && pair == 0 ? A.plane : 0, k_begin + k * kBK, lds + st * kStage, lane);
      lb.issue(NP == 2 && pair == 1 ? B.plane : 0, k_begin + k * kBK, lds + st * kStage + BM * kBK * 2, lane);
    };
    const int total = NP == 2 ? 3 * steps : steps;
    if (total <= 0) return;
    issue(0, 0);
    __syncthreads();
    for (int t = 0; t < total; ++t) {
      const int st = t & 1;
      if (t + 1 < total) issue(t + 1, st ^ 1);
      if constexpr (NP == 2) {
        if (t == 2 * steps) {
#pragma unroll
          for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] *= kLoInv;
        }
      }
      const lds_t* ta = lds + st * kStage;
      const lds_t* tb = ta + BM * kBK * 2;
#pragma unroll
      for (int kk = 0; kk < kBK / 32; ++kk) {
        u4 a[TM], b[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) b[j] = fragment<SB_, BN>(tb, wn * TN * 16, j, kk, lane);
#pragma unroll
        for (int i = 0; i < TM; ++i) a[i] = fragment<SA_, BM>(ta, wm * TM * 16, i, kk, lane);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = mma<BF_>(a[i], b[j], acc[i][j]);
      }
      __syncthreads();
    }
  }
};

// Workgroup `id` of tm x tn tiles as (mt, nt): each of the eight XCDs takes a run of them, in bands of eight nt
// tiles (what is read again soon stays in its L2).
__device__ inline void tile_of(int id, int count, int tm, int tn, int& mt, int& nt) {
  const int x = id & 7, q = count / 8, r = count % 8;
  id = x * q + min(x, r) + (id >> 3);
  const int band = id / (8 * tm), first = band * 8, wide = min(8, tn - first), in = id - band * 8 * tm;
  nt = first + in % wide, mt = in / wide;
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
