// What the gated Kronecker block's sources share (glu.hip, glu_rows.hip, glu_param.hip): operand parts and
// blocks of the bf16 matrix instruction, and the kernels' arguments.
//
// All products run on the bf16 matrix instruction with fp32 accumulation.  A factor wider than
// bf16 is the sum of bf16 parts.  Of three the first is cut off the top bits (rounded, values next to fp32's
// largest would be infinite) and the second rounded to nearest, which leaves less than 2^-7, at most 2^-16
// of either sign, and nothing: an fp32 value is exactly three.  A product keeps the pairs of parts whose orders sum
// to at most two: six instructions for fp32 times fp32, dropped terms below 2^-22 of the product.  The bf16
// instruction has sixteen times the rate of the fp32 one, so six of them are still 2.7 times faster; bf16 inputs
// need fewer parts and keep their intermediates exact to fp32 in the backward (its parameter gradients are
// fp32).  What a bf16 y or dX is summed from has two parts, each rounded to nearest: off by at most
// 2^-17 either way (off the top bits they left up to 2^-15, always toward zero), and products of two such
// values keep all four terms.  A non-finite input gives non-finite outputs, and so does such an
// intermediate within half a bf16 step of fp32's largest value.
//
// Operand blocks.  The instruction takes 16 (row or column) x 32 (k): lane l = 16 g + c holds
// k-slots 8 g .. 8 g + 7 of row c.  Its result has lane (g, c) holding rows 4 g .. 4 g + 3 of
// column c.  Two results stacked (rows 0..15 and 16..31) are, lane by lane, an operand with
// k-slots {4g..4g+3, 16+4g..16+4g+3} ("chained" order), so Z goes from the first product into the
// second without leaving its registers; the other operand is laid out in the same order.  The
// factors are laid out as such blocks once per call by glu_pack_kernel.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kron_internal.h"
#include "row_tile.h"

namespace kron {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

struct GluRows {
  int64_t N;
  int p, q, m, n, r;       // of these products (MODE 2: q, p, n, m of the layer)
  int ldm;                 // elements from one row of X_f to the next
  int64_t ldx;             // elements from one X to the next
  int act;
  int qsplit;              // workgroups that share the q tiles
  const void* x[2];
  const u4* tb;            // B blocks
  const u4* tc;            // C blocks
  const void* bias;        // 2 x q n, or NULL
  const void* dy;
  void* y;
  float* d[2];             // dg, du: rows of q x n4
  int n4;
};

struct GluParam {
  int64_t N;
  int p, q, m, n, r, n4;
  int groups[2];           // row groups of each kind
  int pair_groups;         // workgroups that share the pairs
  int rs;                  // rows of a step (set by launch_glu_param)
  int share;               // wavefronts of a pair
  int add;                 // to the partial rows of the launch before (set by launch_glu_param)
  const void* x;
  const float* d[2];
  const u4* tb;            // B blocks (k = m)
  const u4* tc;            // C^T blocks (k = q)
  float* part[2];          // partial rows: kind 0 dC (2 r p q) | dbias (2 q n), kind 1 dB (2 r m n)
};

hipError_t launch_glu_rows0(const GluRows& k, bool bf16, bool with_S, hipStream_t s);      // y
hipError_t launch_glu_rows1(const GluRows& k, bool bf16, bool with_S, hipStream_t s);      // dg, du
hipError_t launch_glu_rows2(const GluRows& k, bool bf16, bool with_S, hipStream_t s);      // dX
hipError_t launch_glu_param_f32(const GluParam& k, hipStream_t s);
hipError_t launch_glu_param_bf16(const GluParam& k, hipStream_t s);
hipError_t launch_glu_param_bf16_S(const GluParam& k, hipStream_t s);
// Wavefronts of a workgroup of the parameters' kernel: eight, four where the sums and parts of sides over 32
// (p, n, q or m) take the registers of two.
constexpr int param_waves(bool bf16, bool p, bool n, bool qm) {
  return qm && (bf16 ? p && n : p || n) ? 4 : 8;
}

namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

union Op {        // an operand block's registers
  u4 u;
  bf8 b;
};

__device__ inline f4 mfma(const Op& a, const Op& b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.b, b.b, c, 0, 0, 0);
}
// the top halves of a (low) and b (high)
__device__ inline uint32_t tops(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
// What the bf16 parts in `t` (a's low, b's high) leave of a and b: exact, in one instruction each, as a
// two-term product whose other factor is 0.  (The pairs (-1, 0) and (0, -1) come from registers: as a
// constant of the instruction 0x0000bf80 stands for both halves.)
__device__ inline void rest(uint32_t t, float& a, float& b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  uint32_t lo = 0x0000bf80u, hi = 0xbf800000u;
  asm("" : "+s"(lo), "+s"(hi));
  a = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, t), __builtin_bit_cast(b2, lo), a, false);
  b = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, t), __builtin_bit_cast(b2, hi), b, false);
}

// The s-th of `of` bf16 parts of a (low) and b (high): rounded to nearest, but the first of three cut off the top bits.
__device__ inline uint32_t part(int s, int of, float a, float b) {
  return s == 0 && of == 3 ? tops(a, b) : bf16_pair(a, b);
}
// Eight fp32 values (two f4) as NP bf16 operand parts.
template <int NP>
__device__ inline void split(f4 lo, f4 hi, Op* o) {
#pragma unroll
  for (int s = 0; s < NP; ++s) {
    o[s].u[0] = part(s, NP, lo[0], lo[1]);
    o[s].u[1] = part(s, NP, lo[2], lo[3]);
    o[s].u[2] = part(s, NP, hi[0], hi[1]);
    o[s].u[3] = part(s, NP, hi[2], hi[3]);
    if (s + 1 < NP) {
      float l[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
      for (int v = 0; v < 4; ++v) rest(o[s].u[v], l[2 * v], l[2 * v + 1]);
      lo = f4{l[0], l[1], l[2], l[3]};
      hi = f4{l[4], l[5], l[6], l[7]};
    }
  }
}

// c += a b over the pairs of parts of order at most LIM, smallest first
template <int NA, int NB, int LIM>
__device__ inline f4 dot(const Op* a, const Op* b, f4 c) {
#pragma unroll
  for (int o = LIM; o >= 0; --o)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (o - i >= 0 && o - i < NB) c = mfma(a[i], b[o - i], c);
  return c;
}

template <bool BF>
__device__ inline float load1(const void* p, int64_t i) {
  return BF ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

constexpr size_t kLds = 160 * 1024;

// Lets a kernel have all of a CU's LDS, once for each device.
template <auto kernel>
hipError_t allow_lds() {
  static std::atomic<uint64_t> done{0};
  int device = 0;
  hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return e;
  const uint64_t bit = uint64_t(1) << (device & 63);
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)kLds);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace
}  // namespace kron
