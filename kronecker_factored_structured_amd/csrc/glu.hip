// The gated Kronecker block, forward and backward:
//   g = x Wg + bg,  u = x Wu + bu,  y = act(g) o u,   W_f = sum_i kron(S_f o A_fi, B_fi)
// Row n of x is a p x m matrix X, and with C_fi = S_f o A_fi (the layer's formulas, twice)
//   Z_fi = X B_fi (p x n),   g, u = sum_i C_fi^T Z_fi (q x n)
//   dg = dy u act'(g),  du = dy act(g);   dX = sum_fi C_fi (d_f B_fi^T)
//   dC_fi = sum_rows Z_fi d_f^T,  dB_fi = sum_rows X^T (C_fi d_f),  dA = S o dC,  dS = sum_i A_i o dC_i
//
// All products run on the bf16 matrix instruction with fp32 accumulation.  A factor wider than
// bf16 is the sum of bf16 parts taken off its top bits (8 + 8 + 8 bits: an fp32 value is exactly
// three), and a product keeps the pairs of parts whose orders sum to at most two: six instructions
// for fp32 times fp32, dropped terms below 2^-21 of the product.  The bf16 instruction has sixteen
// times the rate of the fp32 one, so six of them are still 2.7 times faster; bf16 inputs need
// fewer parts and keep their intermediates exact to fp32 in the backward (its parameter gradients
// are fp32) and to 2^-16 in the forward (its y is bf16).  A non-finite input gives non-finite outputs.
//
// Operand blocks.  The instruction takes 16 (row or column) x 32 (k): lane l = 16 g + c holds
// k-slots 8 g .. 8 g + 7 of row c.  Its result has lane (g, c) holding rows 4 g .. 4 g + 3 of
// column c.  Two results stacked (rows 0..15 and 16..31) are, lane by lane, an operand with
// k-slots {4g..4g+3, 16+4g..16+4g+3} ("chained" order), so Z goes from the first product into the
// second without leaving its registers; the other operand is laid out in the same order.  The
// factors are laid out as such blocks once per call by glu_pack_kernel.
#include <algorithm>
#include <type_traits>

#include "kron_internal.h"
#include "row_tile.h"

namespace kron {
namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

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

// Eight fp32 values (two f4) as NP bf16 operand parts, off the top bits.
template <int NP>
__device__ inline void split(f4 lo, f4 hi, Op* o) {
#pragma unroll
  for (int s = 0; s < NP; ++s) {
    o[s].u[0] = tops(lo[0], lo[1]);
    o[s].u[1] = tops(lo[2], lo[3]);
    o[s].u[2] = tops(hi[0], hi[1]);
    o[s].u[3] = tops(hi[2], hi[3]);
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

// The activation and its derivative.
__device__ inline float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
}
template <bool GRAD>
__device__ inline float activate(int act, float v, float* d) {
  if (act == KRON_ACT_SILU) {
    const float s = sigmoid(v);
    if (GRAD) *d = s * (1.f + v * (1.f - s));
    return v * s;
  }
  if (act == KRON_ACT_GELU) {
    const float c = 0.5f + 0.5f * erff(v * 0.70710678118654752f);
    if (GRAD) *d = c + v * 0.39894228040143268f * __builtin_amdgcn_exp2f(-0.72134752044448170f * v * v);
    return v * c;
  }
  if (act == KRON_ACT_GELU_TANH) {      // 0.5 v (1 + tanh(w)) = v sigmoid(2 w)
    const float a = 0.79788456080286536f, b = 0.044715f;
    const float vv = fminf(v * v, 1e4f);      // (s is 0 or 1 long before; nothing overflows)
    const float s = sigmoid(2.f * a * v * (1.f + b * vv));
    if (GRAD) *d = s + v * s * (1.f - s) * (2.f * a) * (1.f + 3.f * b * vv);
    return v * s;
  }
  if (GRAD) *d = v > 0.f ? 1.f : 0.f;
  return v < 0.f ? 0.f : v;
}

// Of four values: the activation, and its derivative.
template <bool GRAD>
__device__ inline void activate4(int act, const f4& v, f4& out, f4& d) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float t = 0.f;
    out[i] = activate<GRAD>(act, v[i], &t);
    d[i] = t;
  }
}

// ---------------------------------------------------------------------------------
// The factors as operand blocks.  A table holds, for projection f and rank i, the blocks
// [tile of 16 columns][step of 32 k][part], 64 lanes x 16 bytes each.
// ---------------------------------------------------------------------------------
struct PackArgs {
  int p, q, m, n, r;
  int bf16, parts_b, parts_c;
  int tables;             // 2: the forward's, 4: the backward's too
  const void* S;
  const void* A;
  const void* B;
  u4* t[4];               // see GluTables
  int64_t lanes[4];       // lanes of each table (all f, i): tile x step x 64, without parts
};

__device__ inline float raw(const void* t, int64_t i, int bf16) {
  return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)t)[i] << 16) : ((const float*)t)[i];
}
__device__ inline int chained(int g, int e) { return e < 4 ? 4 * g + e : 12 + 4 * g + e; }

__global__ __launch_bounds__(256) void glu_pack_kernel(PackArgs a) {
  int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  int w = 0;
  while (w < a.tables && id >= a.lanes[w]) id -= a.lanes[w++];
  if (w >= a.tables) return;
  // table 0: B, k = m, columns n; 1: C, k = p, columns q; 2: B^T, k = n, columns m; 3: C^T, k = q, columns p
  const int kd = w == 0 ? a.m : w == 1 ? a.p : w == 2 ? a.n : a.q;
  const int cd = w == 0 ? a.n : w == 1 ? a.q : w == 2 ? a.m : a.p;
  const int steps = (kd + 31) / 32, tiles = (cd + 15) / 16;
  const int lane = (int)(id & 63), g = lane >> 4, c = lane & 15;
  int64_t b = id >> 6;
  const int ks = (int)(b % steps);
  b /= steps;
  const int tile = (int)(b % tiles);
  const int fi = (int)(b / tiles), f = fi / a.r;
  const bool isb = (w & 1) == 0;
  const int col = 16 * tile + c;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int k = 32 * ks + (isb ? 8 * g + e : chained(g, e));
    float x = 0.f;
    if (k < kd && col < cd) {
      if (isb) {
        const int mi = w == 0 ? k : col, ni = w == 0 ? col : k;
        x = raw(a.B, ((int64_t)fi * a.m + mi) * a.n + ni, a.bf16);
      } else {
        const int pi = w == 1 ? k : col, qi = w == 1 ? col : k;
        x = raw(a.A, ((int64_t)fi * a.p + pi) * a.q + qi, a.bf16);
        // the product of two bf16 values has 16 bits: exact in fp32 and in two parts
        if (a.S) x *= raw(a.S, ((int64_t)f * a.p + pi) * a.q + qi, a.bf16);
      }
    }
    v[e] = x;
  }
  Op o[3];
  split<3>(f4{v[0], v[1], v[2], v[3]}, f4{v[4], v[5], v[6], v[7]}, o);
  const int parts = isb ? a.parts_b : a.parts_c;
  u4* dst = a.t[w] + (id >> 6) * parts * 64 + lane;
  for (int s = 0; s < parts; ++s) dst[s * 64] = s == 0 ? o[0].u : s == 1 ? o[1].u : o[2].u;
}

// ---------------------------------------------------------------------------------
// Two products for each row: out (q x n) = sum_fi C_fi^T (X_f B_fi), with the gate at its end.
//   MODE 0  y = act(g) o u           MODE 1  dg and du, from dy
//   MODE 2  dX: the same products with X_f = d_f, B^T and C^T, summed over both projections
// A wavefront owns a row and at most two of its n tiles: X in registers as operand parts, out in
// accumulators (4 x 2 tiles of each projection).  The factors' blocks are read from LDS:
//   RES  all of them, put there once; the wavefronts then run through their rows without a barrier, so that
//        one's activations and memory stand beside another's products
//   else one (f, i) at a time through two buffers: the next one's blocks are on their way (global to LDS
//        directly) while this one's are multiplied; a wavefront has one row
// Few rows: the q tiles are spread over gridDim.y workgroups.
// ---------------------------------------------------------------------------------
struct RowsArgs {
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

constexpr int kTiles = 4;       // of 16: sides up to 64

template <bool BF>
__device__ inline float load1(const void* p, int64_t i) {
  return BF ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}

// Four values from i on, of which the first `left` exist; vec: all do and the place is aligned.
template <bool BF>
__device__ inline f4 load4(const void* p, int64_t i, int left, bool vec) {
  f4 r = f4{0.f, 0.f, 0.f, 0.f};
  if (vec) {
    if (!BF) return *reinterpret_cast<const f4*>((const float*)p + i);
    typedef uint32_t u2v __attribute__((ext_vector_type(2)));
    const u2v h = *reinterpret_cast<const u2v*>((const uint16_t*)p + i);
    return f4{bf16_lo(h[0]), bf16_hi(h[0]), bf16_lo(h[1]), bf16_hi(h[1])};
  }
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (v < left) r[v] = load1<BF>(p, i + v);
  return r;
}

// 1 KB (64 lanes x 16 bytes) from global memory into LDS at a wavefront-uniform place.
__device__ inline void block_to_lds(const u4* src_lane, u4* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src_lane,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// What becomes of four accumulated values of q row qi from n0 on (ag; au: the up-projection's).
template <int MODE, bool OBF, int ACT>
__device__ inline void rows_out(const RowsArgs& a, int64_t row, int qi, int n0, f4 ag, f4 au) {
  const int64_t qn = (int64_t)a.q * a.n, at = (int64_t)qi * a.n + n0, o = row * qn + at;
  const bool vec = (a.n & 3) == 0;
  const int left = a.n - n0;
  if (MODE != 2 && a.bias) {
    ag += load4<OBF>(a.bias, at, left, vec);
    au += load4<OBF>(a.bias, qn + at, left, vec);
  }
  if (MODE == 1) {      // (the padding of the workspace's rows gets zero)
    const f4 dy = load4<OBF>(a.dy, o, left, vec);
    f4 dg, du;
    activate4<true>(ACT, ag, du, dg);
    dg *= dy * au;
    du *= dy;
    if (!vec) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (v >= left) dg[v] = du[v] = 0.f;
    }
    const int64_t od = (row * a.q + qi) * a.n4 + n0;
    *reinterpret_cast<f4*>(a.d[0] + od) = dg;
    *reinterpret_cast<f4*>(a.d[1] + od) = du;
    return;
  }
  f4 out = ag;
  if (MODE == 0) {
    f4 unused;
    activate4<false>(ACT, ag, out, unused);
    out *= au;
  }
  if (OBF) {
    uint16_t* y = (uint16_t*)a.y + o;
    const uint32_t h0 = bf16_pair(out[0], out[1]), h1 = bf16_pair(out[2], out[3]);
    if (vec) {
      typedef uint32_t u2v __attribute__((ext_vector_type(2)));
      *reinterpret_cast<u2v*>(y) = u2v{h0, h1};
    } else {
      y[0] = (uint16_t)h0;
      if (left > 1) y[1] = (uint16_t)(h0 >> 16);
      if (left > 2) y[2] = (uint16_t)h1;
      if (left > 3) y[3] = (uint16_t)(h1 >> 16);
    }
  } else {
    float* y = (float*)a.y + o;
    if (vec) {
      *reinterpret_cast<f4*>(y) = out;
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (v < left) y[v] = out[v];
    }
  }
}

// XBF: X is bf16 (one part); else fp32 in NX parts.  OBF: bias, dy and the output are bf16.  W wavefronts.
template <int MODE, bool XBF, bool OBF, int NX, int NB, int NZ, int NC, int LIM, int MK, int PK, int W, bool RES>
__global__ __launch_bounds__(64 * W, W / 4) void glu_rows_kernel(RowsArgs a) {
  constexpr int NF = MODE == 2 ? 1 : 2;
  extern __shared__ u4 lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, c = lane & 15;
  const int QT = (a.q + 15) / 16, NT = (a.n + 15) / 16;
  const int qt0 = QT * blockIdx.y / a.qsplit, qtn = QT * (blockIdx.y + 1) / a.qsplit - qt0;
  const int nbB = NT * MK * NB, nbC = qtn * PK * NC, nb = nbB + nbC;      // blocks of one (f, i)

  auto stage = [&](int fi) {
    u4* dst = lds + (RES ? fi : fi & 1) * nb * 64;
    const u4* sb = a.tb + (int64_t)fi * NT * (MK * NB * 64) + lane;
    const u4* sc = a.tc + (int64_t)(fi * QT + qt0) * (PK * NC * 64) + lane;
    for (int b = wave; b < nb; b += W) block_to_lds(b < nbB ? sb + b * 64 : sc + (b - nbB) * 64, dst + b * 64);
  };
  if (RES) {
    for (int fi = 0; fi < 2 * a.r; ++fi) stage(fi);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  } else {
    stage(0);
  }

  const bool vec = XBF ? (a.ldm & 7) == 0 : (a.ldm & 3) == 0;
  for (int64_t unit = (int64_t)blockIdx.x * W + wave;; unit += (int64_t)gridDim.x * W) {
    const int64_t row = NT > 2 ? unit >> 1 : unit;
    const int nt0 = NT > 2 ? 2 * (int)(unit & 1) : 0, ntn = min(2, NT - nt0);
    const bool live = row < a.N;
    if (RES && !live) return;

    Op xa[PK][2][MK][NX];
    auto load_x = [&](int f) {
#pragma unroll
      for (int pk = 0; pk < PK; ++pk)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int mk = 0; mk < MK; ++mk) {
            const int pi = 32 * pk + 16 * t + c, k = 32 * mk + 8 * g;
            const int64_t at = row * a.ldx + (int64_t)(pi * a.ldm + k);
            const bool in = live && pi < a.p;
            if (XBF) {
              Op o;
              o.u = u4{0u, 0u, 0u, 0u};
              if (in && vec) {
                if (k < a.m) o.u = *reinterpret_cast<const u4*>((const uint16_t*)a.x[f] + at);
              } else if (in) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (k + e < a.m) o.u[e / 2] |= (uint32_t)((const uint16_t*)a.x[f])[at + e] << (16 * (e & 1));
              }
              xa[pk][t][mk][0] = o;
            } else {
              f4 lo = f4{0.f, 0.f, 0.f, 0.f}, hi = lo;
              const float* xp = (const float*)a.x[f] + at;
              if (in && vec) {
                if (k < a.m) lo = *reinterpret_cast<const f4*>(xp);
                if (k + 4 < a.m) hi = *reinterpret_cast<const f4*>(xp + 4);
              } else if (in) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if (k + e < a.m) lo[e] = xp[e];
                  if (k + 4 + e < a.m) hi[e] = xp[4 + e];
                }
              }
              split<NX>(lo, hi, xa[pk][t][mk]);
            }
          }
    };

    f4 acc[NF][kTiles][2];      // [projection][q tile][n tile]
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int t = 0; t < 2; ++t) acc[f][j][t] = f4{0.f, 0.f, 0.f, 0.f};

#pragma unroll
    for (int f = 0; f < 2; ++f) {
      if (f == 0 || MODE == 2) load_x(f);
      for (int i = 0; i < a.r; ++i) {
        const int fi = f * a.r + i;
        if (!RES) {
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // this (f, i)'s blocks have landed
          __syncthreads();                                      // everybody's; and the other buffer has been read
          if (fi + 1 < 2 * a.r) stage(fi + 1);
          if (!live) continue;
        }
        const u4* tc = lds + (RES ? fi : fi & 1) * nb * 64 + nbB * 64 + lane;
        const u4* tb = tc + (nt0 * MK * NB - nbB) * 64;
#pragma unroll
        for (int pk = 0; pk < PK; ++pk) {
          // (both n tiles always, so that no branch stands between the products: beside an odd last one, whatever
          // the next blocks hold goes into accumulators that nothing reads)
          Op zb[2][NZ];
          f4 zt[2][2];
#pragma unroll
          for (int t = 0; t < 2; ++t) zt[t][0] = zt[t][1] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int mk = 0; mk < MK; ++mk) {
            Op b[2][NB];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int s = 0; s < NB; ++s) b[t][s].u = tb[((t * MK + mk) * NB + s) * 64];
#pragma unroll
            for (int o = LIM; o >= 0; --o)
#pragma unroll
              for (int s = 0; s < NX; ++s)
                if (o - s >= 0 && o - s < NB)
#pragma unroll
                  for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) zt[t][h] = mfma(xa[pk][h][mk][s], b[t][o - s], zt[t][h]);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) split<NZ>(zt[t][0], zt[t][1], zb[t]);
          // the q tiles in twos as well (the terms of one order over four products before the next)
#pragma unroll
          for (int j0 = 0; j0 < kTiles; j0 += 2)
            if (j0 < qtn) {
              Op b[2][NC];
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int s = 0; s < NC; ++s) b[j][s].u = tc[(((j0 + j) * PK + pk) * NC + s) * 64];
#pragma unroll
              for (int o = LIM; o >= 0; --o)
#pragma unroll
                for (int s = 0; s < NZ; ++s)
                  if (o - s >= 0 && o - s < NC)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                      for (int t = 0; t < 2; ++t)
                        acc[f % NF][j0 + j][t] = mfma(zb[t][s], b[j][o - s], acc[f % NF][j0 + j][t]);
            }
        }
      }
    }
    if (!live) return;

    auto write = [&](auto act) {
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int qi = 16 * (qt0 + j) + c, n0 = 16 * (nt0 + t) + 4 * g;
          if (j < qtn && t < ntn && qi < a.q && n0 < a.n)
            rows_out<MODE, OBF, decltype(act)::value>(a, row, qi, n0, acc[0][j][t], acc[NF - 1][j][t]);
        }
    };
    if (MODE == 2 || a.act == KRON_ACT_SILU) write(std::integral_constant<int, KRON_ACT_SILU>{});
    else if (a.act == KRON_ACT_GELU) write(std::integral_constant<int, KRON_ACT_GELU>{});
    else if (a.act == KRON_ACT_GELU_TANH) write(std::integral_constant<int, KRON_ACT_GELU_TANH>{});
    else write(std::integral_constant<int, KRON_ACT_RELU>{});
    if (!RES) return;
  }
}

// ---------------------------------------------------------------------------------
// The factors' gradients.  A workgroup has one kind and a group of pairs (f, i):
//   kind 0  dC_fi (p x q) += Z_fi d_f^T, Z_fi = X B_fi       kind 1  dB_fi (m x n) += X^T G_fi, G_fi = C_fi d_f
// Each wavefront owns a pair's sum in registers, with B_fi (or C_fi) beside it; with fewer pairs than
// wavefronts several share a pair and take rows in turn.  A step's rows of X and d_f are split
// into parts once and staged in LDS as operand blocks in the order that the kind contracts over (4 x 4
// patches, which a thread turns in its registers).  Two buffers: while one step is multiplied the next
// is staged, half of the wavefronts staging first and half multiplying first, and the values of the one
// after that are on their way.
//
// Slots of a block are permuted so that neither side has bank conflicts: column c of k-group g stands
// at 16 g + 4 ((c % 4) ^ g) + c / 4.  A wavefront stores columns of one residue mod 4 at a time: their
// quarters of a 256-byte row differ by g.
// ---------------------------------------------------------------------------------
struct ParamArgs {
  int64_t N;
  int p, q, m, n, r, n4;
  int groups[2];           // row groups of each kind
  int pair_groups;
  int rs;                  // rows of a step
  int share;               // wavefronts of a pair
  const void* x;
  const float* d[2];
  const u4* tb;            // B blocks (k = m)
  const u4* tc;            // C^T blocks (k = q)
  float* part[2];          // partial rows: kind 0 dC (2 r p q) | dbias (2 q n), kind 1 dB (2 r m n)
};

// Sizes of a step that both the host and the kernel use.
struct ParamSizes {
  int PT, QT, MT, NT, PK, QK, MK, NK;
  int dk, dpat, xk, xpat;          // patches
  int xa, ya;                      // u4 of a row's X blocks, and of one d_f's
  __host__ __device__ ParamSizes(const ParamArgs& a, int nx, int kind) {
    PT = (a.p + 15) / 16; QT = (a.q + 15) / 16; MT = (a.m + 15) / 16; NT = (a.n + 15) / 16;
    PK = (a.p + 31) / 32; QK = (a.q + 31) / 32; MK = (a.m + 31) / 32; NK = (a.n + 31) / 32;
    dk = a.n4 / 4; dpat = (a.q + 3) / 4 * dk;
    xk = (a.m + 3) / 4; xpat = (a.p + 3) / 4 * xk;
    // [k step][tile][part].  Kind 0: X k = m, p tiles; d_f k = n, q tiles.  Kind 1: X k = p, m tiles; d_f k = q,
    // n tiles.  The tiles of the inner loops (p and n) are made even.
    xa = (kind == 0 ? MK * 2 * PK : PK * MT) * nx * 64;
    ya = (kind == 0 ? NK * QT : QK * 2 * NK) * 3 * 64;
  }
  __host__ __device__ int row(int nf) const { return xa + nf * ya; }
};

// TC: tiles of a side at most (2: all sides up to 32, a fraction of the registers; 4).
template <bool XBF, int NX, int NTAB, int KIND, int TC, int NTH>
__device__ inline void param_body(const ParamArgs& a, int rowgroup, int pairgroup, const u4* table, u4* lds) {
  constexpr int NY = 3, KC = TC / 2;
  constexpr int SLOTS = 1024 / NTH;            // patches of a thread: at most 1024 a step
  constexpr int BS = 512 / NTH;                // of them of d_f: at most 512
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, c = lane & 15;
  const int slot = 16 * g + 4 * ((c & 3) ^ g) + (c >> 2);
  const ParamSizes z(a, NX, KIND);
  const int pairs = 2 * a.r, ppw = (pairs + a.pair_groups - 1) / a.pair_groups, pair0 = pairgroup * ppw;
  const int pairn = min(ppw, pairs - pair0);
  const int f_lo = pair0 / a.r, nf = (pair0 + pairn - 1) / a.r - f_lo + 1;
  const int area = z.row(nf), buf = area * a.rs;
  for (int i = tid; i < 2 * buf; i += NTH) lds[i] = u4{0u, 0u, 0u, 0u};      // the tiles' padding stays zero

  const int pl = wave % ppw, sub = wave / ppw;
  const bool active = pl < pairn && sub < a.share;
  const int fi = pair0 + (active ? pl : 0), f = fi / a.r;
  Op tab[TC][KC][NTAB];    // kind 0: B_fi [NT][MK]; kind 1: C_fi^T [PT][QK]
  const int tabT = KIND == 0 ? z.NT : z.PT, tabK = KIND == 0 ? z.MK : z.QK;
#pragma unroll
  for (int t = 0; t < TC; ++t)
#pragma unroll
    for (int k = 0; k < KC; ++k)
#pragma unroll
      for (int s = 0; s < NTAB; ++s) {
        tab[t][k][s].u = u4{0u, 0u, 0u, 0u};
        if (t < tabT && k < tabK) tab[t][k][s].u = table[((int64_t)((fi * tabT + t) * tabK + k) * NTAB + s) * 64 + lane];
      }
  f4 acc[TC][TC];
#pragma unroll
  for (int i = 0; i < TC; ++i)
#pragma unroll
    for (int j = 0; j < TC; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};

  // patches of a step: those of d_f of all its rows, then those of X
  const int nd = nf * z.dpat, ndall = a.rs * nd, npat = ndall + a.rs * z.xpat;
  float bsum[BS][16];
#pragma unroll
  for (int b = 0; b < BS; ++b)
#pragma unroll
    for (int e = 0; e < 16; ++e) bsum[b][e] = 0.f;
  const bool xvec = (a.m & 3) == 0;
  const int64_t rows = (a.N + a.groups[KIND] - 1) / a.groups[KIND];
  const int64_t r0 = rowgroup * rows, r1 = min(a.N, r0 + rows);

  // This thread's patches: where the rows of each come from (advancing by a step's rows) and where it
  // goes in LDS.  A patch (rows j0.., columns k0..) goes into blocks [k step][tile][part].  Kind 0 contracts
  // along the row, kind 1 down the column; chained order, but X of kind 0 natural (its partner is the packed B).
  struct Patch {
    const char* src;
    int step, stride;      // bytes from one step, one row of the patch, to the next
    int kind;              // 0 none, 1 d_f, 2 X
    int rr, rows, cols;    // row of the step; rows, columns of the patch that exist
    int at, gg;            // LDS place (in 8 bytes, of part 0 and column 0), k-group
  } ps[SLOTS];
  f4 v[SLOTS][4];
  constexpr int XS = XBF ? 2 : 4;
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    const int pt = tid + s * NTH;
    Patch& w = ps[s];
    w.kind = pt < ndall ? 1 : pt < npat ? 2 : 0;
    const bool isd = w.kind != 2;
    const int e = isd ? pt : pt - ndall, per = isd ? nd : z.xpat, dk = isd ? z.dk : z.xk;
    w.rr = e / per;
    const int ff = isd ? (e % per) / z.dpat : 0, o = isd ? (e % per) % z.dpat : e % per;
    const int j0 = 4 * (o / dk), k0 = 4 * (o % dk);
    w.rows = (isd ? a.q : a.p) - j0;
    w.cols = isd ? 4 : a.m - k0;
    w.stride = isd ? a.n4 * 4 : a.m * XS;
    w.step = a.rs * (isd ? a.q * a.n4 * 4 : a.p * a.m * XS);
    w.src = isd ? (const char*)(a.d[f_lo + (w.kind == 1 ? ff : 0)] + ((r0 + w.rr) * a.q + j0) * a.n4 + k0)
                : (const char*)a.x + ((r0 + w.rr) * a.p * a.m + (int64_t)j0 * a.m + k0) * XS;
    const int np = isd ? NY : NX, tiles = isd ? (KIND == 0 ? z.QT : 2 * z.NK) : (KIND == 0 ? 2 * z.PK : z.MT);
    const int kc = KIND == 0 ? k0 : j0, cc = KIND == 0 ? j0 : k0, kk = kc & 31;
    const bool natural = KIND == 0 && !isd;
    w.gg = natural ? kk >> 3 : (kk & 15) >> 2;
    const int h = natural ? (kk >> 2) & 1 : kk >> 4, base = w.rr * area + (isd ? z.xa + ff * z.ya : 0);
    w.at = 2 * (base + (((kc >> 5) * tiles + (cc >> 4)) * np) * 64 + w.gg * 16 + ((cc >> 2) & 3)) + h;
  }
  int64_t next = r0;      // the step that fetch() takes
  auto fetch = [&]() {
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      Patch& w = ps[s];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[s][i] = f4{0.f, 0.f, 0.f, 0.f};
      if (w.kind != 0 && next + w.rr < r1) {
        const bool whole = w.kind == 1 || (xvec && !XBF);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i >= w.rows) continue;
          const char* src = w.src + i * w.stride;
          if (whole) {
            v[s][i] = *reinterpret_cast<const f4*>(src);
          } else if (xvec) {
            typedef uint32_t u2v __attribute__((ext_vector_type(2)));
            const u2v h = *reinterpret_cast<const u2v*>(src);
            v[s][i] = f4{bf16_lo(h[0]), bf16_hi(h[0]), bf16_lo(h[1]), bf16_hi(h[1])};
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (e < w.cols) v[s][i][e] = load1<XBF>(src, e);
          }
        }
      }
      w.src += w.step;
    }
    next += a.rs;
  };
  auto store = [&](int base) {
    typedef uint32_t u2v __attribute__((ext_vector_type(2)));
    u2v* l2 = reinterpret_cast<u2v*>(lds + base);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const Patch& w = ps[s];
      if (w.kind == 0) continue;
      f4 u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) u[i][e] = KIND == 0 ? v[s][i][e] : v[s][e][i];
      if (KIND == 0 && s < BS && w.kind == 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) bsum[s < BS ? s : 0][i] += v[s][i / 4][i % 4];
      }
      const int np = w.kind == 1 ? NY : NX;
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        if (part >= np) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const u2v t = u2v{tops(u[i][0], u[i][1]), tops(u[i][2], u[i][3])};
          l2[w.at + 128 * part + 8 * (i ^ w.gg)] = t;
          if (part < 2) {
            float r0 = u[i][0], r1 = u[i][1], r2 = u[i][2], r3 = u[i][3];
            rest(t[0], r0, r1);
            rest(t[1], r2, r3);
            u[i] = f4{r0, r1, r2, r3};
          }
        }
      }
    }
  };
  // One row's products.  First product: into tile pairs; the inner tiles of the second (p or n) in twos, so
  // that no branch stands between the products (an odd one's blocks are zero).
  auto multiply = [&](auto count, const u4* xl, const u4* yl) {
    constexpr int TI = decltype(count)::value;
    const int steps = KIND == 0 ? z.NK : z.PK;
#pragma unroll
    for (int ko = 0; ko < KC; ++ko)
      if (ko < steps) {
        Op h[TI][3];
#pragma unroll
        for (int t = 0; t < TI; ++t) {
          f4 w[2];
          w[0] = w[1] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < KC; ++k)
            if (k < tabK) {
              if (KIND == 0) {
                Op x[NX];
#pragma unroll
                for (int s = 0; s < NX; ++s) x[s].u = xl[k * 2 * z.PK * NX * 64 + (t * NX + s) * 64];
#pragma unroll
                for (int u = 0; u < 2; ++u) w[u] = dot<NTAB, NX, 2>(tab[2 * ko + u][k], x, w[u]);
              } else {
                Op y[NY];
#pragma unroll
                for (int s = 0; s < NY; ++s) y[s].u = yl[k * 2 * z.NK * NY * 64 + (t * NY + s) * 64];
#pragma unroll
                for (int u = 0; u < 2; ++u) w[u] = dot<NTAB, NY, 2>(tab[2 * ko + u][k], y, w[u]);
              }
            }
          split<3>(w[0], w[1], h[t]);
        }
        const int outer = KIND == 0 ? z.QT : z.MT;
#pragma unroll
        for (int t = 0; t < TC; ++t)
          if (t < outer) {
            constexpr int NO = KIND == 0 ? NY : NX;
            Op y[NO];
#pragma unroll
            for (int s = 0; s < NO; ++s)
              y[s].u = KIND == 0 ? yl[ko * z.QT * NY * 64 + (t * NY + s) * 64] : xl[ko * z.MT * NX * 64 + (t * NX + s) * 64];
#pragma unroll
            for (int o = 2; o >= 0; --o)
#pragma unroll
              for (int s = 0; s <= o; ++s)
                if (o - s < NO)
#pragma unroll
                  for (int i = 0; i < TI; ++i) {
                    if (KIND == 0) acc[i][t] = mfma(h[i][s], y[o - s], acc[i][t]);
                    if (KIND == 1) acc[t][i] = mfma(y[o - s], h[i][s], acc[t][i]);
                  }
          }
      }
  };
  auto work = [&](int base) {
    if (!active) return;
#pragma unroll 1
    for (int rr = sub; rr < a.rs; rr += a.share) {
      const u4* xl = lds + base + rr * area + slot;
      const u4* yl = xl + z.xa + (f - f_lo) * z.ya;
      if constexpr (TC == 4) {
        if ((KIND == 0 ? z.PT : z.NT) > 2)
          multiply(std::integral_constant<int, 4>{}, xl, yl);
        else
          multiply(std::integral_constant<int, 2>{}, xl, yl);
      } else {
        multiply(std::integral_constant<int, 2>{}, xl, yl);
      }
    }
  };

  fetch();
  __syncthreads();
  store(0);
  fetch();
  __syncthreads();
  int cur = 0;
  const bool late = wave >= NTH / 128;      // (the second wavefront of a SIMD)
  for (int64_t step = r0; step < r1; step += a.rs) {
    if (late) work(cur);
    if (step + a.rs < r1) store(buf - cur);
    if (step + 2 * a.rs < r1) fetch();
    if (!late) work(cur);
    cur = buf - cur;
    __syncthreads();
  }

  // partial rows: one for each wavefront of a pair
  const int64_t mn = (int64_t)a.m * a.n, pq = (int64_t)a.p * a.q;
  const int64_t prow = (int64_t)rowgroup * a.share, prows = (int64_t)a.groups[KIND] * a.share;
  const PartRow out{a.part[KIND], prows, prow + (active ? sub : 0), 0};
  if (active) {
    const int R = KIND == 0 ? a.p : a.m, Cn = KIND == 0 ? a.q : a.n;
    const int64_t base = KIND == 0 ? fi * pq : fi * mn;
#pragma unroll
    for (int i = 0; i < TC; ++i)
#pragma unroll
      for (int j = 0; j < TC; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ri = 16 * i + 4 * g + e, ci = 16 * j + c;
          if (ri < R && ci < Cn) out[base + (int64_t)ri * Cn + ci] = acc[i][j][e];
        }
  }
  if (KIND != 0) return;
  // dbias: the sums of a step's rows are joined in LDS (row 0's threads first: a fixed order)
  float* bl = reinterpret_cast<float*>(lds);
  for (int rr = 0; rr < a.rs; ++rr) {
#pragma unroll
    for (int s = 0; s < BS; ++s) {
      const int pt = tid + s * NTH;
      if (pt < ndall && pt / nd == rr) {
#pragma unroll
        for (int e = 0; e < 16; ++e) bl[(pt % nd) * 16 + e] = bsum[s][e] + (rr ? bl[(pt % nd) * 16 + e] : 0.f);
      }
    }
    __syncthreads();
  }
  for (int i = tid; i < nd * 16; i += NTH) {
    const int e = i >> 4, ff = f_lo + e / z.dpat, o = e % z.dpat;
    const int j = 4 * (o / z.dk) + ((i >> 2) & 3), k = 4 * (o % z.dk) + (i & 3);
    // (the workgroup with the projection's first pair; its other partial rows have nothing to add)
    if (ff * a.r >= pair0 && ff * a.r < pair0 + pairn && j < a.q && k < a.n)
      for (int w = 0; w < a.share; ++w) {
        const PartRow ow{a.part[0], prows, prow + w, 0};
        ow[pairs * pq + (int64_t)ff * a.q * a.n + (int64_t)j * a.n + k] = w == 0 ? bl[i] : 0.f;
      }
  }
}

template <bool XBF, int NX, int NB, int NC, int TC, int NTH>
__global__ __launch_bounds__(NTH) void glu_param_kernel(ParamArgs a) {
  extern __shared__ u4 lds[];
  int b = blockIdx.x;
  const int n0 = a.groups[0] * a.pair_groups;
  if (b < n0) {
    param_body<XBF, NX, NB, 0, TC, NTH>(a, b / a.pair_groups, b % a.pair_groups, a.tb, lds);
  } else {
    b -= n0;
    param_body<XBF, NX, NC, 1, TC, NTH>(a, b / a.pair_groups, b % a.pair_groups, a.tc, lds);
  }
}

// ---------------------------------------------------------------------------------
// The partial rows summed in 64 bits in a fixed order, and dA = S o dC, dS = sum_i A_i o dC_i from dC.  A
// workgroup has a block of 32 columns (part_index): of dB, of dbias, or with S of dC's e-th elements of
// every rank.
// ---------------------------------------------------------------------------------
struct ReduceArgs {
  const float* part[2];
  int rows[2];             // partial rows of each kind
  int nB, nC, nbias;       // columns: dB, dC, dbias
  int pq, r, bf16;
  const void* S;
  const void* A;
  float* dB;
  float* dA;
  float* dS;
  float* dbias;
};

// Sum over `rows` of column c0 + col (32 consecutive ones; they may cross a block's end): thread (col, y).
__device__ inline double column_sum(const float* part, int rows, int64_t column, bool in, int y, double (*red)[33],
                                    int col) {
  double s0 = 0.0, s1 = 0.0;
  if (in) {
    const float* src = part + part_index(rows, 0, column);
    int g = y;
    for (; g + 8 < rows; g += 16) {
      const float u = src[(int64_t)g * kRedCols], w = src[(int64_t)(g + 8) * kRedCols];
      s0 += (double)u;
      s1 += (double)w;
    }
    if (g < rows) s0 += (double)src[(int64_t)g * kRedCols];
  }
  __syncthreads();
  red[y][col] = s0 + s1;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) t += red[i][col];
  return t;
}

__global__ __launch_bounds__(256) void glu_reduce_kernel(ReduceArgs a) {
  __shared__ double red[8][33];
  const int col = threadIdx.x & 31, y = threadIdx.x >> 5;
  int b = blockIdx.x;
  const int bB = (a.nB + 31) / 32, bb = a.dbias ? (a.nbias + 31) / 32 : 0;
  if (b < bB) {
    const int c = 32 * b + col;
    const double t = column_sum(a.part[1], a.rows[1], c, c < a.nB, y, red, col);
    if (y == 0 && c < a.nB) a.dB[c] = (float)t;
    return;
  }
  b -= bB;
  if (b < bb) {
    const int c = 32 * b + col;
    const double t = column_sum(a.part[0], a.rows[0], a.nC + c, c < a.nbias, y, red, col);
    if (y == 0 && c < a.nbias) a.dbias[c] = (float)t;
    return;
  }
  b -= bb;
  if (!a.S) {
    const int c = 32 * b + col;
    const double t = column_sum(a.part[0], a.rows[0], c, c < a.nC, y, red, col);
    if (y == 0 && c < a.nC) a.dA[c] = (float)t;
    return;
  }
  const int per = (a.pq + 31) / 32, f = b / per, e = 32 * (b % per) + col;
  const bool in = e < a.pq;
  const float s = in ? raw(a.S, (int64_t)f * a.pq + e, a.bf16) : 0.f;
  double ds = 0.0;
  for (int i = 0; i < a.r; ++i) {
    const int64_t c = ((int64_t)f * a.r + i) * a.pq + e;
    const double t = column_sum(a.part[0], a.rows[0], c, in, y, red, col);
    if (y == 0 && in) {
      a.dA[c] = (float)((double)s * t);
      ds += (double)raw(a.A, c, a.bf16) * t;
    }
  }
  if (y == 0 && in) a.dS[(int64_t)f * a.pq + e] = (float)ds;
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

struct Sizes {
  int parts_b, parts_c;
  int64_t lanes[4], bytes[4];
  int n4, groups[2], waves, share, pair_groups;
  bool small;
  int64_t off_d, off_part[2], fwd_bytes, bwd_bytes;
};

Sizes sizes_of(const GluArgs& a) {
  Sizes z{};
  z.parts_b = a.bf16 ? 1 : 3;
  z.parts_c = a.bf16 ? (a.S ? 2 : 1) : 3;
  const int dims[4][2] = {{a.m, a.n}, {a.p, a.q}, {a.n, a.m}, {a.q, a.p}};
  int64_t off = 0;
  for (int t = 0; t < 4; ++t) {
    z.lanes[t] = (int64_t)2 * a.r * ceil_div(dims[t][0], 32) * ceil_div(dims[t][1], 16) * 64;
    z.bytes[t] = z.lanes[t] * 16 * ((t & 1) ? z.parts_c : z.parts_b);
    off += z.bytes[t];
    if (t == 1) z.fwd_bytes = off;
  }
  z.n4 = (a.n + 3) & ~3;
  z.off_d = (off + 255) & ~int64_t(255);
  z.off_part[0] = z.off_d + ((2 * a.N * a.q * z.n4 * 4 + 255) & ~int64_t(255));
  // The parameters' kernel: eight wavefronts; four for fp32 with a side over 32, whose parts take the registers
  // of two.  One workgroup a CU, the kinds' numbers of them by their numbers of products, each with at least
  // four rows where there are that many.
  z.small = std::max(std::max(a.p, a.q), std::max(a.m, a.n)) <= 32;
  z.waves = !z.small && !a.bf16 ? 4 : 8;
  z.share = 1;
  while (2 * z.share * 2 * a.r <= z.waves) z.share *= 2;
  z.pair_groups = ceil_div(2 * a.r, z.waves / z.share);
  const int PT = ceil_div(a.p, 16), QT = ceil_div(a.q, 16), MT = ceil_div(a.m, 16), NT = ceil_div(a.n, 16);
  const int PK = ceil_div(a.p, 32), QK = ceil_div(a.q, 32), MK = ceil_div(a.m, 32), NK = ceil_div(a.n, 32);
  const int tb = a.bf16 ? 1 : 6, tc = a.bf16 ? (a.S ? 5 : 3) : 6, tx = a.bf16 ? 3 : 6;      // instructions of a product
  const double w0 = PT * 2 * NK * MK * tb + PT * QT * NK * 6, w1 = 2 * PK * NT * QK * tc + MT * NT * PK * tx;
  const int total = std::max(2, 256 / z.pair_groups);
  const int64_t most = (a.N + 3) / 4;
  z.groups[0] = std::min(std::max((int)(total * w0 / (w0 + w1) + 0.5), 1), total - 1);
  z.groups[1] = total - z.groups[0];
  for (int k = 0; k < 2; ++k) z.groups[k] = (int)std::max<int64_t>(1, std::min<int64_t>(z.groups[k], most));
  const int64_t PW0 = (int64_t)2 * a.r * a.p * a.q + 2 * a.q * a.n, PW1 = (int64_t)2 * a.r * a.m * a.n;
  z.off_part[1] = z.off_part[0] + ((part_floats(z.groups[0] * z.share, PW0) * 4 + 255) & ~int64_t(255));
  z.bwd_bytes = z.off_part[1] + part_floats(z.groups[1] * z.share, PW1) * 4;
  return z;
}

hipError_t launch_pack(const GluArgs& a, const Sizes& z, int tables, u4* const t[4], hipStream_t s) {
  PackArgs k{a.p, a.q, a.m, a.n, a.r, a.bf16, z.parts_b, z.parts_c, tables, a.S, a.A, a.B, {}, {}};
  int64_t total = 0;
  for (int i = 0; i < tables; ++i) {
    k.t[i] = t[i];
    k.lanes[i] = z.lanes[i];
    total += z.lanes[i];
  }
  hipLaunchKernelGGL(glu_pack_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, s, k);
  return hipGetLastError();
}

constexpr size_t kLds = 160 * 1024;

template <auto kernel, int W>
hipError_t launch_rows_g(const RowsArgs& k, int64_t groups, size_t lds, hipStream_t s) {
  static const hipError_t attr =
      hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)kLds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(kernel, dim3((unsigned)groups, (unsigned)k.qsplit), dim3(64 * W), lds, s, k);
  return hipGetLastError();
}

template <int MODE, bool XBF, bool OBF, int NX, int NB, int NZ, int NC, int LIM, int MK, int PK>
hipError_t launch_rows_k(RowsArgs k, hipStream_t s) {
  // wavefronts of a workgroup that has a CU to itself: as many as the parts leave registers for
  constexpr int WR = NX == 3 ? (MK * PK == 4 ? 8 : 12) : NZ == 3 && MK * PK == 4 ? 12 : 16;
  constexpr int WS = 8;
  const int NT = ceil_div(k.n, 16), QT = ceil_div(k.q, 16);
  const int64_t units = k.N * (NT > 2 ? 2 : 1);
  // few rows: the q tiles of a row are spread until there are 256 workgroups
  k.qsplit = 1;
  while (k.qsplit < QT && (units + WS - 1) / WS * k.qsplit < 256) ++k.qsplit;
  // the blocks of one (f, i); those beside an odd last tile are read too
  const size_t one = (size_t)(NT * MK * NB + ceil_div(QT, k.qsplit) * PK * NC) * 1024, over = (MK * NB + PK * NC) * 1024;
  const size_t all = 2 * k.r * one + over;
  if (all <= kLds && units > 256 * WS)
    return launch_rows_g<glu_rows_kernel<MODE, XBF, OBF, NX, NB, NZ, NC, LIM, MK, PK, WR, true>, WR>(
        k, std::min<int64_t>(256, (units + WR - 1) / WR), all, s);
  return launch_rows_g<glu_rows_kernel<MODE, XBF, OBF, NX, NB, NZ, NC, LIM, MK, PK, WS, false>, WS>(
      k, (units + WS - 1) / WS, 2 * one + over, s);
}

template <int MODE, bool XBF, bool OBF, int NX, int NB, int NZ, int NC, int LIM>
hipError_t launch_rows(const RowsArgs& k, hipStream_t s) {
  if (k.m <= 32)
    return k.p <= 32 ? launch_rows_k<MODE, XBF, OBF, NX, NB, NZ, NC, LIM, 1, 1>(k, s)
                     : launch_rows_k<MODE, XBF, OBF, NX, NB, NZ, NC, LIM, 1, 2>(k, s);
  return k.p <= 32 ? launch_rows_k<MODE, XBF, OBF, NX, NB, NZ, NC, LIM, 2, 1>(k, s)
                   : launch_rows_k<MODE, XBF, OBF, NX, NB, NZ, NC, LIM, 2, 2>(k, s);
}

template <bool XBF, int NX, int NB, int NC, int TC, int NTH>
hipError_t launch_param_k(const ParamArgs& k, size_t lds, hipStream_t s) {
  constexpr auto kernel = glu_param_kernel<XBF, NX, NB, NC, TC, NTH>;
  static const hipError_t attr =
      hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)kLds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(kernel, dim3((unsigned)((k.groups[0] + k.groups[1]) * k.pair_groups)), dim3(NTH), lds, s, k);
  return hipGetLastError();
}

template <bool XBF, int NX, int NB, int NC>
hipError_t launch_param(ParamArgs k, const Sizes& sz, hipStream_t s) {
  k.share = sz.share;
  k.pair_groups = sz.pair_groups;
  for (int i = 0; i < 2; ++i) k.groups[i] = sz.groups[i];
  const int ppw = ceil_div(2 * k.r, sz.pair_groups);
  int nf = 1;      // most projections of a workgroup
  for (int y = 0; y < sz.pair_groups; ++y)
    if ((std::min(2 * k.r, (y + 1) * ppw) - 1) / k.r != y * ppw / k.r) nf = 2;
  // as many rows a step as two LDS buffers and the threads' slots hold (but no more than four a wavefront)
  const ParamSizes z0(k, NX, 0), z1(k, NX, 1);
  const size_t one = (size_t)std::max(z0.row(nf), z1.row(nf)) * 16;
  const int nd = nf * z0.dpat, np = nd + z0.xpat;
  const int64_t rows = (k.N + k.groups[0] - 1) / k.groups[0];
  k.rs = 1;
  while (k.rs < 4 * k.share && k.rs < rows && 2 * (k.rs + 1) * one <= kLds && (k.rs + 1) * nd <= 512 &&
         (k.rs + 1) * np <= 1024)
    ++k.rs;
  // (dbias is joined in the same LDS: 64 bytes a patch of d_f)
  const size_t lds = std::max(2 * one * k.rs, (size_t)nd * 64);
  if (sz.small) return launch_param_k<XBF, NX, NB, NC, 2, 512>(k, lds, s);
  return launch_param_k<XBF, NX, NB, NC, 4, XBF ? 512 : 256>(k, lds, s);
}

}  // namespace

size_t glu_workspace_bytes(const GluArgs& a, bool backward) {
  const Sizes z = sizes_of(a);
  return (size_t)(backward ? z.bwd_bytes : z.fwd_bytes);
}

hipError_t launch_glu_fwd(const GluArgs& a, void* ws, hipStream_t s) {
  const Sizes z = sizes_of(a);
  u4* t[4] = {(u4*)ws, (u4*)((char*)ws + z.bytes[0]), nullptr, nullptr};
  hipError_t e = launch_pack(a, z, 2, t, s);
  if (e != hipSuccess) return e;
  RowsArgs k{};
  k.N = a.N; k.p = a.p; k.q = a.q; k.m = a.m; k.n = a.n; k.r = a.r;
  k.ldm = a.m; k.ldx = (int64_t)a.p * a.m; k.act = a.act;
  k.x[0] = k.x[1] = a.x; k.tb = t[0]; k.tc = t[1]; k.bias = a.bias; k.y = a.y; k.n4 = z.n4;
  if (!a.bf16) return launch_rows<0, false, false, 3, 3, 3, 3, 2>(k, s);
  return a.S ? launch_rows<0, true, true, 1, 1, 2, 2, 1>(k, s) : launch_rows<0, true, true, 1, 1, 2, 1, 1>(k, s);
}

hipError_t launch_glu_bwd(const GluArgs& a, void* ws, hipStream_t s) {
  const Sizes z = sizes_of(a);
  char* w = (char*)ws;
  u4* t[4];
  for (int i = 0; i < 4; ++i) {
    t[i] = (u4*)w;
    w += z.bytes[i];
  }
  float* d = (float*)((char*)ws + z.off_d);
  hipError_t e = launch_pack(a, z, 4, t, s);
  if (e != hipSuccess) return e;
  float* d2 = d + a.N * a.q * z.n4;
  if (a.N > 0) {
    RowsArgs k{};
    k.N = a.N; k.p = a.p; k.q = a.q; k.m = a.m; k.n = a.n; k.r = a.r;
    k.ldm = a.m; k.ldx = (int64_t)a.p * a.m; k.act = a.act;
    k.x[0] = k.x[1] = a.x; k.tb = t[0]; k.tc = t[1]; k.bias = a.bias; k.dy = a.dy;
    k.d[0] = d; k.d[1] = d2; k.n4 = z.n4;
    if (!a.bf16) e = launch_rows<1, false, false, 3, 3, 3, 3, 2>(k, s);
    else if (a.S) e = launch_rows<1, true, true, 1, 1, 3, 2, 2>(k, s);
    else e = launch_rows<1, true, true, 1, 1, 3, 1, 2>(k, s);
    if (e != hipSuccess) return e;
    if (a.dx) {
      RowsArgs x{};
      x.N = a.N; x.p = a.q; x.q = a.p; x.m = a.n; x.n = a.m; x.r = a.r;
      x.ldm = z.n4; x.ldx = (int64_t)a.q * z.n4; x.n4 = (a.m + 3) & ~3;
      x.x[0] = d; x.x[1] = d2; x.tb = t[2]; x.tc = t[3]; x.y = a.dx;
      if (!a.bf16) e = launch_rows<2, false, false, 3, 3, 3, 3, 2>(x, s);
      else if (a.S) e = launch_rows<2, false, true, 2, 1, 2, 2, 1>(x, s);
      else e = launch_rows<2, false, true, 2, 1, 2, 1, 1>(x, s);
      if (e != hipSuccess) return e;
    }
  }
  ParamArgs k{};
  k.N = a.N; k.p = a.p; k.q = a.q; k.m = a.m; k.n = a.n; k.r = a.r; k.n4 = z.n4;
  k.x = a.x; k.d[0] = d; k.d[1] = d2; k.tb = t[0]; k.tc = t[3];
  for (int i = 0; i < 2; ++i) k.part[i] = (float*)((char*)ws + z.off_part[i]);
  if (!a.bf16) e = launch_param<false, 3, 3, 3>(k, z, s);
  else if (a.S) e = launch_param<true, 1, 1, 2>(k, z, s);
  else e = launch_param<true, 1, 1, 1>(k, z, s);
  if (e != hipSuccess) return e;
  ReduceArgs ra{};
  for (int i = 0; i < 2; ++i) {
    ra.part[i] = k.part[i];
    ra.rows[i] = z.groups[i] * z.share;
  }
  ra.pq = a.p * a.q; ra.r = a.r; ra.bf16 = a.bf16;
  ra.nB = 2 * a.r * a.m * a.n; ra.nC = 2 * a.r * ra.pq; ra.nbias = 2 * a.q * a.n;
  ra.S = a.S; ra.A = a.A; ra.dB = a.dB; ra.dA = a.dA; ra.dS = a.dS; ra.dbias = a.dbias;
  const int blocks = ceil_div(ra.nB, 32) + (a.dbias ? ceil_div(ra.nbias, 32) : 0) +
                     (a.S ? 2 * ceil_div(ra.pq, 32) : ceil_div(ra.nC, 32));
  hipLaunchKernelGGL(glu_reduce_kernel, dim3((unsigned)blocks), dim3(256), 0, s, ra);
  return hipGetLastError();
}

}  // namespace kron
