// The gated Kronecker block's products by rows (see glu_parts.h for the operands).
//
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
//
// Why in registers and LDS: nothing but X and the outputs passes through memory.  8192 x (1024 -> 4096) bf16, r = 4:
// at the rate of a large library product (1206 TFLOP/s) the formula's work is 21 us and the 320 products a row that are
// made of it (42.9 GFLOP: Z in two parts) 36; the bytes need 17.  Measured 51 us (506 TFLOP/s of the formula's work);
// streamed factors took 64.  What bounds it, by counters: the matrix cores are busy 0.34 of the time, and vector
// instructions (Z's parts, the activation, y) fill another 0.34; they alternate in a wavefront, which waits a quarter
// of its time, and four wavefronts a SIMD overlap them in part.
// 3001 x (750 -> 2021) fp32, r = 3: 48 us; six products for one and sides of 25, 43, 30 and 47 in tiles make 42.5 GFLOP
// of 3.1 (35 us at that rate); matrix 0.34, vector 0.26.
// MODE 1 and 2 (8192 x (768 -> 2048) bf16): 57 and 44 us, of which the fp32 dg, du in the workspace (134 MB
// written, then read) take 27 and 27 at the rate of a large copy; MODE 1 waits 0.70 of its time for them.
//
// Compiled once for each MODE (KRON_GLU_MODE).
#include "glu_parts.h"

namespace kron {
namespace {

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

constexpr int kTiles = 4;       // of 16: sides up to 64

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
__device__ inline void rows_out(const GluRows& a, int64_t row, int qi, int n0, f4 ag, f4 au) {
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
__global__ __launch_bounds__(64 * W, W / 4) void glu_rows_kernel(GluRows a) {
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
  // pairs of units (a row's two, or two rows) go round the workgroups, so that few rows are spread over the CUs
  for (int64_t unit = 2 * ((int64_t)(wave >> 1) * gridDim.x + blockIdx.x) + (wave & 1);; unit += (int64_t)gridDim.x * W) {
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

template <auto kernel, int W>
hipError_t launch_rows_g(const GluRows& k, int64_t groups, size_t lds, hipStream_t s) {
  const hipError_t e = allow_lds<kernel>();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3((unsigned)groups, (unsigned)k.qsplit), dim3(64 * W), lds, s, k);
  return hipGetLastError();
}

template <int MODE, bool XBF, bool OBF, int NX, int NB, int NZ, int NC, int LIM, int MK, int PK>
hipError_t launch_rows_k(GluRows k, hipStream_t s) {
  // wavefronts of a workgroup that has a CU to itself: as many as the parts leave registers for (X, the
  // accumulators and the parts of Z: 128 registers hold one bf16 part, 168 three fp32 ones of sides up to 32)
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
  // Resident wherever they fit.  (Streamed, 2048 rows of 32 x 32 fp32 factors take 23 + 18 us for dg, du and dX, resident
  // 21 + 16.5; 61 rows of 9 x 17 and 11 x 13 9 + 8, resident 7.7 + 6.8; r = 4 of 64 x 64 fp32 does not fit.)
  if (all <= kLds)
    return launch_rows_g<glu_rows_kernel<MODE, XBF, OBF, NX, NB, NZ, NC, LIM, MK, PK, WR, true>, WR>(
        k, std::min<int64_t>(std::max(1, 256 / k.qsplit), (units + 1) / 2), all, s);
  // a grid has less than 2^32 threads: more rows take several launches
  constexpr int64_t kMost = int64_t(1) << 24;
  for (int64_t r0 = 0; r0 < k.N; r0 += kMost) {
    GluRows part = k;
    const int64_t out = r0 * k.q * k.n * (OBF ? 2 : 4);
    part.N = std::min(kMost, k.N - r0);
    for (int f = 0; f < 2; ++f) {
      part.x[f] = (const char*)k.x[f] + r0 * k.ldx * (XBF ? 2 : 4);
      if (MODE == 1) part.d[f] = k.d[f] + r0 * k.q * k.n4;
    }
    if (MODE == 1) part.dy = (const char*)k.dy + out;
    else part.y = (char*)k.y + out;
    const int64_t groups = (part.N * (NT > 2 ? 2 : 1) + WS - 1) / WS;
    const hipError_t e = launch_rows_g<glu_rows_kernel<MODE, XBF, OBF, NX, NB, NZ, NC, LIM, MK, PK, WS, false>, WS>(
        part, groups, 2 * one + over, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int MODE, bool XBF, bool OBF, int NX, int NB, int NZ, int NC, int LIM>
hipError_t launch_rows(const GluRows& k, hipStream_t s) {
  if (k.m <= 32)
    return k.p <= 32 ? launch_rows_k<MODE, XBF, OBF, NX, NB, NZ, NC, LIM, 1, 1>(k, s)
                     : launch_rows_k<MODE, XBF, OBF, NX, NB, NZ, NC, LIM, 1, 2>(k, s);
  return k.p <= 32 ? launch_rows_k<MODE, XBF, OBF, NX, NB, NZ, NC, LIM, 2, 1>(k, s)
                   : launch_rows_k<MODE, XBF, OBF, NX, NB, NZ, NC, LIM, 2, 2>(k, s);
}

}  // namespace

// Parts: fp32 three of everything.  bf16 inputs are one part (C = S o A two: the product of two bf16 values has
// 16 bits).  What a bf16 y or dX is summed from has two, what the fp32 parameter gradients come from three.
#if KRON_GLU_MODE == 0
hipError_t launch_glu_rows0(const GluRows& k, bool bf16, bool with_S, hipStream_t s) {
  if (!bf16) return launch_rows<0, false, false, 3, 3, 3, 3, 2>(k, s);
  return with_S ? launch_rows<0, true, true, 1, 1, 2, 2, 2>(k, s) : launch_rows<0, true, true, 1, 1, 2, 1, 1>(k, s);
}
#elif KRON_GLU_MODE == 1
hipError_t launch_glu_rows1(const GluRows& k, bool bf16, bool with_S, hipStream_t s) {
  if (!bf16) return launch_rows<1, false, false, 3, 3, 3, 3, 2>(k, s);
  return with_S ? launch_rows<1, true, true, 1, 1, 3, 2, 2>(k, s) : launch_rows<1, true, true, 1, 1, 3, 1, 2>(k, s);
}
#else
hipError_t launch_glu_rows2(const GluRows& k, bool bf16, bool with_S, hipStream_t s) {
  if (!bf16) return launch_rows<2, false, false, 3, 3, 3, 3, 2>(k, s);
  return with_S ? launch_rows<2, false, true, 2, 1, 2, 2, 2>(k, s) : launch_rows<2, false, true, 2, 1, 2, 1, 1>(k, s);
}
#endif

}  // namespace kron
