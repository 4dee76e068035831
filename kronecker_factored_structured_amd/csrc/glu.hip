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
__device__ inline float top(float a) { return __uint_as_float(__float_as_uint(a) & 0xffff0000u); }

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
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        lo[v] -= top(lo[v]);
        hi[v] -= top(hi[v]);
      }
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
// A wavefront takes RW rows and one 16-column tile of n, and for it all q (at most 64).
// ---------------------------------------------------------------------------------
struct RowsArgs {
  int64_t N;
  int p, q, m, n, r;       // of these products (MODE 2: q, p, n, m of the layer)
  int ldm;                 // elements from one row of X_f to the next
  int64_t ldx;             // elements from one X to the next
  int act;
  int ntiles, qsplit;      // tiles of n; workgroups that share the q tiles
  const void* x[2];
  const u4* tb;            // B blocks
  const u4* tc;            // C blocks
  const void* bias;        // 2 x q n, or NULL
  const void* dy;
  void* y;
  float* d[2];             // dg, du: rows of q x n4
  int n4;
};

constexpr int kQT = 4;

template <bool BF>
__device__ inline float load1(const void* p, int64_t i) {
  return BF ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}

// XBF: X is bf16 (one part); else fp32 in NX parts.  OBF: bias, dy and the output are bf16.
template <int MODE, bool XBF, bool OBF, int NX, int NB, int NZ, int NC, int LIM, int MK, int RW>
__global__ __launch_bounds__(256) void glu_rows_kernel(RowsArgs a) {
  constexpr int NF = MODE == 2 ? 1 : 2;
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int nt = (int)(unit % a.ntiles);
  const int64_t u2 = unit / a.ntiles;
  const int qs = (int)(u2 % a.qsplit);
  const int64_t row0 = (u2 / a.qsplit) * RW;
  if (row0 >= a.N) return;
  const int QT = (a.q + 15) / 16, PK = (a.p + 31) / 32;
  const int qt0 = QT * qs / a.qsplit, qtn = QT * (qs + 1) / a.qsplit - qt0;
  f4 acc[NF][kQT][RW];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int j = 0; j < kQT; ++j)
#pragma unroll
      for (int w = 0; w < RW; ++w) acc[f][j][w] = f4{0.f, 0.f, 0.f, 0.f};

  const bool vec = XBF ? (a.ldm & 7) == 0 : (a.ldm & 3) == 0;
  for (int pk = 0; pk < PK; ++pk) {
    Op xa[RW][2][MK][NX];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      if (f == 0 || MODE == 2) {
#pragma unroll
        for (int w = 0; w < RW; ++w)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int mk = 0; mk < MK; ++mk) {
              const int pi = 32 * pk + 16 * t + c, k = 32 * mk + 8 * g;
              const int64_t at = (row0 + w) * a.ldx + (int64_t)pi * a.ldm + k;
              const bool in = row0 + w < a.N && pi < a.p;
              if (XBF) {
                Op o;
                o.u = u4{0u, 0u, 0u, 0u};
                if (in && vec) {
                  if (k < a.m) o.u = *reinterpret_cast<const u4*>((const uint16_t*)a.x[f] + at);
                } else if (in) {
#pragma unroll
                  for (int e = 0; e < 8; ++e)
                    if (k + e < a.m)
                      o.u[e / 2] |= (uint32_t)((const uint16_t*)a.x[f])[at + e] << (16 * (e & 1));
                }
                xa[w][t][mk][0] = o;
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
                split<NX>(lo, hi, xa[w][t][mk]);
              }
            }
      }
      for (int i = 0; i < a.r; ++i) {
        const int fi = f * a.r + i;
        Op zb[RW][NZ];
        {
          f4 z[RW][2];
#pragma unroll
          for (int w = 0; w < RW; ++w) z[w][0] = z[w][1] = f4{0.f, 0.f, 0.f, 0.f};
          const u4* tb = a.tb + ((int64_t)(fi * a.ntiles + nt) * MK * NB) * 64 + lane;
#pragma unroll
          for (int mk = 0; mk < MK; ++mk) {
            Op b[NB];
#pragma unroll
            for (int s = 0; s < NB; ++s) b[s].u = tb[(mk * NB + s) * 64];
#pragma unroll
            for (int w = 0; w < RW; ++w)
#pragma unroll
              for (int t = 0; t < 2; ++t) z[w][t] = dot<NX, NB, LIM>(xa[w][t][mk], b, z[w][t]);
          }
#pragma unroll
          for (int w = 0; w < RW; ++w) split<NZ>(z[w][0], z[w][1], zb[w]);
        }
        const u4* tc = a.tc + ((int64_t)(fi * QT + qt0) * PK + pk) * NC * 64 + lane;
#pragma unroll
        for (int j = 0; j < kQT; ++j)
          if (j < qtn) {
            Op b[NC];
#pragma unroll
            for (int s = 0; s < NC; ++s) b[s].u = tc[((int64_t)j * PK * NC + s) * 64];
#pragma unroll
            for (int w = 0; w < RW; ++w) acc[MODE == 2 ? 0 : f][j][w] = dot<NZ, NC, LIM>(zb[w], b, acc[MODE == 2 ? 0 : f][j][w]);
          }
      }
    }
  }

  const int n0 = 16 * nt + 4 * g;
  const int64_t qn = (int64_t)a.q * a.n;
  const bool ovec = (a.n & 3) == 0;
#pragma unroll
  for (int j = 0; j < kQT; ++j) {
    const int qi = 16 * (qt0 + j) + c;
    if (j >= qtn || qi >= a.q || n0 >= a.n) continue;
    const int64_t at = (int64_t)qi * a.n + n0;
    float bg[4] = {0.f, 0.f, 0.f, 0.f}, bu[4] = {0.f, 0.f, 0.f, 0.f};
    if (MODE != 2 && a.bias) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (n0 + v < a.n) {
          bg[v] = load1<OBF>(a.bias, at + v);
          bu[v] = load1<OBF>(a.bias, qn + at + v);
        }
    }
#pragma unroll
    for (int w = 0; w < RW; ++w) {
      const int64_t row = row0 + w;
      if (row >= a.N) continue;
      const int64_t o = row * qn + at;
      f4 out;
      if (MODE == 1) {
        f4 dg, du;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float dy = n0 + v < a.n ? load1<OBF>(a.dy, o + v) : 0.f;
          const float gv = acc[0][j][w][v] + bg[v], uv = acc[NF - 1][j][w][v] + bu[v];
          float dact;
          const float av = activate<true>(a.act, gv, &dact);
          dg[v] = dy * uv * dact;
          du[v] = dy * av;
          if (n0 + v >= a.n) dg[v] = du[v] = 0.f;      // (the padding of the workspace's rows)
        }
        const int64_t od = (row * a.q + qi) * a.n4 + n0;
        *reinterpret_cast<f4*>(a.d[0] + od) = dg;
        *reinterpret_cast<f4*>(a.d[1] + od) = du;
        continue;
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if (MODE == 0)
          out[v] = activate<false>(a.act, acc[0][j][w][v] + bg[v], nullptr) * (acc[NF - 1][j][w][v] + bu[v]);
        else
          out[v] = acc[0][j][w][v];
      }
      if (OBF) {
        uint16_t* y = (uint16_t*)a.y + o;
        const uint32_t h0 = bf16_rne(out[0]), h1 = bf16_rne(out[1]), h2 = bf16_rne(out[2]), h3 = bf16_rne(out[3]);
        if (ovec) {
          typedef uint32_t u2v __attribute__((ext_vector_type(2)));
          *reinterpret_cast<u2v*>(y) = u2v{h0 | (h1 << 16), h2 | (h3 << 16)};
        } else {
          y[0] = (uint16_t)h0;
          if (n0 + 1 < a.n) y[1] = (uint16_t)h1;
          if (n0 + 2 < a.n) y[2] = (uint16_t)h2;
          if (n0 + 3 < a.n) y[3] = (uint16_t)h3;
        }
      } else {
        float* y = (float*)a.y + o;
        if (ovec) {
          *reinterpret_cast<f4*>(y) = out;
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (n0 + v < a.n) y[v] = out[v];
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------------
// The factors' gradients.  A workgroup takes rows in turn; each of its wavefronts owns one of
//   dC_fi (p x q) += Z_fi d_f^T, Z_fi = X B_fi       dB_fi (m x n) += X^T G_fi, G_fi = C_fi d_f
// in registers.  A row's X and d_f are split into parts once and staged in LDS as operand blocks
// in both orders that the products contract over.
// ---------------------------------------------------------------------------------
struct ParamArgs {
  int64_t N;
  int p, q, m, n, r, n4;
  int64_t rows;            // rows of a workgroup
  const void* x;
  const float* d[2];
  const u4* tb;            // B blocks (k = m)
  const u4* tc;            // C^T blocks (k = q)
  float* part;             // partial rows: dB (2 r m n) | dC (2 r p q) | dbias (2 q n)
};

constexpr int kPPW = 4;    // pairs (f, i) of a workgroup: wavefronts 0..3 take dC, 4..7 dB

template <bool XBF, int NX, int NB, int NC>
__global__ __launch_bounds__(512) void glu_param_kernel(ParamArgs a) {
  extern __shared__ u4 lds[];
  constexpr int NY = 3;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;
  const int PT = (a.p + 15) / 16, QT = (a.q + 15) / 16, MT = (a.m + 15) / 16, NT = (a.n + 15) / 16;
  const int PK = (a.p + 31) / 32, QK = (a.q + 31) / 32, MK = (a.m + 31) / 32, NK = (a.n + 31) / 32;
  const int pair0 = blockIdx.y * kPPW, pairs = 2 * a.r;
  const int pairn = min(kPPW, pairs - pair0);
  const int f_lo = pair0 / a.r, f_hi = (pair0 + pairn - 1) / a.r;
  // LDS: XA [PT][MK][NX] k = m; XB [MT][PK][NX] k = p; for each f: YA [QT][NK][NY] k = n; YB [NT][QK][NY] k = q
  const int xa0 = 0, xb0 = xa0 + PT * MK * NX * 64, y0 = xb0 + MT * PK * NX * 64;
  const int ysz = (QT * NK + NT * QK) * NY * 64;
  const int all = y0 + ysz * (f_hi - f_lo + 1);
  for (int i = tid; i < all; i += 512) lds[i] = u4{0u, 0u, 0u, 0u};      // the tiles' padding stays zero

  const int pl = wave % kPPW, kind = wave / kPPW;
  const bool active = pl < pairn;
  const int fi = pair0 + (active ? pl : 0), f = fi / a.r;
  Op tab[4][2][3];         // kind 0: B_fi [NT][MK]; kind 1: C_fi^T [PT][QK]
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        tab[t][k][s].u = u4{0u, 0u, 0u, 0u};
        if (kind == 0) {
          if (s < NB && t < NT && k < MK) tab[t][k][s].u = a.tb[((int64_t)((fi * NT + t) * MK + k) * NB + s) * 64 + lane];
        } else {
          if (s < NC && t < PT && k < QK) tab[t][k][s].u = a.tc[((int64_t)((fi * PT + t) * QK + k) * NC + s) * 64 + lane];
        }
      }
  f4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};

  // 4 x 4 patches of a row's matrices: of d_f first (at most 512: one a thread), then of X
  const int dj = (a.q + 3) / 4, dk = a.n4 / 4, dpat = dj * dk;
  const int xj = (a.p + 3) / 4, xk = (a.m + 3) / 4, xpat = xj * xk;
  const int nf = f_hi - f_lo + 1, npat = nf * dpat + xpat;
  float bsum[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) bsum[e] = 0.f;
  const bool xvec = XBF ? (a.m & 3) == 0 : (a.m & 3) == 0;

  const int64_t r0 = (int64_t)blockIdx.x * a.rows, r1 = min(a.N, r0 + a.rows);
  for (int64_t row = r0; row < r1; ++row) {
    __syncthreads();       // the previous row's operands have been read
    for (int pt = tid; pt < npat; pt += 512) {
      f4 v[4];
      int j0, k0;
      const bool isd = pt < nf * dpat;
      if (isd) {
        const int ff = pt / dpat, e = pt - ff * dpat;
        j0 = 4 * (e / dk);
        k0 = 4 * (e % dk);
        const float* src = a.d[f_lo + ff] + (row * a.q + j0) * a.n4 + k0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = j0 + i < a.q ? *reinterpret_cast<const f4*>(src + (int64_t)i * a.n4) : f4{0.f, 0.f, 0.f, 0.f};
        if (pt == tid) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e2 = 0; e2 < 4; ++e2) bsum[4 * i + e2] += v[i][e2];
        }
      } else {
        const int e = pt - nf * dpat;
        j0 = 4 * (e / xk);
        k0 = 4 * (e % xk);
        const int64_t src = (row * a.p + j0) * a.m + k0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = f4{0.f, 0.f, 0.f, 0.f};
          if (j0 + i < a.p) {
            if (!XBF && xvec) {
              v[i] = *reinterpret_cast<const f4*>((const float*)a.x + src + (int64_t)i * a.m);
            } else {
#pragma unroll
              for (int e2 = 0; e2 < 4; ++e2)
                if (k0 + e2 < a.m) v[i][e2] = load1<XBF>(a.x, src + (int64_t)i * a.m + e2);
            }
          }
        }
      }
      // into the blocks: [column tile][k step][part], lane (g, c), slots 0..3 or 4..7
      const int np = isd ? NY : NX;
      const int ff = isd ? pt / dpat : 0;
      const int baseA = isd ? y0 + ff * ysz : xa0, baseB = isd ? y0 + ff * ysz + QT * NK * NY * 64 : xb0;
      const int ksA = isd ? NK : MK, ksB = isd ? QK : PK;
      typedef uint32_t u2v __attribute__((ext_vector_type(2)));
      u2v* l2 = reinterpret_cast<u2v*>(lds);
      // order A: k along the row.  d_f: chained; X: natural (its partner is the packed B)
      const int kk = k0 & 31;
      const int gA = isd ? (kk & 15) >> 2 : kk >> 3, hA = isd ? kk >> 4 : (kk >> 2) & 1;
      // order B: k down the column, chained
      const int jj = j0 & 31;
      const int gB = (jj & 15) >> 2, hB = jj >> 4;
      for (int s = 0; s < np; ++s) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = j0 + i;
          const int blk = baseA + (((j >> 4) * ksA + (k0 >> 5)) * np + s) * 64 + gA * 16 + (j & 15);
          if (j < 16 * (isd ? QT : PT)) l2[2 * blk + hA] = u2v{tops(v[i][0], v[i][1]), tops(v[i][2], v[i][3])};
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = k0 + i;
          const int blk = baseB + (((k >> 4) * ksB + (j0 >> 5)) * np + s) * 64 + gB * 16 + (k & 15);
          l2[2 * blk + hB] = u2v{tops(v[0][i], v[1][i]), tops(v[2][i], v[3][i])};
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e2 = 0; e2 < 4; ++e2) v[i][e2] -= top(v[i][e2]);
      }
    }
    __syncthreads();
    if (!active) continue;
    const u4* ya = lds + y0 + (f - f_lo) * ysz;
    const u4* yb = ya + QT * NK * NY * 64;
    if (kind == 0) {
#pragma unroll
      for (int nk = 0; nk < 2; ++nk)
        if (nk < NK) {
          Op zp[4][3];
#pragma unroll
          for (int pt = 0; pt < 4; ++pt)
            if (pt < PT) {
              f4 z[2];
              z[0] = z[1] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int mk = 0; mk < 2; ++mk)
                if (mk < MK) {
                  Op x[NX];
#pragma unroll
                  for (int s = 0; s < NX; ++s) x[s].u = lds[xa0 + ((pt * MK + mk) * NX + s) * 64 + lane];
#pragma unroll
                  for (int t = 0; t < 2; ++t) z[t] = dot<NB, NX, 2>(tab[2 * nk + t][mk], x, z[t]);
                }
              split<3>(z[0], z[1], zp[pt]);
            }
#pragma unroll
          for (int qt = 0; qt < 4; ++qt)
            if (qt < QT) {
              Op y[NY];
#pragma unroll
              for (int s = 0; s < NY; ++s) y[s].u = ya[((qt * NK + nk) * NY + s) * 64 + lane];
#pragma unroll
              for (int pt = 0; pt < 4; ++pt)
                if (pt < PT) acc[pt][qt] = dot<3, NY, 2>(zp[pt], y, acc[pt][qt]);
            }
        }
    } else {
#pragma unroll
      for (int pk = 0; pk < 2; ++pk)
        if (pk < PK) {
          Op gp[4][3];
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
            if (nt < NT) {
              f4 z[2];
              z[0] = z[1] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int qk = 0; qk < 2; ++qk)
                if (qk < QK) {
                  Op y[NY];
#pragma unroll
                  for (int s = 0; s < NY; ++s) y[s].u = yb[((nt * QK + qk) * NY + s) * 64 + lane];
#pragma unroll
                  for (int t = 0; t < 2; ++t) z[t] = dot<NC, NY, 2>(tab[2 * pk + t][qk], y, z[t]);
                }
              split<3>(z[0], z[1], gp[nt]);
            }
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
            if (mt < MT) {
              Op x[NX];
#pragma unroll
              for (int s = 0; s < NX; ++s) x[s].u = lds[xb0 + ((mt * PK + pk) * NX + s) * 64 + lane];
#pragma unroll
              for (int nt = 0; nt < 4; ++nt)
                if (nt < NT) acc[mt][nt] = dot<NX, 3, 2>(x, gp[nt], acc[mt][nt]);
            }
        }
    }
  }

  // this workgroup's partial row
  const int64_t mn = (int64_t)a.m * a.n, pq = (int64_t)a.p * a.q;
  const PartRow out{a.part, (int64_t)gridDim.x, (int64_t)blockIdx.x, 0};
  if (active) {
    const int R = kind == 0 ? a.p : a.m, Cn = kind == 0 ? a.q : a.n;
    const int64_t base = kind == 0 ? pairs * mn + fi * pq : fi * mn;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int ri = 16 * i + 4 * g + v, ci = 16 * j + c;
          if (ri < R && ci < Cn) out[base + (int64_t)ri * Cn + ci] = acc[i][j][v];
        }
  }
  if (tid < nf * dpat) {
    const int ff = f_lo + tid / dpat, e = tid % dpat;
    if (ff * a.r >= pair0 && ff * a.r < pair0 + pairn) {      // the workgroup with f's first pair
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e2 = 0; e2 < 4; ++e2) {
          const int j = 4 * (e / dk) + i, k = 4 * (e % dk) + e2;
          if (j < a.q && k < a.n)
            out[pairs * (mn + pq) + (int64_t)ff * a.q * a.n + (int64_t)j * a.n + k] = bsum[4 * i + e2];
        }
    }
  }
}

// dA = S o dC, dS = sum_i A_i o dC_i from the summed dC (2 x r x p x q).
__global__ __launch_bounds__(256) void glu_ds_kernel(int pq, int r, int bf16, const void* S, const void* A,
                                                     const float* __restrict__ dC, float* __restrict__ dS,
                                                     float* __restrict__ dA) {
  const int e = blockIdx.x * 256 + threadIdx.x;
  if (e >= 2 * pq) return;
  const int f = e / pq, o = e - f * pq;
  const float s = raw(S, e, bf16);
  float sum = 0.f;
  for (int i = 0; i < r; ++i) {
    const int64_t at = ((int64_t)f * r + i) * pq + o;
    const float d = dC[at];
    dA[at] = s * d;
    sum = fmaf(raw(A, at, bf16), d, sum);
  }
  dS[e] = sum;
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

struct Sizes {
  int parts_b, parts_c;
  int64_t lanes[4], bytes[4];
  int n4, groups;
  int64_t PW, off_d, off_part, off_dc, fwd_bytes, bwd_bytes;
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
  z.off_part = z.off_d + ((2 * a.N * a.q * z.n4 * 4 + 255) & ~int64_t(255));
  const int Y = ceil_div(2 * a.r, kPPW);
  // one workgroup a CU (its LDS), every one with at least four rows where there are that many
  int64_t G = 256 / Y;
  if (G > (a.N + 3) / 4) G = (a.N + 3) / 4;
  z.groups = G < 1 ? 1 : (int)G;
  z.PW = (int64_t)2 * a.r * (a.m * a.n + a.p * a.q) + 2 * a.q * a.n;
  z.off_dc = z.off_part + ((part_floats(z.groups, z.PW) * 4 + 255) & ~int64_t(255));
  z.bwd_bytes = z.off_dc + (int64_t)2 * a.r * a.p * a.q * 4;
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

template <int MODE, bool XBF, bool OBF, int NX, int NB, int NZ, int NC, int LIM>
hipError_t launch_rows(RowsArgs k, hipStream_t s) {
  constexpr int RW = 2;
  k.ntiles = ceil_div(k.n, 16);
  const int QT = ceil_div(k.q, 16);
  const int64_t groups = (k.N + RW - 1) / RW;
  k.qsplit = 1;
  while (k.qsplit < QT && groups * k.ntiles * k.qsplit < 1024) ++k.qsplit;
  const int64_t units = groups * k.ntiles * k.qsplit;
  const dim3 grid((unsigned)((units + 3) / 4));
  if (k.m <= 32)
    hipLaunchKernelGGL((glu_rows_kernel<MODE, XBF, OBF, NX, NB, NZ, NC, LIM, 1, RW>), grid, dim3(256), 0, s, k);
  else
    hipLaunchKernelGGL((glu_rows_kernel<MODE, XBF, OBF, NX, NB, NZ, NC, LIM, 2, RW>), grid, dim3(256), 0, s, k);
  return hipGetLastError();
}

template <bool XBF, int NX, int NB, int NC>
hipError_t launch_param(const ParamArgs& k, int G, hipStream_t s) {
  const int PT = ceil_div(k.p, 16), QT = ceil_div(k.q, 16), MT = ceil_div(k.m, 16), NT = ceil_div(k.n, 16);
  const int PK = ceil_div(k.p, 32), QK = ceil_div(k.q, 32), MK = ceil_div(k.m, 32), NK = ceil_div(k.n, 32);
  const int nf = k.r >= 4 && k.r % kPPW == 0 ? 1 : 2;
  const size_t lds = (size_t)((PT * MK + MT * PK) * NX + nf * (QT * NK + NT * QK) * 3) * 1024;
  static const hipError_t attr = hipFuncSetAttribute((const void*)glu_param_kernel<XBF, NX, NB, NC>,
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL((glu_param_kernel<XBF, NX, NB, NC>), dim3((unsigned)G, (unsigned)ceil_div(2 * k.r, kPPW)),
                     dim3(512), lds, s, k);
  return hipGetLastError();
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
  k.x[0] = k.x[1] = a.x; k.tb = t[0]; k.tc = t[1]; k.bias = a.bias; k.y = a.y;
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
  float* part = (float*)((char*)ws + z.off_part);
  float* dC = (float*)((char*)ws + z.off_dc);
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
      x.ldm = z.n4; x.ldx = (int64_t)a.q * z.n4;
      x.x[0] = d; x.x[1] = d2; x.tb = t[2]; x.tc = t[3]; x.y = a.dx;
      if (!a.bf16) e = launch_rows<2, false, false, 3, 3, 3, 3, 2>(x, s);
      else if (a.S) e = launch_rows<2, false, true, 2, 1, 2, 2, 1>(x, s);
      else e = launch_rows<2, false, true, 2, 1, 2, 1, 1>(x, s);
      if (e != hipSuccess) return e;
    }
  }
  ParamArgs k{};
  k.N = a.N; k.p = a.p; k.q = a.q; k.m = a.m; k.n = a.n; k.r = a.r; k.n4 = z.n4;
  k.rows = (a.N + z.groups - 1) / z.groups;
  k.x = a.x; k.d[0] = d; k.d[1] = d2; k.tb = t[0]; k.tc = t[3]; k.part = part;
  if (!a.bf16) e = launch_param<false, 3, 3, 3>(k, z.groups, s);
  else if (a.S) e = launch_param<true, 1, 1, 2>(k, z.groups, s);
  else e = launch_param<true, 1, 1, 1>(k, z.groups, s);
  if (e != hipSuccess) return e;
  RedPlan rp{};
  rp.nseg = 3;
  rp.seg[0] = RedSeg{a.dB, 2 * a.r * a.m * a.n, 1.f, 0};
  rp.seg[1] = RedSeg{a.S ? dC : a.dA, 2 * a.r * a.p * a.q, 1.f, 0};
  rp.seg[2] = RedSeg{a.dbias, 2 * a.q * a.n, 1.f, 0};
  e = launch_column_reduce(part, z.groups, (int32_t)z.PW, rp, s);
  if (e != hipSuccess || !a.S) return e;
  const int pq = a.p * a.q;
  hipLaunchKernelGGL(glu_ds_kernel, dim3((unsigned)((2 * pq + 255) / 256)), dim3(256), 0, s, pq, a.r, a.bf16, a.S, a.A,
                     dC, a.dS, a.dA);
  return hipGetLastError();
}

}  // namespace kron
