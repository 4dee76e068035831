// The gated Kronecker block: the factors' gradients.  A workgroup has one kind and a group of pairs (f, i):
//   kind 0  dC_fi (p x q) += Z_fi d_f^T, Z_fi = X B_fi       kind 1  dB_fi (m x n) += X^T G_fi, G_fi = C_fi d_f
// Each wavefront owns a pair's sum in registers, with B_fi (or C_fi) beside it; with fewer pairs than
// wavefronts several share a pair and take rows in turn.  A step's rows of X and d_f are split
// into parts once and staged in LDS as operand blocks in the order that the kind contracts over (4 x 4
// patches, which a thread turns in its registers).  Two buffers: while one step is multiplied the next
// is staged, half of the wavefronts staging first and half multiplying first, and the values of the one
// after that are on their way.
//
// Slots of a block are permuted against bank conflicts: column c of k-group g stands at 16 g + 4 ((c % 4) ^ g) + c / 4.
// A wavefront stores columns of one residue mod 4 at a time: their quarters of a 256-byte row differ by g.  (Conflicts
// are a quarter of the LDS cycles that are left, by counter 3.6 M of 14.9 M at the size below.)
//
// Measured at 8192 x (768 -> 2048) bf16, r = 4: 125 us; its products (5,666 instructions a SIMD) would take 38 at the
// matrix cores' peak and 79 at the rate of a large library product, its reads of d_f 27.  What bounds it: matrix
// cores 0.32 of the time, vector instructions 0.30, and a wavefront waits 0.39 of its time; two wavefronts a SIMD
// (their sums and B take 190 registers) do not cover the LDS reads, the splits of d_f, Z and G into parts and the
// staging beside the products.  Without the products the staging alone took 82 us.  2048 x 1024^2 fp32: 35 us.  Operands read one product ahead and
// instances by the sides' tiles took it from 156 to 140 us, the kinds' shares of the workgroups (glu.hip) to
// 125; raised wave priorities and first products four side by side changed nothing beyond 3%.
//
// A run of fp32 additions covers at most 512 rows of a group (8192 rows in all with 16 groups of each kind, 65536
// with 128); more rows take several launches, which add to the partial rows.
//
// Compiled once for each type (KRON_GLU_TYPE: 0 fp32, 1 bf16, 2 bf16 with S).
#include "glu_parts.h"

namespace kron {
namespace {

constexpr int64_t kRunRows = 512;      // rows of a group in one run of additions

// Sizes of a step that both the host and the kernel use.
struct ParamSizes {
  int PT, QT, MT, NT, PK, QK, MK, NK;
  int dk, dpat, xk, xpat;          // patches
  int xa, ya;                      // u4 of a row's X blocks, and of one d_f's
  __host__ __device__ ParamSizes(const GluParam& a, int nx, int kind) {
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

// TI: tiles of the inner side of the second product (kind 0: p, kind 1: n) at most, TK: of the side that it
// contracts (kind 0: n, kind 1: p), TO: of q and m (2 or 4: sides up to 32 take fewer registers).
template <bool XBF, int NX, int NTAB, int KIND, int TI, int TK, int TO, int NTH>
__device__ inline void param_body(const GluParam& a, int rowgroup, int pairgroup, const u4* table, u4* lds) {
  constexpr int NY = 3, KI = TK / 2, KO = TO / 2;      // steps of 32
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
  Op tab[TK][KO][NTAB];    // kind 0: B_fi [NT][MK]; kind 1: C_fi^T [PT][QK]
  const int tabT = KIND == 0 ? z.NT : z.PT, tabK = KIND == 0 ? z.MK : z.QK;
#pragma unroll
  for (int t = 0; t < TK; ++t)
#pragma unroll
    for (int k = 0; k < KO; ++k)
#pragma unroll
      for (int s = 0; s < NTAB; ++s) {
        tab[t][k][s].u = u4{0u, 0u, 0u, 0u};
        if (t < tabT && k < tabK) tab[t][k][s].u = table[((int64_t)((fi * tabT + t) * tabK + k) * NTAB + s) * 64 + lane];
      }
  f4 acc[TI][TO];          // kind 0: [p][q]; kind 1: [n][m]
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TO; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};

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
          const u2v t = u2v{kron::part(part, 3, u[i][0], u[i][1]), kron::part(part, 3, u[i][2], u[i][3])};
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
  // One row's products.  The first product into tile pairs; the inner tiles of the second (p or n) all at
  // once (those that are not there have zero blocks), so that no branch stands between the products.  The
  // operands of a product are read one ahead of it (past the last tile: whatever stands there, unused).
  auto multiply = [&](const u4* xl, const u4* yl) {
    constexpr int N1 = KIND == 0 ? NX : NY, NO = KIND == 0 ? NY : NX;
    const u4* l1 = KIND == 0 ? xl : yl;      // of the first product: [k step][tile][part]
    const int s1 = (KIND == 0 ? 2 * z.PK : 2 * z.NK) * N1 * 64;
    const u4* l2 = KIND == 0 ? yl : xl;      // of the second
    const int s2 = (KIND == 0 ? z.QT : z.MT) * NO * 64;
    const int steps = KIND == 0 ? z.NK : z.PK, outer = KIND == 0 ? z.QT : z.MT;
    auto read1 = [&](int t, Op (&o)[KO][N1]) {
#pragma unroll
      for (int k = 0; k < KO; ++k)
        if (k < tabK) {
#pragma unroll
          for (int s = 0; s < N1; ++s) o[k][s].u = l1[k * s1 + (t * N1 + s) * 64];
        }
    };
    auto read2 = [&](int ko, int t, Op (&o)[NO]) {
#pragma unroll
      for (int s = 0; s < NO; ++s) o[s].u = l2[ko * s2 + (t * NO + s) * 64];
    };
    Op o1[2][KO][N1], o2[2][NO];
    read1(0, o1[0]);
    read1(1, o1[1]);
#pragma unroll
    for (int ko = 0; ko < KI; ++ko)
      if (ko < steps) {
        Op h[TI][3];
        read2(ko, 0, o2[0]);
        // tiles in pairs: four products side by side, so that none waits for the one before it
#pragma unroll
        for (int t = 0; t < TI; t += 2) {
          f4 w[2][2];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i / 2][i % 2] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < KO; ++k)
            if (k < tabK) {
#pragma unroll
              for (int o = 2; o >= 0; --o)
#pragma unroll
                for (int i = 0; i < NTAB; ++i)
                  if (o - i >= 0 && o - i < N1)
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j / 2][j % 2] = mfma(tab[2 * ko + j % 2][k][i], o1[j / 2][k][o - i], w[j / 2][j % 2]);
            }
          if (TI > 2 && (t + 2 < TI || ko + 1 < KI)) {      // (two tiles stay for the next step)
            read1((t + 2) % TI, o1[0]);
            read1((t + 3) % TI, o1[1]);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) split<3>(w[j][0], w[j][1], h[t + j]);
        }
#pragma unroll
        for (int t = 0; t < TO; ++t)
          if (t < outer) {
            if (t + 1 < TO) read2(ko, t + 1, o2[(t + 1) & 1]);
#pragma unroll
            for (int o = 2; o >= 0; --o)
#pragma unroll
              for (int s = 0; s <= o; ++s)
                if (o - s < NO)
#pragma unroll
                  for (int i = 0; i < TI; ++i) {
                    if (KIND == 0) acc[i][t] = mfma(h[i][s], o2[t & 1][o - s], acc[i][t]);
                    if (KIND == 1) acc[i][t] = mfma(o2[t & 1][o - s], h[i][s], acc[i][t]);
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
      multiply(xl, yl);
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
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TO; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ri = 16 * (KIND == 0 ? i : j) + 4 * g + e, ci = 16 * (KIND == 0 ? j : i) + c;
          if (ri < R && ci < Cn) {
            float& o = out[base + (int64_t)ri * Cn + ci];
            o = a.add ? o + acc[i][j][e] : acc[i][j][e];
          }
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
        float& o = ow[pairs * pq + (int64_t)ff * a.q * a.n + (int64_t)j * a.n + k];
        const float d = w == 0 ? bl[i] : 0.f;
        o = a.add ? o + d : d;
      }
  }
}

template <bool XBF, int NX, int NB, int NC, int TP, int TN, int TO, int NTH>
__global__ __launch_bounds__(NTH) void glu_param_kernel(GluParam a) {
  extern __shared__ u4 lds[];
  int b = blockIdx.x;
  const int n0 = a.groups[0] * a.pair_groups;
  if (b < n0) {
    param_body<XBF, NX, NB, 0, TP, TN, TO, NTH>(a, b / a.pair_groups, b % a.pair_groups, a.tb, lds);
  } else {
    b -= n0;
    param_body<XBF, NX, NC, 1, TN, TP, TO, NTH>(a, b / a.pair_groups, b % a.pair_groups, a.tc, lds);
  }
}

template <bool XBF, int NX, int NB, int NC, int TP, int TN, int TO>
hipError_t launch_param_k(const GluParam& k, size_t lds, hipStream_t s) {
  constexpr int NTH = 64 * param_waves(XBF, TP > 2, TN > 2, TO > 2);
  constexpr auto kernel = glu_param_kernel<XBF, NX, NB, NC, TP, TN, TO, NTH>;
  hipError_t e = allow_lds<kernel>();
  if (e != hipSuccess) return e;
  // A group sums at most kRunRows rows in one run of fp32 additions; more rows take several launches, each of which
  // adds its runs to the partial rows.  (Runs of 131072 equal rows were off by 4.7e-3.)
  const int64_t most = kRunRows * std::min(k.groups[0], k.groups[1]), parts = std::max<int64_t>(1, (k.N + most - 1) / most);
  const int64_t rows = (k.N + parts - 1) / parts;
  for (int64_t i = 0; i < parts; ++i) {
    GluParam part = k;
    const int64_t r0 = i * rows;
    part.N = std::min(rows, k.N - r0);
    part.x = (const char*)k.x + r0 * k.p * k.m * (XBF ? 2 : 4);
    for (int f = 0; f < 2; ++f) part.d[f] = k.d[f] + r0 * k.q * k.n4;
    part.add = i > 0;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((k.groups[0] + k.groups[1]) * k.pair_groups)), dim3(NTH), lds, s, part);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool XBF, int NX, int NB, int NC>
hipError_t launch_param(GluParam k, hipStream_t s) {
  const int ppw = ceil_div(2 * k.r, k.pair_groups);
  int nf = 1;      // most projections of a workgroup
  for (int y = 0; y < k.pair_groups; ++y)
    if ((std::min(2 * k.r, (y + 1) * ppw) - 1) / k.r != y * ppw / k.r) nf = 2;
  // as many rows a step as two LDS buffers and the threads' slots hold (but no more than four a wavefront)
  const ParamSizes z0(k, NX, 0), z1(k, NX, 1);
  const size_t one = (size_t)std::max(z0.row(nf), z1.row(nf)) * 16;
  constexpr size_t over = 8 * 1024;      // what is read of tiles past the last (two of three parts, and one ahead)
  const int nd = nf * z0.dpat, np = nd + z0.xpat;
  const int64_t rows = (k.N + k.groups[0] - 1) / k.groups[0];
  k.rs = 1;
  while (k.rs < 4 * k.share && k.rs < rows && 2 * (k.rs + 1) * one + over <= kLds && (k.rs + 1) * nd <= 512 &&
         (k.rs + 1) * np <= 1024)
    ++k.rs;
  // (dbias is joined in the same LDS: 64 bytes a patch of d_f)
  const size_t lds = std::max(2 * one * k.rs + over, (size_t)nd * 64);
  if (std::max(k.q, k.m) <= 32) {
    if (k.p <= 32) return k.n <= 32 ? launch_param_k<XBF, NX, NB, NC, 2, 2, 2>(k, lds, s) : launch_param_k<XBF, NX, NB, NC, 2, 4, 2>(k, lds, s);
    return k.n <= 32 ? launch_param_k<XBF, NX, NB, NC, 4, 2, 2>(k, lds, s) : launch_param_k<XBF, NX, NB, NC, 4, 4, 2>(k, lds, s);
  }
  if (k.p <= 32) return k.n <= 32 ? launch_param_k<XBF, NX, NB, NC, 2, 2, 4>(k, lds, s) : launch_param_k<XBF, NX, NB, NC, 2, 4, 4>(k, lds, s);
  return k.n <= 32 ? launch_param_k<XBF, NX, NB, NC, 4, 2, 4>(k, lds, s) : launch_param_k<XBF, NX, NB, NC, 4, 4, 4>(k, lds, s);
}

}  // namespace

#if KRON_GLU_TYPE == 0
hipError_t launch_glu_param_f32(const GluParam& k, hipStream_t s) { return launch_param<false, 3, 3, 3>(k, s); }
#elif KRON_GLU_TYPE == 1
hipError_t launch_glu_param_bf16(const GluParam& k, hipStream_t s) { return launch_param<true, 1, 1, 1>(k, s); }
#else
hipError_t launch_glu_param_bf16_S(const GluParam& k, hipStream_t s) { return launch_param<true, 1, 1, 2>(k, s); }
#endif

}  // namespace kron
