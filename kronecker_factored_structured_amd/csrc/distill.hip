// Distillation of a student's logits z (N x V) from a teacher's top k tokens of each row, with
// an optional cross-entropy on labels, forward and backward.  Row n, with T the temperature and
// q = softmax(z / T):
//   no teacher_lse:  p_j = softmax over the kept tokens of t_j / T
//                    KD = sum_j p_j (log p_j - log q[id_j])
//   teacher_lse:     p_j = exp(t_j / T - lse), p_t = 1 - sum_j p_j, q_t = sum of q off the kept
//                    tokens;  KD = sum_j p_j (log p_j - log q[id_j]) + p_t (log p_t - log q_t)
//   loss  = sum_n w_n (alpha T^2 KD_n + (1 - alpha) (logsumexp(z_n) - z_n[label]))
//   dKD/dz_v = (M q_v - p_v) / T           on the kept tokens,  M = sum_j p_j + p_t
//            = q_v (M - p_t / q_t) / T     elsewhere (p_t = 0 without a tail)
//
// Many rows: one workgroup per row (distill_row_kernel).  The row stays in registers between its one
// read and the write of its gradient: V logits in, V gradients out is all the traffic, and what bounds it.
// Few rows, rows longer than the registers hold, and the two-call form: chunks of rows, one workgroup
// each.  distill_part_kernel takes a chunk's maximum and sums, distill_emit_kernel joins a row's chunks
// and writes a chunk's gradient; the logits are read twice, the second time mostly from cache.
//
// The kept tokens are marked in a bitmap in LDS.  It tells the sum over the tail which exponentials
// to leave out (q_t as a sum of its own: total minus kept would cancel), it finds repeated tokens,
// and it keeps the thread that writes a vector of gradients off the kept tokens, which their own
// threads write: no address is written twice, so nothing waits.
//
// Exponentials are 2^(z s - c) with c = m s rounded once: the rounding of c is a factor of every one
// and cancels in every softmax, as long as it is a moderate one (see Scale::at).  One exponential serves
// a row that needs one temperature (KD or CE alone, or T = 1); at T = 2 the one of CE is the square of
// KD's; otherwise CE takes a second one (`two`).
//
// With a tail the gradient off the kept tokens needs q_v / q_t.  Where the kept tokens stand so far above
// the rest that exponentials beside the row's maximum cannot hold it (cold_rest), the rest has a maximum of
// its own: one more pass over the registers, and its sum and gradients beside that one.
//
// Measured: 8192 x 50257 bf16, k = 64, tail and labels: 392 us for 1.65 GB, 4.2 TB/s (a large copy reaches 4.9); 27
// of them the loss kernel's one workgroup (under the profiler).
// Two workgroups of 512 threads a CU hold 13 vectors each in registers; the passes over them (maximum, sums,
// gradient) run while the other workgroup loads or stores.  Two calls over 2050 x 32003 fp32, k = 256: 205
// to 211 us (part 53 at 5.0 TB/s, statistics 13, gradient 131 at 4.0, loss 7).
// 16 x 50257 fp32: 18.6 us, three launches of 5, 9 and 2.
#include <algorithm>

#include "kron_internal.h"
#include "row_tile.h"

namespace kron {
namespace {

constexpr int kMaxK = kDistillMaxK;
constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.69314718055994531;

// stats of a row (8 floats), from the forward for the backward
enum { kStM = 0, kStInvT, kStInv1, kStBase, kStMass, kStTa, kStTb, kStRest, kStN = kDistillStats };

__device__ inline int64_t kept_id(const DistillArgs& a, int64_t row, int j) {
  const int64_t i = row * a.k + j;
  return a.ids64 ? ((const int64_t*)a.ids)[i] : (int64_t)((const int32_t*)a.ids)[i];
}

// e^x for x <= 0 in 64 bits: 2^n times a polynomial of the rest r = x - n ln 2, |r| <= ln 2 / 2 (the series to the
// 13th power is exact to 2^-58).  The rest is taken in two steps (Cody and Waite): ln 2 rounded to 40 binary places,
// whose product with n < 2^11 is exact, and what that leaves of ln 2.  Few registers, while the row holds most of them.
__device__ inline double exp64(double x) {
  if (x < -700.0) return 0.0;
  const double n = rint(x * 1.4426950408889634);
  const double r = fma(n, 1.7239444525614835e-13, fma(n, -0x1.62e42fefa4p-1, x));
  double p = 1.0 / 6227020800.0;
  const double c[13] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0,
                        1.0 / 5040.0,      1.0 / 720.0,      1.0 / 120.0,     1.0 / 24.0,     1.0 / 6.0,
                        0.5,               1.0,              1.0};
#pragma unroll
  for (int i = 0; i < 13; ++i) p = fma(p, r, c[i]);
  return ldexp(p, (int)n);
}

// Bits of vector j's kept tokens: the bitmap counts from a vector's first element, so a vector's bits
// are one byte (bf16) or half of one.
template <int VE>
__device__ inline uint32_t kept_bits(const uint32_t* bits, int j) {
  const uint8_t* b = reinterpret_cast<const uint8_t*>(bits);
  return VE == 8 ? b[j] : (b[j >> 1] >> (4 * (j & 1))) & 15u;
}

// How the exponentials of a row are taken.
struct Scale {
  bool kd, ce;
  int two;          // CE's exponential: 0 the first one, 1 its square, 2 one of its own
  float invT, sA;   // of the first exponential
  float m0, cA, cB; // the maximum, and the shifts
  bool far;

  __device__ Scale(const DistillArgs& a) {
    kd = a.alpha > 0.f;
    ce = a.alpha < 1.f;
    invT = 1.f / a.T;
    sA = kd ? invT * kLog2e : kLog2e;
    two = !(kd && ce) || a.T == 1.f ? 0 : a.T == 2.f ? 1 : 2;
  }
  // The rounding of c = m s stays in every exponential as a factor of up to 2^(half a unit of c): 2^8 below 2^28, but
  // no number any more for a row of -1e10 or -1e30.  From there on the maximum is subtracted first (exact next to it).
  __device__ void at(float m) {
    m0 = m;
    far = fabsf(m) < INFINITY && !(fabsf(m) * fmaxf(sA, kLog2e) < 0x1p28f);
    if (far) m = 0.f;
    cA = m * sA;
    cB = two == 1 ? 2.f * cA : m * kLog2e;
  }
  __device__ float place(float x) const { return far ? x - m0 : x; }
  // log2 of what takes sums of this shift to those of `to`, a larger maximum; sums of first exponentials, of CE's
  __device__ float change(const Scale& to, float s, float c, float cto) const {
    if (far) return to.far ? (m0 - to.m0) * s : fmaf(m0, s, -cto);
    return to.far ? -fmaf(to.m0, s, -c) : c - cto;
  }
  __device__ float changeA(const Scale& to) const { return change(to, sA, cA, to.cA); }
  __device__ float changeB(const Scale& to) const {
    return two == 0 ? changeA(to) : two == 1 ? 2.f * changeA(to) : change(to, kLog2e, cB, to.cB);
  }
  __device__ float first(float x) const { return __builtin_amdgcn_exp2f(fmaf(x, sA, -cA)); }
  __device__ float second(float x) const { return __builtin_amdgcn_exp2f(fmaf(x, kLog2e, -cB)); }
};

template <bool BF>
struct Sums {      // of first exponentials off the kept tokens, and of second ones
  using Tile = RowTile<BF>;
  static constexpr int VE = Tile::VE;
  float sr = 0.f, s1 = 0.f;
  __device__ void add(const Scale& c, const u32x4& v, uint32_t kept) {
    float x[VE], y[VE];
    Tile::values(v, x);
    if (c.far) {
#pragma unroll
      for (int e = 0; e < VE; ++e) x[e] = c.place(x[e]);
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) y[e] = c.first(x[e]);
    if (c.two == 1) {
#pragma unroll
      for (int e = 0; e < VE; ++e) s1 = fmaf(y[e], y[e], s1);
    } else if (c.two == 2) {
#pragma unroll
      for (int e = 0; e < VE; ++e) s1 += c.second(x[e]);
    }
    if (kept != 0u) {
#pragma unroll
      for (int e = 0; e < VE; ++e) y[e] = (kept >> e) & 1u ? 0.f : y[e];
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) sr += y[e];
  }
};

template <bool BF>
__device__ inline float vec_max(const u32x4& v) {
  float x[RowTile<BF>::VE];
  RowTile<BF>::values(v, x);
  float m = x[0];
#pragma unroll
  for (int e = 1; e < RowTile<BF>::VE; ++e) m = fmaxf(m, x[e]);
  return m;
}

// Whether the sum off the kept tokens, beside the whole maximum, is too small to be relied on: terms below
// 2^-126 are lost, and with them the gradients p_t q_v / q_t of tokens that have less than 2^-86 of the rest.
__device__ inline bool cold_rest(const DistillArgs& a, const Scale& c, float sr) {
  return c.kd && a.teacher_lse && sr < 0x1p-40f;
}
// The largest value of a vector off the kept tokens, and the sum of their first exponentials beside it.
template <bool BF>
__device__ inline float rest_max(const u32x4& v, uint32_t kept) {
  float x[RowTile<BF>::VE], m = -INFINITY;
  RowTile<BF>::values(v, x);
#pragma unroll
  for (int e = 0; e < RowTile<BF>::VE; ++e) m = (kept >> e) & 1u ? m : fmaxf(m, x[e]);
  return m;
}
template <bool BF>
__device__ inline float rest_sum(const Scale& c, const u32x4& v, uint32_t kept) {
  float x[RowTile<BF>::VE], s = 0.f;
  RowTile<BF>::values(v, x);
#pragma unroll
  for (int e = 0; e < RowTile<BF>::VE; ++e) s += (kept >> e) & 1u ? 0.f : c.first(c.place(x[e]));
  return s;
}

// Shared memory of a workgroup of NT threads; thread j < k has the row's kept token j.
template <int NT>
struct Shared {
  float red[NT / 64], redT[NT / 64], red1[NT / 64], redk[NT / 64], reds[NT / 64];
  double redp[NT / 64], redd[NT / 64];
  int32_t kid[kMaxK];
  float kp[kMaxK];
  int flag[4];        // a repeated token, a bad id, a used slot, the label is kept
};

struct Kept {
  int64_t id = -1;
  float t = 0.f, z = 0.f;
  bool have = false, own = false, near = false;      // near: inside this workgroup's chunk
};

template <int NT>
__device__ inline float block_max(float v, float* red) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = red[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) r = fmaxf(r, red[w]);
  return r;
}

// The rest's own maximum into cr (left as it is where the rest has no finite value) and its sum beside it into sr,
// over the vectors [j0, j1) in registers.
template <int NT, int NV, bool BF>
__device__ inline void rest_alone(u32x4 (&reg)[NV], int j0, int j1, const uint32_t* bits, Scale& cr, float& sr, Shared<NT>& sh) {
  constexpr int VE = RowTile<BF>::VE;
  const int tid = threadIdx.x;
  float m = -INFINITY;
  fresh(reg);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = tid + i * NT;
    if (j0 + j < j1) m = fmaxf(m, rest_max<BF>(reg[i], kept_bits<VE>(bits, j)));
  }
  m = block_max<NT>(m, sh.red);
  sr = 0.f;
  if (m == -INFINITY) return;
  cr.at(m);
  float s = 0.f;
  fresh(reg);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = tid + i * NT;
    if (j0 + j < j1) s += rest_sum<BF>(cr, reg[i], kept_bits<VE>(bits, j));
  }
  s = wave_sum(s);
  if ((tid & 63) == 0) sh.redT[tid >> 6] = s;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < NT / 64; ++v) sr += sh.redT[v];
}

// Clears the bitmap of the chunk [bit0, bit0 + 32 nwords) and marks the row's kept tokens in it
// (positions are token + off).  A barrier has to follow; then settle().
template <int NT, bool BF>
__device__ inline Kept mark_kept(const DistillArgs& a, int64_t row, const RowTile<BF>& z, int64_t lab, uint32_t* bits,
                                 int bit0, int nwords, Shared<NT>& sh) {
  const int tid = threadIdx.x;
  for (int i = tid; i < nwords; i += NT) bits[i] = 0u;
  if (tid < 4) sh.flag[tid] = 0;
  __syncthreads();
  Kept k;
  if (tid < a.k) {
    k.id = kept_id(a, row, tid);
    k.t = a.teacher[row * a.k + tid];
    if (k.id >= a.V) sh.flag[1] = 1;
    k.have = k.id >= 0 && k.id < a.V;
    if (k.have) {
      if (!(k.t == -INFINITY)) sh.flag[2] = 1;      // (a teacher of -infinity has p = 0)
      const int at = (int)k.id + z.off - bit0;
      k.near = at >= 0 && at < 32 * nwords;
      k.own = true;
      if (k.near) {
        const uint32_t bit = 1u << (at & 31);
        k.own = !(atomicOr(&bits[at >> 5], bit) & bit);
        if (!k.own) sh.flag[0] = 1;
      }
      if (k.id == lab) sh.flag[3] = 1;
    }
    sh.kid[tid] = k.have ? (int32_t)k.id : -1;
  }
  return k;
}
// Of a token given twice the first slot owns it, whichever came first to the bitmap.
template <int NT>
__device__ inline void settle(Kept& k, const Shared<NT>& sh) {
  if (!sh.flag[0] || !k.near) return;
  k.own = true;
  for (int l = 0; l < (int)threadIdx.x; ++l) k.own = k.own && sh.kid[l] != (int32_t)k.id;
}

// log p of a kept token and p, short of tb: `ta` is teacher_lse with a tail, else the teacher's largest value.  In 64
// bits, because t / T may be thousands.  (A teacher of -infinity has p = 0, also beside a teacher_lse of -infinity.)
__device__ inline double kept_p(const DistillArgs& a, const Kept& k, float ta, double& logp) {
  logp = 0.0;
  if (!k.have || k.t == -INFINITY) return 0.0;
  logp = a.teacher_lse ? (double)k.t / (double)a.T - (double)ta : ((double)k.t - (double)ta) / (double)a.T;
  return exp64(logp);
}

// What the gradient needs of a row.
struct RowStats {
  float invsT, invs1, base, mass, ta, tb;
};

// The row's sums into its statistics.  tr, t1: the sums off the kept tokens (beside the maximum of cr) and of the
// second exponentials (without one: anything); k.own marks each token once over the whole row.  Thread 0 leaves
// what the loss needs in a.rows[row].  zl: the label's logit (thread 0, if the label is one).
template <int NT>
__device__ inline RowStats finish_row(const DistillArgs& a, int64_t row, float w, const Scale& c, const Scale& cr, bool cold,
                                      const Kept& k, float tr, float t1, bool labok, float zl, Shared<NT>& sh) {
  constexpr int NW = NT / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  RowStats r;
  const bool tail = a.teacher_lse != nullptr;
  float tm = -INFINITY;
  if (c.kd && !tail) {
    tm = wave_max(k.have ? k.t : -INFINITY);
    if (lane == 0) sh.redk[wave] = tm;
  }
  const float sk = wave_sum(k.own ? c.first(k.z) : 0.f);
  if (lane == 0) sh.reds[wave] = sk;
  __syncthreads();
  float tk = 0.f;
#pragma unroll
  for (int v = 0; v < NW; ++v) tk += sh.reds[v];
  const float lift = cr.changeA(c);      // (0 but for a cold rest)
  const float total = (cold ? tr * __builtin_amdgcn_exp2f(lift) : tr) + tk;
  if (c.two == 0) t1 = total;
  r.invsT = 1.f / total;
  r.invs1 = 1.f / t1;
  r.ta = 0.f;
  r.tb = 1.f;
  r.mass = r.base = 1.f;
  double kl = 0.0, pmass = 0.0, ptail = 0.0;
  if (c.kd) {
    if (tail) {
      r.ta = a.teacher_lse[row];
    } else {
      tm = sh.redk[0];
#pragma unroll
      for (int v = 1; v < NW; ++v) tm = fmaxf(tm, sh.redk[v]);
      r.ta = sh.flag[2] ? tm : 0.f;
    }
    // the masses of the teacher are sums next to one: 64 bits, one exponential a thread
    double logp;
    const double pj = kept_p(a, k, r.ta, logp);
    if (threadIdx.x < a.k) sh.kp[threadIdx.x] = (float)pj;
    // sum p and sum p (log p - log q), log q short of the sum's logarithm
    const double lq = ((double)k.z * (double)c.sA - (double)c.cA) * kLn2;
    double term = pj != 0.0 ? pj * (logp - lq) : 0.0;
    const double sp = wave_sum(pj);
    term = wave_sum(term);
    if (lane == 0) { sh.redp[wave] = sp; sh.redd[wave] = term; }
    __syncthreads();
    double psum = 0.0;
#pragma unroll
    for (int v = 0; v < NW; ++v) { psum += sh.redp[v]; kl += sh.redd[v]; }
    if (!tail) {
      r.mass = r.base = sh.flag[2] ? 1.f : 0.f;
      r.tb = sh.flag[2] ? (float)(1.0 / psum) : 1.f;
      pmass = sh.flag[2] ? psum : 0.0;
    } else {
      // (with every token kept there is no tail, whatever rounding leaves of its mass)
      const bool rest = psum < 1.0 && !(tr == 0.f && a.k >= a.V);
      ptail = rest ? 1.0 - psum : 0.0;
      const double qt = cold ? (double)tr * exp64((double)lift * kLn2) / (double)total : 1.0;
      // Beside a q_t below 2^-80 what the rounding of teacher_lse (half a step, and the error of a sum in 32 bits) leaves
      // of p_t would be all of the loss, and infinite where the rest is masked: it is no mass.  (An infinity is exact.)
      if (qt < 0x1p-80 && fabsf(r.ta) < INFINITY && ptail <= 0x1p-20 + 0x1p-23 * fabs((double)r.ta)) ptail = 0.0;
      pmass = psum;
      r.mass = (float)(psum + ptail);
      r.base = r.mass;      // (a rest of -infinity throughout has gradient 0 whatever this is)
      if (cold && tr > 0.f)
        r.base = (float)(((double)r.mass * qt - ptail) * ((double)total / (double)tr));
      else if (!cold && ptail > 0.0)
        r.base = (float)((double)r.mass - ptail * ((double)total / (double)tr));
    }
  }
  const bool bad = sh.flag[1] || !labok;
  if (threadIdx.x == 0) {
    DistillRow o;
    o.kl = kl;
    o.psum = pmass;
    o.pt = ptail;
    o.total = total;
    o.rest = tr;
    o.t1 = t1;
    // the label's logit beside the maximum as CE's exponentials had it, in 64 bits: z s - c of the type's lowest value
    // is beyond 32
    const double s = c.two == 0 ? c.sA : c.two == 1 ? 2.f * c.sA : kLog2e;
    o.zl = !c.ce || !labok ? 0.f : (float)(((double)c.place(zl) * s - (double)(c.two == 0 ? c.cA : c.cB)) * kLn2);
    o.w = bad ? __builtin_nanf("") : w;
    o.lift = cold ? lift : 0.f;
    a.rows[row] = o;
  }
  if (bad) r.invsT = r.invs1 = __builtin_nanf("");
  return r;
}

// The gradient's factors of a row, `up` its weight times the upstream gradient; kb and cb are those of the
// exponentials off the kept tokens (beside cr's maximum).
struct Grad {
  float kw, cc, kc, kb, c1, cb;
  __device__ Grad(const DistillArgs& a, const Scale& c, const Scale& cr, const RowStats& r, float up) {
    kw = c.kd ? a.alpha * a.T * up : 0.f;
    cc = c.ce ? (1.f - a.alpha) * up : 0.f;
    kc = kw * r.invsT;
    kb = kc * r.base;
    c1 = cc * r.invs1;
    cb = cr.m0 == c.m0 ? c1 : c1 * __builtin_amdgcn_exp2f(cr.changeB(c));
  }
  // of a value: kq times the first exponential, and cq times CE's
  __device__ float one(const Scale& c, float x, float kq, float cq) const {
    const float y = c.first(x);
    if (c.two == 0) return y * (kq + cq);
    if (c.two == 1) return y * fmaf(y, cq, kq);
    return fmaf(y, kq, c.second(x) * cq);
  }
  template <bool BF>
  __device__ void vec(const Scale& c, const u32x4& v, float (&g)[RowTile<BF>::VE]) const {
    constexpr int VE = RowTile<BF>::VE;
    float x[VE];
    RowTile<BF>::values(v, x);
    if (c.far) {
#pragma unroll
      for (int e = 0; e < VE; ++e) x[e] = c.place(x[e]);
    }
    if (c.two == 0) {
#pragma unroll
      for (int e = 0; e < VE; ++e) g[e] = c.first(x[e]) * (kb + cb);
    } else if (c.two == 1) {
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float y = c.first(x[e]);
        g[e] = y * fmaf(y, cb, kb);
      }
    } else {
#pragma unroll
      for (int e = 0; e < VE; ++e) g[e] = fmaf(c.first(x[e]), kb, c.second(x[e]) * cb);
    }
  }
};

// Writes the gradients of the kept tokens near this workgroup, and of its label where that is not
// kept (zl: thread 0's, if `putlab`).  In place every gather has to be done before the first store of
// the workgroup: the gradients wait for the gathered logits, and written to LDS they are there before
// any thread passes the barrier.
template <int NT, bool BF>
__device__ inline void emit_kept(const DistillArgs& a, const Scale& c, const Scale& cr, const RowStats& r, const Grad& g, const Kept& k,
                                 int64_t lab, bool putlab, float zl, int bit0, const RowTile<BF>& z, const RowTile<BF>& o,
                                 uint32_t* bits, Shared<NT>& sh) {
  const int tid = threadIdx.x;
  __syncthreads();
  const bool mine = k.own && k.near;
  float gk = 0.f, gl = 0.f;
  if (mine) {
    float p = sh.kp[tid];      // (times tb)
    if (sh.flag[0])      // (the owner is the first slot)
      for (int l = tid + 1; l < a.k; ++l) p += sh.kid[l] == (int32_t)k.id ? sh.kp[l] : 0.f;
    gk = g.one(c, k.z, g.kc * r.mass, g.c1) - g.kw * (p * r.tb) - (k.id == lab ? g.cc : 0.f);
  }
  if (putlab) {
    gl = g.one(cr, cr.place(zl), g.kb, g.cb) - g.cc;
    const int at = (int)lab + z.off - bit0;
    atomicOr(&bits[at >> 5], 1u << (at & 31));
  }
  __syncthreads();      // (kp has been read)
  if (mine) sh.kp[tid] = gk;
  if (putlab) sh.redT[0] = gl;
  __syncthreads();
  if (mine) o.put((int)k.id, gk);
  if (putlab) o.put((int)lab, gl);
}

// A vector's gradients, element by element: those inside the row and not kept.
template <bool BF>
__device__ inline void emit_slow(const Scale& c, const Grad& g, int j, uint32_t kept, const RowTile<BF>& z,
                                 const RowTile<BF>& o) {
  constexpr int VE = RowTile<BF>::VE;
  float x[VE];
  g.vec<BF>(c, z.load(j), x);
  const int e0 = z.first(j);
#pragma unroll
  for (int e = 0; e < VE; ++e)
    if (e0 + e >= 0 && e0 + e < z.V && !((kept >> e) & 1u)) o.put(e0 + e, x[e]);
}

// Zero gradients for vectors [j0, j1) of a row.
template <bool BF>
__device__ inline void emit_zero(const RowTile<BF>& o, int j0, int j1, int nt) {
  for (int j = j0 + threadIdx.x; j < j1; j += nt) {
    if (o.inside(j)) {
      o.store(j, u32x4{0u, 0u, 0u, 0u});
    } else {
      for (int i = 0; i < RowTile<BF>::VE; ++i)
        if (o.first(j) + i >= 0 && o.first(j) + i < o.V) o.put(o.first(j) + i, 0.f);
    }
  }
}

// ---------------------------------------------------------------------------------
// One workgroup per row, the row in registers.
// ---------------------------------------------------------------------------------
template <bool BF, int NT, int NV>
__global__ __launch_bounds__(NT, 4) void distill_row_kernel(DistillArgs a) {
  using Tile = RowTile<BF>;
  constexpr int VE = Tile::VE;
  constexpr int NW = NT / 64;
  extern __shared__ uint32_t bits[];
  __shared__ Shared<NT> sh;
  const int64_t row = a.row0 + blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const float w = a.weights ? a.weights[row] : 1.f / (float)a.N;
  const Tile z(a.logits, row, a.ld, a.V), o(a.dlogits, row, a.ldd, a.V);
  if (w == 0.f) {      // a row without weight: nothing of it is read
    if (tid == 0) a.rows[row].w = 0.f;
    emit_zero<BF>(o, 0, o.vectors(), NT);
    return;
  }
  u32x4 reg[NV];
  const int nvec = z.vectors();
  z.template fetch<NT>(reg, tid, 0, nvec);
  Scale c(a);
  const int64_t lab = c.ce ? a.labels[row] : -1;
  const bool labok = !c.ce || (lab >= 0 && lab < a.V);
  Kept k = mark_kept<NT, BF>(a, row, z, lab, bits, 0, (a.V + z.off + 31) / 32, sh);
  if (k.have) k.z = z.at((int)k.id);
  const float zl = c.ce && labok && tid == 0 ? z.at((int)lab) : 0.f;

  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) mx = fmaxf(mx, vec_max<BF>(reg[i]));
  c.at(block_max<NT>(mx, sh.red));      // (its barrier also completes the bitmap)
  settle(k, sh);
  k.z = c.place(k.z);

  Sums<BF> s;
  fresh(reg);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = tid + i * NT;
    if (j < nvec) s.add(c, reg[i], c.kd ? kept_bits<VE>(bits, j) : 0u);
  }
  s.sr = wave_sum(s.sr);
  s.s1 = wave_sum(s.s1);
  if (lane == 0) { sh.red1[wave] = s.s1; sh.redT[wave] = s.sr; }
  __syncthreads();
  float tr = 0.f, t1 = 0.f;
#pragma unroll
  for (int v = 0; v < NW; ++v) { tr += sh.redT[v]; t1 += sh.red1[v]; }
  Scale cr = c;
  const bool cold = cold_rest(a, c, tr);
  if (cold) rest_alone<NT, NV, BF>(reg, 0, nvec, bits, cr, tr, sh);
  const RowStats r = finish_row<NT>(a, row, w, c, cr, cold, k, tr, t1, labok, zl, sh);

  const Grad g(a, c, cr, r, w);
  emit_kept<NT, BF>(a, c, cr, r, g, k, lab, c.ce && labok && tid == 0 && !sh.flag[3], zl, 0, z, o, bits, sh);
  // vectors without a kept token and inside the row go out whole; the others (a few) are read again, and
  // go out element by element.  (In place those are still as they were, but for the kept tokens.)
  const bool same = z.off == o.off;
  uint32_t left = 0u;
  fresh(reg);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = tid + i * NT;
    if (j < nvec) {
      if (same && kept_bits<VE>(bits, j) == 0u && z.inside(j)) {
        float x[VE];
        g.vec<BF>(cr, reg[i], x);
        o.store(j, Tile::packed(x));
      } else {
        left |= 1u << i;
      }
    }
  }
  while (left) {
    const int j = tid + (__ffs(left) - 1) * NT;
    emit_slow<BF>(cr, g, j, kept_bits<VE>(bits, j), z, o);
    left &= left - 1;
  }
}

// ---------------------------------------------------------------------------------
// Chunks of rows: workgroup (row, chunk) has the vectors [chunk cv, (chunk + 1) cv).
// ---------------------------------------------------------------------------------
constexpr int kCT = 256;      // threads
constexpr int kCV = 8;        // vectors of a thread at most
struct PartSum {
  float m, sr, s1;      // the maximum, and the sums beside it (sr beside mr)
  float mr;             // the maximum off the kept tokens where it is far below, else m
};

template <bool BF>
__global__ __launch_bounds__(kCT) void distill_part_kernel(DistillArgs a) {
  using Tile = RowTile<BF>;
  constexpr int VE = Tile::VE;
  __shared__ uint32_t bits[kCT * kCV * VE / 32];
  __shared__ Shared<kCT> sh;
  const int64_t row = a.row0 + blockIdx.x / a.chunks;
  const int chunk = (int)(blockIdx.x % a.chunks), tid = threadIdx.x;
  const float w = a.weights ? a.weights[row] : 1.f / (float)a.N;
  if (w == 0.f) return;
  const Tile z(a.logits, row, a.ld, a.V);
  const int j0 = chunk * a.cv, j1 = min(j0 + a.cv, z.vectors());
  u32x4 reg[kCV];
  z.template fetch<kCT>(reg, tid, j0, j1);
  Scale c(a);
  const int64_t lab = c.ce ? a.labels[row] : -1;
  const int bit0 = j0 * VE;
  Kept k = mark_kept<kCT, BF>(a, row, z, lab, bits, bit0, (max(j1 - j0, 0) * VE + 31) / 32, sh);
  if (k.near) a.zk[row * a.k + tid] = z.at((int)k.id);
  if (tid == 0 && c.ce && lab >= 0 && lab < a.V) {
    const int j = ((int)lab + z.off) / VE;
    if (j >= j0 && j < j1) a.zl[row] = z.at((int)lab);
  }
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < kCV; ++i) mx = fmaxf(mx, vec_max<BF>(reg[i]));
  const float m = block_max<kCT>(mx, sh.red);
  c.at(m);
  Sums<BF> s;
  fresh(reg);
  if (m > -INFINITY) {
#pragma unroll
    for (int i = 0; i < kCV; ++i) {
      const int j = j0 + tid + i * kCT;
      if (j < j1) s.add(c, reg[i], c.kd ? kept_bits<VE>(bits, j - j0) : 0u);
    }
  } else {      // a chunk of -infinity has no mass; one of NaN (which no maximum shows) has NaN
#pragma unroll
    for (int i = 0; i < kCV; ++i) {
      float x[VE];
      Tile::values(reg[i], x);
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (x[e] != x[e]) s.sr = s.s1 = x[e];
    }
  }
  s.sr = wave_sum(s.sr);
  s.s1 = wave_sum(s.s1);
  if ((tid & 63) == 0) { sh.red1[tid >> 6] = s.s1; sh.redT[tid >> 6] = s.sr; }
  __syncthreads();
  PartSum p{m, 0.f, 0.f, m};
#pragma unroll
  for (int v = 0; v < kCT / 64; ++v) { p.sr += sh.redT[v]; p.s1 += sh.red1[v]; }
  if (m > -INFINITY && cold_rest(a, c, p.sr)) {
    rest_alone<kCT, kCV, BF>(reg, j0, j1, bits, c, p.sr, sh);
    p.mr = p.sr > 0.f ? c.m0 : -INFINITY;
  }
  if (tid == 0) reinterpret_cast<PartSum*>(a.part)[row * a.chunks + chunk] = p;
}

// A row's chunks joined: the maximum into c, the sums rescaled to it; a cold rest's maximum into cr, and tr beside
// that.  One thread a chunk.
static_assert((kVocabMax / 4 + 2 + 2 * kCT - 1) / (2 * kCT) <= kCT, "a row's chunks fit one to a thread");
// A thread's sum at the maximum m, rescaled by `change` (log2) to another one; a NaN stays.
__device__ inline float rescaled(float sum, float m, float to, float change) {
  const float f = m == to ? 1.f : m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(change);
  return f > 0.f || sum != sum ? sum * f : 0.f;
}
__device__ inline void join_row(const DistillArgs& a, int64_t row, Scale& c, Scale& cr, bool& cold, float& tr, float& t1,
                                Shared<kCT>& sh) {
  const int tid = threadIdx.x;
  PartSum p{-INFINITY, 0.f, 0.f, -INFINITY};
  if (tid < a.chunks) p = reinterpret_cast<const PartSum*>(a.part)[row * a.chunks + tid];
  c.at(block_max<kCT>(p.m, sh.red));
  cr = c;
  Scale d = c, dr = c;      // the chunk's own shifts
  d.at(p.m);
  dr.at(p.mr);
  // (a row of -infinity throughout has no distribution: NaN)
  const float bad = c.m0 == -INFINITY ? __builtin_nanf("") : 0.f;
  const float x = wave_sum(rescaled(p.sr, p.mr, c.m0, dr.changeA(c)) + bad);
  const float y = wave_sum(rescaled(p.s1, p.m, c.m0, d.changeB(c)) + bad);
  if ((tid & 63) == 0) { sh.redT[tid >> 6] = x; sh.red1[tid >> 6] = y; }
  __syncthreads();
  tr = t1 = 0.f;
#pragma unroll
  for (int v = 0; v < kCT / 64; ++v) { tr += sh.redT[v]; t1 += sh.red1[v]; }
  cold = cold_rest(a, c, tr);
  if (!cold) return;
  tr = 0.f;
  const float m = block_max<kCT>(p.sr > 0.f ? p.mr : -INFINITY, sh.red);
  if (m == -INFINITY) return;
  cr.at(m);
  const float u = wave_sum(p.sr > 0.f ? rescaled(p.sr, p.mr, m, dr.changeA(cr)) : 0.f);
  if ((tid & 63) == 0) sh.redT[tid >> 6] = u;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kCT / 64; ++v) tr += sh.redT[v];
}

// STATS: joins the row's chunks and keeps the statistics (one workgroup a row, nothing emitted).
// JOIN: joins them and emits; else emits from kept statistics.
template <bool BF, bool STATS, bool JOIN>
__global__ __launch_bounds__(kCT) void distill_emit_kernel(DistillArgs a) {
  using Tile = RowTile<BF>;
  constexpr int VE = Tile::VE;
  __shared__ uint32_t bits[kCT * kCV * VE / 32];
  __shared__ int32_t seen[STATS || JOIN ? 2 * kMaxK : 1];      // the row's tokens, hashed
  __shared__ Shared<kCT> sh;
  const int64_t row = a.row0 + (STATS ? blockIdx.x : blockIdx.x / a.chunks);
  const int chunk = STATS ? 0 : (int)(blockIdx.x % a.chunks), tid = threadIdx.x;
  const float w = a.weights ? a.weights[row] : 1.f / (float)a.N;
  const Tile z(a.logits, row, a.ld, a.V), o(a.dlogits, row, a.ldd, a.V);
  const int j0 = chunk * a.cv, j1 = min(j0 + a.cv, z.vectors());
  if (w == 0.f) {
    if (STATS && tid < kStN) a.stats[row * kStN + tid] = 0.f;
    if ((STATS || JOIN) && chunk == 0 && tid == 0) a.rows[row].w = 0.f;
    // (the last chunk takes what rounding of the two starts to vectors leaves over)
    if (!STATS) emit_zero<BF>(o, j0, chunk == a.chunks - 1 ? o.vectors() : min(j0 + a.cv, o.vectors()), kCT);
    return;
  }
  u32x4 reg[STATS ? 1 : kCV];
  if (!STATS) {
#pragma unroll
    for (int i = 0; i < kCV; ++i) {
      const int j = j0 + tid + i * kCT;
      reg[STATS ? 0 : i] = j < j1 ? z.whole(j) : Tile::empty();
    }
  }
  Scale c(a), cr(a);
  const int64_t lab = c.ce ? a.labels[row] : -1;
  const bool labok = !c.ce || (lab >= 0 && lab < a.V);
  const int bit0 = j0 * VE;
  if (STATS || JOIN)
    for (int i = tid; i < 2 * kMaxK; i += kCT) seen[i] = -1;
  Kept k = mark_kept<kCT, BF>(a, row, z, lab, bits, bit0, STATS ? 0 : (max(j1 - j0, 0) * VE + 31) / 32, sh);
  const bool lnear = labok && c.ce && !STATS && ((int)lab + z.off) / VE >= j0 && ((int)lab + z.off) / VE < j1;
  float zl = 0.f, tr = 0.f, t1 = 0.f;
  RowStats r;
  if (STATS || JOIN) {
    // the gathered logits come from the parts: in place, other workgroups may have written theirs
    if (k.have) k.z = a.zk[row * a.k + tid];
    if (c.ce && labok) zl = a.zl[row];
    // over the whole row a token may be repeated far from this chunk (the table is twice what there can be:
    // a free place ends the search)
    if (k.have) {
      uint32_t h = (uint32_t)k.id * 2654435761u >> 23;
      static_assert(2 * kMaxK == 1 << (32 - 23), "the table's size");
      for (int old; (old = atomicCAS(&seen[h], -1, (int32_t)k.id)) != -1; h = (h + 1) % (2 * kMaxK))
        if (old == (int32_t)k.id) {
          sh.flag[0] = 1;
          break;
        }
    }
    bool cold;
    join_row(a, row, c, cr, cold, tr, t1, sh);      // (its barriers also complete the slots)
    if (k.have && sh.flag[0]) {
      k.own = true;
      for (int l = 0; l < tid; ++l) k.own = k.own && sh.kid[l] != (int32_t)k.id;
    }
    k.z = c.place(k.z);
    r = finish_row<kCT>(a, row, w, c, cr, cold, k, tr, t1, labok, zl, sh);
    if (STATS) {
      if (tid == 0) {
        float* st = a.stats + row * kStN;
        st[kStM] = c.m0; st[kStInvT] = r.invsT; st[kStInv1] = r.invs1;
        st[kStBase] = r.base; st[kStMass] = r.mass; st[kStTa] = r.ta; st[kStTb] = r.tb; st[kStRest] = cr.m0;
      }
      return;
    }
  } else {
    const float* st = a.stats + row * kStN;
    c.at(st[kStM]);
    cr.at(st[kStRest]);
    r.invsT = st[kStInvT]; r.invs1 = st[kStInv1]; r.base = st[kStBase];
    r.mass = st[kStMass]; r.ta = st[kStTa]; r.tb = st[kStTb];
    double logp;
    if (tid < a.k) sh.kp[tid] = (float)kept_p(a, k, r.ta, logp);
    if (k.near) k.z = c.place(z.at((int)k.id));
    if (lnear && tid == 0) zl = z.at((int)lab);
    __syncthreads();
    settle(k, sh);
  }
  const Grad g(a, c, cr, r, a.gout ? w * a.gout[0] : w);
  emit_kept<kCT, BF>(a, c, cr, r, g, k, lab, lnear && tid == 0 && !sh.flag[3], zl, bit0, z, o, bits, sh);
  const bool same = z.off == o.off;
  uint32_t left = 0u;
#pragma unroll
  for (int i = 0; i < kCV; ++i) {
    const int j = j0 + tid + i * kCT;
    if (j < j1) {
      if (same && kept_bits<VE>(bits, j - j0) == 0u && z.inside(j)) {
        float x[VE];
        g.vec<BF>(cr, reg[STATS ? 0 : i], x);
        o.store(j, Tile::packed(x));
      } else {
        left |= 1u << i;
      }
    }
  }
  while (left) {
    const int j = j0 + tid + (__ffs(left) - 1) * kCT;
    emit_slow<BF>(cr, g, j, kept_bits<VE>(bits, j - j0), z, o);
    left &= left - 1;
  }
}

// The rows' losses from their sums, added up by one workgroup in 64 bits in a fixed order.  (The
// logarithms stand here because 64-bit ones take registers that the rows' kernel has no room for.)
__global__ __launch_bounds__(1024) void distill_loss_kernel(DistillArgs a) {
  __shared__ double red[16];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < a.N; i += 1024) {
    const DistillRow r = a.rows[i];
    if (r.w == 0.f) continue;
    double l = 0.0;
    if (a.alpha > 0.f) {
      // sum p (log p - log q) with log q = (as summed) - log total, and p over its sum without a tail
      double kl = r.kl + r.psum * log((double)r.total);
      if (!a.teacher_lse)
        kl = r.psum > 0.0 ? kl / r.psum - log(r.psum) : 0.0;
      else if (r.pt > 0.0)
        kl += r.pt * (log(r.pt) - log((double)r.rest / (double)r.total) - (double)r.lift * kLn2);
      l += (double)a.alpha * (double)a.T * (double)a.T * kl;
    }
    if (a.alpha < 1.f) l += (1.0 - (double)a.alpha) * (log((double)r.t1) - (double)r.zl);
    s += (double)(float)((double)r.w * l);
  }
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int v = 0; v < 16; ++v) t += red[v];
    a.loss[0] = (float)t;
  }
}

int64_t max_vectors(int V, bool bf16) { return ((int64_t)V + 7) / (bf16 ? 8 : 4) + 1; }   // of a row that starts anywhere

// Rows in registers for enough rows to fill the GPU (two workgroups a CU), else chunks.  Loss and gradient, k = 64 and a
// tail, by rows and by chunks:
//   bf16       N = 16        256         512         1024         4096
//   5000       20 / 27    21 / 28     24 / 32      34 / 34     93 / 91 us
//   32003      26 / 26    28 / 35     34 / 44      57 / 69   171 / 210
//   50257      27 / 19    32 / 41     40 / 63     66 / 103   205 / 337
//   100003     31 / 26    40 / 56     68 / 86    125 / 145   465 / 495
//   fp32 50257 23 / 25    36 / 53     64 / 81    118 / 137   426 / 464
// (From 128 rows on rows have the better of it as well, 22 to 33 against 26 to 43 us; at 64 it is even.)
constexpr int kRowVectors = 13 * 1024;
bool whole_rows(const DistillArgs& a) { return a.N >= 512 && max_vectors(a.V, a.bf16) <= kRowVectors; }

// Vectors of a chunk: as many as a workgroup holds, fewer while there are not 1024 workgroups, at least two a
// thread.  Depends on the sizes alone.  (With 512 workgroups instead all sizes of the table below are within 5% but
// 512 x 5000, 29 us for 32; with 2048 bf16 32003 takes 44 and 52 us at 256 and 512 rows for 35 and 44, and 1024 x 5000
// 48 for 34.)
int chunk_vectors(int64_t N, int V, bool bf16) {
  const int64_t nv = max_vectors(V, bf16);
  int per = kCV;
  while (per > 2 && N * ((nv + per * kCT - 1) / (per * kCT)) < 1024) per /= 2;
  return per * kCT;
}

template <bool BF, int NT, int NV>
hipError_t launch_row(const DistillArgs& a, int64_t rows, hipStream_t s) {
  const size_t lds = ((size_t)a.V + 7 + 31) / 32 * 4;
  hipLaunchKernelGGL((distill_row_kernel<BF, NT, NV>), dim3((unsigned)rows), dim3(NT), lds, s, a);
  return hipGetLastError();
}

template <bool BF>
hipError_t launch_type(const DistillArgs& a, int mode, int64_t rows, hipStream_t s) {
  if (mode == 0 && whole_rows(a)) {
    const int64_t nv = max_vectors(a.V, BF);
    if (nv <= 4 * 512) return launch_row<BF, 512, 4>(a, rows, s);
    if (nv <= 7 * 512) return launch_row<BF, 512, 7>(a, rows, s);
    if (nv <= 10 * 512) return launch_row<BF, 512, 10>(a, rows, s);
    if (nv <= 13 * 512) return launch_row<BF, 512, 13>(a, rows, s);
    if (nv <= 8 * 1024) return launch_row<BF, 1024, 8>(a, rows, s);
    return launch_row<BF, 1024, 13>(a, rows, s);
  }
  const dim3 grid((unsigned)(rows * a.chunks)), nt(kCT);
  if (mode != 2) {
    hipLaunchKernelGGL((distill_part_kernel<BF>), grid, nt, 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (mode == 0)
    hipLaunchKernelGGL((distill_emit_kernel<BF, false, true>), grid, nt, 0, s, a);
  else if (mode == 1)
    hipLaunchKernelGGL((distill_emit_kernel<BF, true, true>), dim3((unsigned)rows), nt, 0, s, a);
  else
    hipLaunchKernelGGL((distill_emit_kernel<BF, false, false>), grid, nt, 0, s, a);
  return hipGetLastError();
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

size_t distill_workspace_bytes(int64_t N, int V, int k, bool bf16) {
  const int64_t chunks = (max_vectors(V, bf16) + chunk_vectors(N, V, bf16) - 1) / chunk_vectors(N, V, bf16);
  return up256(N * sizeof(DistillRow)) + up256(N * chunks * sizeof(PartSum)) + up256((size_t)N * k * 4) + up256(N * 4) + 256;
}

hipError_t launch_distill(DistillArgs a, int mode, void* ws, hipStream_t s) {
  a.cv = chunk_vectors(a.N, a.V, a.bf16);
  a.chunks = (int)((max_vectors(a.V, a.bf16) + a.cv - 1) / a.cv);
  if (mode != 2) {
    char* w = (char*)ws;
    a.rows = (DistillRow*)w;
    w += up256(a.N * sizeof(DistillRow));
    a.part = (float*)w;
    w += up256(a.N * a.chunks * sizeof(PartSum));
    a.zk = (float*)w;
    w += up256((size_t)a.N * a.k * 4);
    a.zl = (float*)w;
  }
  const int64_t most = kMaxGroups / a.chunks;
  for (a.row0 = 0; a.row0 < a.N; a.row0 += most) {
    const int64_t rows = std::min(most, a.N - a.row0);
    const hipError_t e = a.bf16 ? launch_type<true>(a, mode, rows, s) : launch_type<false>(a, mode, rows, s);
    if (e != hipSuccess) return e;
  }
  if (mode != 2) {
    hipLaunchKernelGGL(distill_loss_kernel, dim3(1), dim3(1024), 0, s, a);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace kron
