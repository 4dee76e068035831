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
// One workgroup per row.  The row stays in registers between its one read and the write of its
// gradient; only rows longer than the registers hold are read twice more.  What bounds it is
// memory: V logits in, V gradients out.
//
// The kept tokens are marked in a bitmap of the row in LDS.  It tells the sum over the tail
// which exponentials to leave out (q_t as a sum of its own: total minus kept would cancel), it
// finds repeated tokens, and it keeps the thread that writes a vector of gradients off the kept
// tokens, which their own threads write: no address is written twice, so nothing waits.
#include "kron_internal.h"
#include "row_tile.h"

namespace kron {
namespace {

constexpr int kMaxK = kDistillMaxK;
constexpr float kLog2e = 1.4426950408889634f;

// stats of a row (8 floats), from the forward for the backward
enum { kStM = 0, kStInvT, kStInv1, kStBase, kStMass, kStTa, kStTb, kStBad, kStN };

__device__ inline int64_t kept_id(const DistillArgs& a, int64_t row, int j) {
  const int64_t i = row * a.k + j;
  return a.ids64 ? ((const int64_t*)a.ids)[i] : (int64_t)((const int32_t*)a.ids)[i];
}

// The packed row as new values: what one pass unpacked is not kept for the next (it would take
// twice the row's registers or more).
template <int NV>
__device__ inline void fresh(u32x4 (&reg)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) asm volatile("" : "+v"(reg[i]));
}

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

// MODE 0: loss and gradient;  1: loss and stats;  2: gradient from stats
template <bool BF, int NT, int NV, bool RES, int MODE>
__global__ __launch_bounds__(NT) void distill_kernel(DistillArgs a) {
  using Tile = RowTile<BF>;
  constexpr int VE = Tile::VE;
  constexpr int NW = NT / 64;
  extern __shared__ uint32_t bits[];      // bitmap of the kept tokens, (V + 31) / 32 + 1 words
  __shared__ float red[NW], redT[NW], red1[NW], redk[NW];
  __shared__ double redp[NW], redd[NW];
  __shared__ int32_t kid[kMaxK];
  __shared__ float kp[kMaxK];             // p of the kept tokens
  __shared__ int sflag[4];                // a repeated token, a bad id, a used slot, the label is kept

  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const float w = a.weights ? a.weights[row] : 1.f / (float)a.N;
  const Tile z(a.logits, row, a.ld, a.V);
  const int nvec = z.vectors();
  if (w == 0.f) {      // a row without weight: nothing of it is read
    if (MODE != 2 && tid == 0) a.lossrow[row] = 0.f;
    if (MODE == 1 && tid < kStN) a.stats[row * kStN + tid] = 0.f;
    if (MODE != 1) {
      const Tile o(a.dlogits, row, a.ldd, a.V);
      const int no = o.vectors();
      for (int j = tid; j < no; j += NT) {
        if (o.inside(j)) {
          *reinterpret_cast<u32x4*>(o.base + (uint64_t)j * 16) = u32x4{0u, 0u, 0u, 0u};
        } else {
          for (int i = 0; i < VE; ++i)
            if (o.first(j) + i >= 0 && o.first(j) + i < a.V) o.put(o.first(j) + i, 0.f);
        }
      }
    }
    return;
  }

  u32x4 reg[RES ? NV : 1];
  if (RES) {
#pragma unroll
    for (int i = 0; i < NV; ++i) reg[RES ? i : 0] = z.load(tid + i * NT);
  }
  const float invT = 1.f / a.T, sT = invT * kLog2e;
  const bool kd = a.alpha > 0.f, ce = a.alpha < 1.f;
  const int nwords = (a.V + 31) / 32 + 1;
  for (int i = tid; i < nwords; i += NT) bits[i] = 0u;
  if (tid < 4) sflag[tid] = 0;
  __syncthreads();

  // the kept tokens: thread j < k has token j
  const int64_t lab = ce ? a.labels[row] : -1;
  int64_t id = -1;
  float t = 0.f, zk = 0.f;
  bool have = false, own = false;
  if (kd && tid < a.k) {
    id = kept_id(a, row, tid);
    t = a.teacher[row * a.k + tid];
    if (id >= a.V) sflag[1] = 1;
    have = id >= 0 && id < a.V;
    if (have) {
      if (!(t == -INFINITY)) sflag[2] = 1;      // (a teacher of -infinity has p = 0)
      zk = z.at((int)id);
      const uint32_t bit = 1u << (id & 31);
      own = !(atomicOr(&bits[id >> 5], bit) & bit);
      if (!own) sflag[0] = 1;
      if (id == lab) sflag[3] = 1;
    }
    kid[tid] = have ? (int32_t)id : -1;
  }
  // of a token given twice the first slot owns it, whichever came first to the bitmap
  auto settle = [&]() {
    if (!sflag[0] || !have) return;
    own = true;
    for (int l = 0; l < tid; ++l) own = own && kid[l] != (int32_t)id;
  };
  const bool labok = !ce || (lab >= 0 && lab < a.V);

  float m, invsT, invs1 = 0.f, base, mass, ta, tb;
  if (MODE == 2) {
    const float* st = a.stats + row * kStN;
    m = st[kStM]; invsT = st[kStInvT]; invs1 = st[kStInv1];
    base = st[kStBase]; mass = st[kStMass]; ta = st[kStTa]; tb = st[kStTb];
    __syncthreads();
    settle();
  } else {
    // the row's maximum
    float mx = -INFINITY;
    if (RES) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) mx = fmaxf(mx, Tile::value(reg[RES ? i : 0], e));
    } else {
      for (int j = tid; j < nvec; j += NT) {
        const u32x4 v = z.load(j);
#pragma unroll
        for (int e = 0; e < VE; ++e) mx = fmaxf(mx, Tile::value(v, e));
      }
    }
    m = block_max<NT>(mx, red);      // (its barrier also completes the bitmap)
    settle();
    fresh(reg);
    // sums of exp((z - m) / T) off and on the kept tokens, and of exp(z - m)
    float sr = 0.f, sk = 0.f, s1 = 0.f;
    auto add = [&](const u32x4& v, int j) {
      const int e0 = z.first(j);
      uint32_t b = 0u;
      if (kd && e0 < a.V) {
        const int f = e0 < 0 ? 0 : e0;
        const uint64_t two = (uint64_t)bits[f >> 5] | ((uint64_t)bits[(f >> 5) + 1] << 32);
        b = (uint32_t)(two >> (f & 31)) << (f - e0);
      }
      float p = 0.f, o = 0.f;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float d = Tile::value(v, e) - m;
        if (kd) {
          const float x = __builtin_amdgcn_exp2f(d * sT);
          p += (b >> e) & 1u ? 0.f : x;
        }
        if (ce) o += __builtin_amdgcn_exp2f(d * kLog2e);
      }
      sr += p;
      s1 += o;
    };
    if (RES) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (tid + i * NT < nvec) add(reg[RES ? i : 0], tid + i * NT);
    } else {
      for (int j = tid; j < nvec; j += NT) add(z.load(j), j);
    }
    if (own) sk = __builtin_amdgcn_exp2f((zk - m) * sT);
    // the teacher's p: over the kept tokens, or with the rest of the vocabulary
    const bool tail = a.teacher_lse != nullptr;
    float tm = -INFINITY;
    if (kd && !tail) {
      tm = have ? t : -INFINITY;
      tm = wave_max(tm);
      if (lane == 0) redk[wave] = tm;
    }
    sr = wave_sum(sr);
    s1 = wave_sum(s1);
    sk = wave_sum(sk);
    if (lane == 0) { red1[wave] = s1; redT[wave] = sr; redp[wave] = (double)sk; }
    __syncthreads();
    float tr = 0.f, tk = 0.f, t1 = 0.f;
#pragma unroll
    for (int v = 0; v < NW; ++v) { tr += redT[v]; tk += (float)redp[v]; t1 += red1[v]; }
    const float total = tr + tk;
    invsT = 1.f / total;
    invs1 = 1.f / t1;
    double pj = 0.0, logp = 0.0;
    if (kd) {
      if (tail) {
        ta = a.teacher_lse[row];
        tb = 1.f;
      } else {
        tm = redk[0];
#pragma unroll
        for (int v = 1; v < NW; ++v) tm = fmaxf(tm, redk[v]);
        ta = sflag[2] ? tm * invT : 0.f;
        tb = 1.f;
      }
    } else {
      ta = 0.f; tb = 1.f;
    }
    // the masses of the teacher are sums next to one: 64 bits, one exponential a thread
    if (have && !(t == -INFINITY)) {
      logp = (double)t / (double)a.T - (double)(tail ? ta : 0.f);
      if (!tail) logp = ((double)t - (double)tm) / (double)a.T;
      pj = exp(logp);
    }
    double sp = wave_sum(pj);
    __syncthreads();
    if (lane == 0) redp[wave] = sp;
    __syncthreads();
    double psum = 0.0;
#pragma unroll
    for (int v = 0; v < NW; ++v) psum += redp[v];
    if (kd && !tail && sflag[2]) {
      tb = (float)(1.0 / psum);
      pj /= psum;
      logp -= log(psum);
    }
    // the row's divergence
    const double ltot = (double)logf(total);
    double term = 0.0;
    if (have && pj != 0.0) term = pj * (logp - ((double)(zk - m) * (double)invT - ltot));
    term = wave_sum(term);
    if (lane == 0) redd[wave] = term;
    __syncthreads();
    double kl = 0.0;
#pragma unroll
    for (int v = 0; v < NW; ++v) kl += redd[v];
    mass = 1.f;
    base = 1.f;
    if (kd) {
      if (!tail) {
        mass = base = sflag[2] ? 1.f : 0.f;
      } else {
        // (with every token kept there is no tail, whatever rounding leaves of its mass)
        const bool rest = psum < 1.0 && !(tr == 0.f && a.k >= a.V);
        const double pt = rest ? 1.0 - psum : 0.0;
        mass = (float)(psum + pt);
        base = mass;
        if (rest) {
          const double qt = (double)tr / (double)total;
          kl += pt * (log(pt) - log(qt));
          base = (float)((double)mass - pt / qt);
        }
      }
    }
    const bool bad = sflag[1] || !labok;
    if (tid == 0) {
      double l = 0.0;
      if (kd) l += (double)a.alpha * (double)a.T * (double)a.T * kl;
      if (ce && labok) l += (1.0 - (double)a.alpha) * ((double)logf(t1) - (double)(z.at((int)lab) - m));
      a.lossrow[row] = bad ? __builtin_nanf("") : (float)((double)w * l);
    }
    if (bad) invsT = invs1 = __builtin_nanf("");
    if (MODE == 1) {
      if (tid == 0) {
        float* st = a.stats + row * kStN;
        st[kStM] = m; st[kStInvT] = invsT; st[kStInv1] = invs1;
        st[kStBase] = base; st[kStMass] = mass; st[kStTa] = ta; st[kStTb] = tb; st[kStBad] = bad ? 1.f : 0.f;
      }
      return;
    }
  }

  // the gradient; kc = alpha w T and cc = (1 - alpha) w, times the upstream gradient
  const float up = MODE == 2 ? w * a.gout[0] : w;
  const float kc = kd ? a.alpha * a.T * up * invsT : 0.f, cc = ce ? (1.f - a.alpha) * up : 0.f;
  const float kb = kc * base, c1 = cc * invs1;
  if (kd && tid < a.k)
    kp[tid] = have ? __builtin_amdgcn_exp2f((t * invT - ta) * kLog2e) * tb : 0.f;
  __syncthreads();
  const Tile o(a.dlogits, row, a.ldd, a.V);
  const bool same = z.off == o.off;      // both rows start at the same place of a vector
  float zl = 0.f;
  const bool putlab = ce && labok && tid == 0 && !sflag[3];
  if (putlab) zl = z.at((int)lab);
  // in place, every gather of the row is done before the first store
  float mine = 0.f;
  if (own) {
    float p = kp[tid];
    if (sflag[0])      // (the owner is the first slot)
      for (int l = tid + 1; l < a.k; ++l) p += kid[l] == (int32_t)id ? kp[l] : 0.f;
    const float d = zk - m;
    const float pk = a.alpha * a.T * up * p;
    mine = __builtin_amdgcn_exp2f(d * sT) * kc * mass - pk;
    if (ce) mine += __builtin_amdgcn_exp2f(d * kLog2e) * c1 - (id == lab ? cc : 0.f);
  }
  float labv = 0.f;
  if (putlab) {
    const float d = zl - m;
    labv = (kd ? __builtin_amdgcn_exp2f(d * sT) * kb : 0.f) + __builtin_amdgcn_exp2f(d * kLog2e) * c1 - cc;
    atomicOr(&bits[lab >> 5], 1u << (lab & 31));
  }
  // the values above wait for the gathered logits: written to LDS, they are there before any
  // thread passes the barrier
  if (own) kp[tid] = mine;
  if (putlab) redT[0] = labv;
  __syncthreads();
  if (own) o.put((int)id, mine);
  if (putlab) o.put((int)lab, labv);
  auto emit = [&](const u32x4& v, int j) {
    const int e0 = z.first(j);
    if (e0 >= a.V) return;
    const int f = e0 < 0 ? 0 : e0;
    const uint64_t two = (uint64_t)bits[f >> 5] | ((uint64_t)bits[(f >> 5) + 1] << 32);
    const uint32_t b = ((uint32_t)(two >> (f & 31)) << (f - e0)) & ((1u << VE) - 1u);
    float g[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float d = Tile::value(v, e) - m;
      float x = 0.f;
      if (kd) x = __builtin_amdgcn_exp2f(d * sT) * kb;
      if (ce) x = fmaf(__builtin_amdgcn_exp2f(d * kLog2e), c1, x);
      g[e] = x;
    }
    if (same && b == 0u && z.inside(j)) {
      u32x4 r;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r[i] = BF ? (bf16_rne(g[(2 * i) % VE]) | (bf16_rne(g[(2 * i + 1) % VE]) << 16)) : __float_as_uint(g[i]);
      *reinterpret_cast<u32x4*>(o.base + (uint64_t)j * 16) = r;
    } else {
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (e0 + e >= 0 && e0 + e < a.V && !((b >> e) & 1u)) o.put(e0 + e, g[e]);
    }
  };
  if (RES) {
    fresh(reg);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (tid + i * NT < nvec) emit(reg[RES ? i : 0], tid + i * NT);
  } else {
    for (int j = tid; j < nvec; j += NT) emit(z.load(j), j);
  }
}

// The rows' losses, summed by one workgroup in 64 bits in a fixed order.
__global__ __launch_bounds__(1024) void distill_loss_kernel(int64_t N, const float* __restrict__ lossrow,
                                                            float* __restrict__ loss) {
  __shared__ double red[16];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < N; i += 1024) s += (double)lossrow[i];
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int v = 0; v < 16; ++v) t += red[v];
    loss[0] = (float)t;
  }
}

template <bool BF, int NT, int NV, bool RES>
hipError_t launch_mode(const DistillArgs& a, int mode, size_t lds, hipStream_t s) {
  const dim3 grid((unsigned)a.N);
  if (mode == 0)
    hipLaunchKernelGGL((distill_kernel<BF, NT, NV, RES, 0>), grid, dim3(NT), lds, s, a);
  else if (mode == 1)
    hipLaunchKernelGGL((distill_kernel<BF, NT, NV, RES, 1>), grid, dim3(NT), lds, s, a);
  else
    hipLaunchKernelGGL((distill_kernel<BF, NT, NV, RES, 2>), grid, dim3(NT), lds, s, a);
  return hipGetLastError();
}

template <bool BF>
hipError_t launch_type(const DistillArgs& a, int mode, hipStream_t s) {
  const size_t lds = ((size_t)(a.V + 31) / 32 + 1) * 4;
  const int64_t nvec = ((int64_t)a.V + 7) / (BF ? 8 : 4) + 1;   // of a row that starts anywhere
  if (nvec <= 256 * 8) return launch_mode<BF, 256, 8, true>(a, mode, lds, s);
  if (nvec <= 512 * 16) return launch_mode<BF, 512, 16, true>(a, mode, lds, s);
  if (nvec <= 1024 * 16) return launch_mode<BF, 1024, 16, true>(a, mode, lds, s);
  return launch_mode<BF, 1024, 1, false>(a, mode, lds, s);
}

}  // namespace

hipError_t launch_distill(const DistillArgs& a, int mode, hipStream_t s) {
  if (a.N > 0) {
    const hipError_t e = a.bf16 ? launch_type<true>(a, mode, s) : launch_type<false>(a, mode, s);
    if (e != hipSuccess) return e;
  }
  if (mode != 2) {
    hipLaunchKernelGGL(distill_loss_kernel, dim3(1), dim3(1024), 0, s, a.N, a.lossrow, a.loss);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace kron
