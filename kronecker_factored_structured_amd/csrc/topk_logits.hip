// The k largest logits of each row of z (N x V), with their tokens, and lse = log sum_v exp(z_v / T):
// what a teacher's answer is kept as for distillation.  Order: largest first, equal values by the
// lower token; -0 equals 0, and a NaN stands above every number.
//
// One workgroup per row; the row is read once into registers.  Each thread's own maximum is a
// lower bound's witness: the k-th largest of the threads' maxima is a threshold that at least k
// values reach, and for k below the thread count few more do (for values in random order about
// NT ln(NT / (NT - k)) in all).  Those candidates go to LDS and are ranked by counting.  Rows
// that defeat the threshold (many equal values, the top in few threads, fewer vectors than k) and
// rows with a NaN, an infinite maximum or one that is large against T take an exact bisection on the value's
// key, then on the token among the equal ones.  Rows beyond 13 vectors a thread are read twice, the second time mostly from cache.
//
// Measured: 8192 x 50257 bf16, k = 64: 233 us, 3.56 TB/s (a large sum reads at 4.0; vector instructions fill 0.65 of the
// time under the profiler); 257 x 131072 fp32, k = 256: 59 us, 55 of them the kernel under the profiler (28 at a copy's
// rate; one workgroup a CU passes twice over its row); one row of 50257 bf16 values 10.4 us, the latency of one
// workgroup's passes.  Cutting long rows into chunks and joining
// their tops took 61 to 80 us at 257 rows (each chunk ranks k candidates of its own) and 276 instead of 363 at
// 2048 rows, k = 64; one row cut over six workgroups 15.6 us: not kept.
#include <algorithm>

#include "kron_internal.h"
#include "row_tile.h"

namespace kron {
namespace {

constexpr int kCap = 1024;      // candidates held in LDS
constexpr float kLog2e = 1.4426950408889634f;

// An order-preserving key: a < b as values iff key(a) < key(b); 0 is below every value's key.
__device__ inline uint32_t key_of(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t u = __float_as_uint(f == 0.f ? 0.f : f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ inline float value_of(uint32_t k) {
  if (k == 0xffffffffu) return __uint_as_float(0x7fc00000u);
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <bool BF, int NT, int NV, bool RES>
__global__ __launch_bounds__(NT, 4) void topk_kernel(TopkArgs a) {
  using Tile = RowTile<BF>;
  constexpr int VE = Tile::VE;
  constexpr int NW = NT / 64;
  __shared__ alignas(16) uint64_t cand[kCap];      // key, then the complement of the token: larger is better
  __shared__ uint32_t tmax[NT];
  __shared__ float red[NW];
  __shared__ uint32_t cnt[2][NW];
  __shared__ uint32_t ncand, tau_s, top_s;

  const int64_t row = a.row0 + blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Tile z(a.logits, row, a.ld, a.V);
  const int nvec = z.vectors();
  u32x4 reg[RES ? NV : 1];
  if constexpr (RES) z.template fetch<NT>(reg, tid, 0, nvec);
  // calls f(vector, its index) for each of this thread's vectors
  auto each_vec = [&](auto f) {
    if constexpr (RES) {
      fresh(reg);
      int first = tid;      // (a new value as well: the masks of every vector's and value's place are not kept either)
      asm volatile("" : "+v"(first));
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (first + i * NT < nvec) f(reg[i], first + i * NT);
    } else {
      for (int j = tid; j < nvec; j += NT) f(z.load(j), j);
    }
  };
  // calls f(value, token) for each of this thread's values
  auto each = [&](auto f) {
    each_vec([&](const u32x4& v, int j) {
      const int e0 = z.first(j);
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (e0 + e >= 0 && e0 + e < a.V) f(Tile::value(v, e), e0 + e);
    });
  };
  int turn = 0;
  auto total = [&](uint32_t c) -> uint32_t {      // over the workgroup
#pragma unroll
    for (int o = 32; o >= 1; o /= 2) c += __shfl_xor(c, o, 64);
    turn ^= 1;      // (the other half is still being read)
    if (lane == 0) cnt[turn][wave] = c;
    __syncthreads();
    uint32_t s = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) s += cnt[turn][w];
    return s;
  };
  auto keep = [&](uint32_t key, int e) {
    const uint32_t at = atomicAdd(&ncand, 1u);
    if (at < kCap) cand[at] = ((uint64_t)key << 32) | (uint32_t)~(uint32_t)e;
  };

  float mx = -INFINITY;      // (a NaN does not show: the sum tells)
  each_vec([&](const u32x4& v, int) {
    float x[VE];
    Tile::values(v, x);
#pragma unroll
    for (int e = 0; e < VE; e += 2) mx = fmaxf(mx, fmaxf(x[e], x[e + 1]));
  });
  tmax[tid] = tid < nvec ? key_of(mx) : 0u;
  if (tid == 0) ncand = 0u;
  __syncthreads();
  // wave 0: the largest 16-bit prefix that at least k of the threads' maxima reach
  if (wave == 0) {
    uint32_t mine[NW], top = 0u;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      mine[i] = tmax[lane + 64 * i];
      top = mine[i] > top ? mine[i] : top;
    }
#pragma unroll
    for (int o = 32; o >= 1; o /= 2) {
      const uint32_t x = __shfl_xor(top, o, 64);
      top = x > top ? x : top;
    }
    uint32_t t = 0u;
    for (int b = 31; b >= 16; --b) {
      const uint32_t c = t | (1u << b);
      int n = 0;
#pragma unroll
      for (int i = 0; i < NW; ++i) n += __popcll(__ballot(mine[i] >= c));
      if (n >= a.k) t = c;
    }
    if (lane == 0) {
      tau_s = t;
      top_s = top;
    }
  }
  __syncthreads();
  const float m = value_of(top_s);
  const float sT = kLog2e / a.T, c = m * sT;
  // the sum, and the candidates.  Below this threshold (or with k >= 2^16 of no witness) it says nothing.
  // The rounding of c is a factor of up to 2^(half a unit of c) of the sum: 2^8 below 2^28, but no number any more for
  // a row of -1e10 or -1e30.  From there on the maximum is subtracted first (exact next to it).
  const bool finite = fabsf(c) < 0x1p28f;
  const bool use = finite && tau_s > key_of(-INFINITY);
  const float tau_f = use ? value_of(tau_s) : INFINITY;
  float s = 0.f;
  if (finite) {
    each_vec([&](const u32x4& v, int j) {
      float x[VE];
      Tile::values(v, x);
      float h = x[0];
#pragma unroll
      for (int e = 1; e < VE; ++e) h = fmaxf(h, x[e]);
#pragma unroll
      for (int e = 0; e < VE; ++e) s += __builtin_amdgcn_exp2f(fmaf(x[e], sT, -c));
      if (h >= tau_f) {      // (the padding of a partial vector is -infinity)
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (x[e] >= tau_f) keep(key_of(x[e]), z.first(j) + e);
      }
    });
  } else {
    const bool some = fabsf(m) < INFINITY;
    each([&](float f, int) { s += f != f ? f : some ? __builtin_amdgcn_exp2f((f - m) * sT) : f == m ? 1.f : 0.f; });
  }
  s = wave_sum(s);
  if (lane == 0) red[wave] = s;
  __syncthreads();
  s = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) s += red[w];
  if (tid == 0) {
    // m / T + ln s, less what the exponentials' rounded shift and scale put into s beside 2^((x - m) sT)
    double base = (double)m / (double)a.T;
    if (finite) base -= ((double)m * (double)sT - (double)c) * 0.69314718055994531;
    a.lse[row] = (float)(base + (double)logf(s));
  }
  uint32_t nc = ncand;
  if (!use || s != s || nc > kCap) {
    // the k-th largest key exactly: tau = max {t : at least k keys >= t}
    uint32_t tau = 0u;
    for (int b = 31; b >= 0; --b) {
      const uint32_t t = tau | (1u << b);
      uint32_t n = 0;
      each([&](float f, int) { n += key_of(f) >= t ? 1u : 0u; });
      if (total(n) >= (uint32_t)a.k) tau = t;
    }
    uint32_t above = 0;
    each([&](float f, int) { above += key_of(f) > tau ? 1u : 0u; });
    const uint32_t need = (uint32_t)a.k - total(above);      // of the equal ones: those with the lowest tokens
    int lim = 0;      // the largest lim such that fewer than `need` equal ones stand below token lim
    for (int b = 17; b >= 0; --b) {
      const int t = lim + (1 << b);
      if (t >= a.V) continue;
      uint32_t n = 0;
      each([&](float f, int e) { n += (key_of(f) == tau && e < t) ? 1u : 0u; });
      if (total(n) < need) lim = t;
    }
    __syncthreads();
    if (tid == 0) ncand = 0u;
    __syncthreads();
    each([&](float f, int e) {
      const uint32_t k = key_of(f);
      if (k > tau || (k == tau && e <= lim)) keep(k, e);
    });
    __syncthreads();
    nc = ncand < (uint32_t)kCap ? ncand : (uint32_t)kCap;      // (exactly k)
  }
  // a candidate's place is the number of better ones (all are distinct: the tokens differ)
  if (tid < 8 && nc + tid < kCap) cand[nc + tid] = 0;
  __syncthreads();
  for (uint32_t i = tid; i < nc; i += NT) {
    const uint64_t x = cand[i];
    int place = 0;
    for (uint32_t l = 0; l < nc; l += 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) place += cand[l + j] > x ? 1 : 0;
    }
    if (place < a.k) {
      a.ids[row * a.k + place] = (int32_t)~(uint32_t)x;
      a.vals[row * a.k + place] = value_of((uint32_t)(x >> 32));
    }
  }
}

// Registers by the row's vectors: fewer of them let more workgroups on a CU.  4096 rows, k = 64, with 4, 8 and 13 vectors
// a thread and with 1024 threads: 5000 bf16 values 46, 50, 65 and 132 us; 16000 59, 61, 81 and 151; 32003 - , 82, 107 and
// 190; 50257 -, -, 127 and 217.  1024 threads hold 100003 bf16 values in 298 us and read them twice in 269, 32003 fp32
// ones in 202 and 172, 50257 in 250 and 248; up to 512 rows the two are within 8% of each other, either way.
template <bool BF>
hipError_t launch_type(const TopkArgs& a, int64_t rows, hipStream_t s) {
  const int64_t nvec = ((int64_t)a.V + 7) / (BF ? 8 : 4) + 1;   // of a row that starts anywhere
  const dim3 grid((unsigned)rows);
  if (nvec <= 512 * 4)
    hipLaunchKernelGGL((topk_kernel<BF, 512, 4, true>), grid, dim3(512), 0, s, a);
  else if (nvec <= 512 * 8)
    hipLaunchKernelGGL((topk_kernel<BF, 512, 8, true>), grid, dim3(512), 0, s, a);
  else if (nvec <= 512 * 13)
    hipLaunchKernelGGL((topk_kernel<BF, 512, 13, true>), grid, dim3(512), 0, s, a);
  else if (nvec <= 1024 * 13)
    hipLaunchKernelGGL((topk_kernel<BF, 1024, 13, true>), grid, dim3(1024), 0, s, a);
  else
    hipLaunchKernelGGL((topk_kernel<BF, 1024, 1, false>), grid, dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_topk(TopkArgs a, hipStream_t s) {
  for (a.row0 = 0; a.row0 < a.N; a.row0 += kMaxGroups) {
    const int64_t rows = std::min(kMaxGroups, a.N - a.row0);
    const hipError_t e = a.bf16 ? launch_type<true>(a, rows, s) : launch_type<false>(a, rows, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace kron
