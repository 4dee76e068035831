// The k largest logits of each row of z (N x V), with their tokens, and lse = log sum_v exp(z_v / T):
// what a teacher's answer is kept as for distillation.  Order: largest first, equal values by the
// lower token; -0 equals 0, and a NaN stands above every number.
//
// One workgroup per row; the row is read once into registers.  Each thread's own maximum is a
// lower bound's witness: the k-th largest of the threads' maxima is a threshold that at least k
// values reach, and for k below the thread count few more do (for values in random order about
// NT ln(NT / (NT - k)) in all).  Those candidates go to LDS and are ranked by counting.  Rows
// that defeat the threshold (many equal values, or the top in few threads) take an exact
// bisection on the value, then on the token among the equal ones.  Bound by the one read of z.
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

// The packed row as new values, so that one pass's unpacked values are not kept for the next.
template <int NV>
__device__ inline void fresh(u32x4 (&reg)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) asm volatile("" : "+v"(reg[i]));
}

template <bool BF, int NT, int NV, bool RES>
__global__ __launch_bounds__(NT) void topk_kernel(TopkArgs a) {
  using Tile = RowTile<BF>;
  constexpr int VE = Tile::VE;
  constexpr int NW = NT / 64;
  __shared__ uint64_t cand[kCap];      // key, then the complement of the token: larger is better
  __shared__ uint32_t tmax[NT];
  __shared__ float red[NW];
  __shared__ uint32_t cnt[NW];
  __shared__ uint32_t ncand, tau_s;

  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Tile z(a.logits, row, a.ld, a.V);
  const int nvec = z.vectors();
  u32x4 reg[RES ? NV : 1];
  if (RES) {
#pragma unroll
    for (int i = 0; i < NV; ++i) reg[RES ? i : 0] = z.load(tid + i * NT);
  }
  // calls f(value, token) for each of this thread's values
  auto each = [&](auto f) {
    auto vec = [&](const u32x4& v, int j) {
      const int e0 = z.first(j);
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (e0 + e >= 0 && e0 + e < a.V) f(Tile::value(v, e), e0 + e);
    };
    if (RES) {
      fresh(reg);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (tid + i * NT < nvec) vec(reg[RES ? i : 0], tid + i * NT);
    } else {
      for (int j = tid; j < nvec; j += NT) vec(z.load(j), j);
    }
  };
  auto total = [&](uint32_t c) -> uint32_t {      // over the workgroup
#pragma unroll
    for (int o = 32; o >= 1; o /= 2) c += __shfl_xor(c, o, 64);
    __syncthreads();
    if (lane == 0) cnt[wave] = c;
    __syncthreads();
    uint32_t s = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) s += cnt[w];
    return s;
  };

  uint32_t best = 0u;
  each([&](float f, int) {
    const uint32_t k = key_of(f);
    best = k > best ? k : best;
  });
  tmax[tid] = best;
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
      red[0] = value_of(top);
    }
  }
  __syncthreads();
  const float m = red[0];
  uint32_t tau = tau_s;
  const float sT = kLog2e / a.T;
  // the sum, and the candidates
  float s = 0.f;
  each([&](float f, int e) {
    s += f == m ? 1.f : __builtin_amdgcn_exp2f((f - m) * sT);      // (equal infinities differ by nothing)
    const uint32_t k = key_of(f);
    if (k >= tau) {
      const uint32_t at = atomicAdd(&ncand, 1u);
      if (at < kCap) cand[at] = ((uint64_t)k << 32) | (uint32_t)~(uint32_t)e;
    }
  });
  s = wave_sum(s);
  __syncthreads();      // (red[0] has been read, the candidates are written)
  if (lane == 0) red[wave] = s;
  uint32_t nc = ncand;
  __syncthreads();
  if (tid == 0) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) t += red[w];
    a.lse[row] = m / a.T + logf(t);
  }
  if (nc > kCap) {
    // the k-th largest key exactly: tau = max {t : at least k keys >= t}
    tau = 0u;
    for (int b = 31; b >= 0; --b) {
      const uint32_t c = tau | (1u << b);
      uint32_t n = 0;
      each([&](float f, int) { n += key_of(f) >= c ? 1u : 0u; });
      if (total(n) >= (uint32_t)a.k) tau = c;
    }
    uint32_t above = 0;
    each([&](float f, int) { above += key_of(f) > tau ? 1u : 0u; });
    const uint32_t need = (uint32_t)a.k - total(above);      // of the equal ones: those with the lowest tokens
    int lim = 0;      // largest lim such that fewer than `need` equal ones stand below token lim
    for (int b = 30; b >= 0; --b) {
      const int64_t c = (int64_t)lim + (int64_t(1) << b);
      if (c >= a.V) continue;
      uint32_t n = 0;
      each([&](float f, int e) { n += (key_of(f) == tau && e < (int)c) ? 1u : 0u; });
      if (total(n) < need) lim = (int)c;
    }
    __syncthreads();
    if (tid == 0) ncand = 0u;
    __syncthreads();
    each([&](float f, int e) {
      const uint32_t k = key_of(f);
      if (k > tau || (k == tau && e <= lim)) {
        const uint32_t at = atomicAdd(&ncand, 1u);
        if (at < kCap) cand[at] = ((uint64_t)k << 32) | (uint32_t)~(uint32_t)e;
      }
    });
    __syncthreads();
    nc = ncand < (uint32_t)kCap ? ncand : (uint32_t)kCap;      // (exactly k)
  }
  // a candidate's place is the number of better ones (all are distinct: the tokens differ)
  for (uint32_t c = tid; c < nc; c += NT) {
    const uint64_t x = cand[c];
    int place = 0;
    for (uint32_t l = 0; l < nc; ++l) place += cand[l] > x ? 1 : 0;
    if (place < a.k) {
      a.ids[row * a.k + place] = (int32_t)~(uint32_t)x;
      a.vals[row * a.k + place] = value_of((uint32_t)(x >> 32));
    }
  }
}

template <bool BF>
hipError_t launch_type(const TopkArgs& a, hipStream_t s) {
  const int64_t nvec = ((int64_t)a.V + 7) / (BF ? 8 : 4) + 1;   // of a row that starts anywhere
  const dim3 grid((unsigned)a.N);
  if (nvec <= 512 * 4)
    hipLaunchKernelGGL((topk_kernel<BF, 512, 4, true>), grid, dim3(512), 0, s, a);
  else if (nvec <= 512 * 16)
    hipLaunchKernelGGL((topk_kernel<BF, 512, 16, true>), grid, dim3(512), 0, s, a);
  else if (nvec <= 1024 * 16)
    hipLaunchKernelGGL((topk_kernel<BF, 1024, 16, true>), grid, dim3(1024), 0, s, a);
  else
    hipLaunchKernelGGL((topk_kernel<BF, 1024, 1, false>), grid, dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_topk(const TopkArgs& a, hipStream_t s) {
  if (a.N == 0) return hipSuccess;
  return a.bf16 ? launch_type<true>(a, s) : launch_type<false>(a, s);
}

}  // namespace kron
