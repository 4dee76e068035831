// Orthogonalised update of matrices (the Muon optimiser's step).  For each rows x cols matrix:
//   m = mu m + g;  u = g + mu m (Nesterov) or m;  X = u / (|u|_F + eps), its smaller side first (s x l)
//   `steps` times  A = X X^T,  X = a X + (b A + c A^2) X  (a Newton-Schulz step on the quintic a v + b v^3 + c v^5
//   of the singular values)
//   W = keep W - lr scale X
// A matrix that fits a CU's LDS is one workgroup's from the gradient to the parameters (fp32 matrix
// instruction).  Others run as tiled products over all matrices of their size; X, A and the polynomial of A
// are fp16 planes (tile_product.h): two for fp32 parameters, one for bf16 ones.
#include <algorithm>
#include <utility>
#include <vector>

#include "row_tile.h"
#include "tile_product.h"

namespace kron {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

template <bool BF>
__device__ inline float get(const void* p, int64_t i) {
  return BF ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}
template <bool BF>
__device__ inline void put(void* p, int64_t i, float v) {
  if (BF) ((uint16_t*)p)[i] = (uint16_t)bf16_rne(v);
  else ((float*)p)[i] = v;
}

// ------------------------------------------------------------------------------ matrices within a workgroup
constexpr int kSmallThreads = 512, kSmallSide = 64, kSmallBatch = 40;
constexpr size_t kSmallLds = 156 * 1024;

struct SmallBatch {
  MuonTensor t[kSmallBatch];
  int first[kSmallBatch + 1];      // workgroups before each tensor's
  int n;
};

int pad16(int v) { return (v + 15) / 16 * 16; }
// Floats of LDS: X (rows of l rounded up to 16 and 4 more, so that 16 rows start in different banks), A and the polynomial, sums.
size_t small_lds(int s, int l) {
  const int sp = pad16(s), ld = pad16(l) + 4;
  return sizeof(float) * ((size_t)sp * ld + 2 * (size_t)sp * (sp + 4) + 8 * 256) + 64 * sizeof(double);
}
bool is_small(int rows, int cols) {
  const int s = std::min(rows, cols), l = std::max(rows, cols);
  return s <= kSmallSide && small_lds(s, l) <= kSmallLds;
}

__device__ inline f4 mma32(float a, float b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

template <bool BF>
__global__ __launch_bounds__(kSmallThreads) void muon_small_kernel(SmallBatch batch, MuonHyper h) {
  extern __shared__ char smem[];
  int ti = 0;
  while (ti + 1 < batch.n && (int)blockIdx.x >= batch.first[ti + 1]) ++ti;
  const MuonTensor T = batch.t[ti];
  const int64_t at = (int64_t)(blockIdx.x - batch.first[ti]) * T.rows * T.cols;
  const bool tall = T.rows > T.cols;
  const int s = tall ? T.cols : T.rows, l = tall ? T.rows : T.cols;
  const int sp = (s + 15) / 16 * 16, lp = (l + 15) / 16 * 16, ld = lp + 4, la = sp + 4;
  double* dred = (double*)smem;
  float* X = (float*)(dred + 64);
  float* A = X + (size_t)sp * ld;
  float* P = A + sp * la;
  float* red = P + sp * la;      // 8 x 256
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;
  constexpr int NW = kSmallThreads / 64;

  for (int i = tid; i < sp * ld; i += kSmallThreads) X[i] = 0.f;
  __syncthreads();
  double sum = 0;
  for (int i = tid; i < T.rows * T.cols; i += kSmallThreads) {
    const int r = i / T.cols, k = i - r * T.cols;
    const float gr = get<BF>(T.g, at + i);
    const float m = fmaf(h.mu, T.m[at + i], gr);
    T.m[at + i] = m;
    const float u = h.nesterov ? fmaf(h.mu, m, gr) : m;
    sum += (double)u * u;
    X[tall ? k * ld + r : r * ld + k] = u;
  }
  sum = wave_sum(sum);
  if (lane == 0) dred[wave] = sum;
  __syncthreads();
  sum = 0;
  for (int i = 0; i < NW; ++i) sum += dred[i];
  const float inv = (float)(1.0 / (sqrt(sum) + (double)h.eps));
  for (int i = tid; i < sp * ld; i += kSmallThreads) X[i] *= inv;
  __syncthreads();

  const int S = sp / 16, tiles = S * S;
  // wavefronts that share a tile's contraction when there are few tiles
  const int share = tiles == 1 ? NW : tiles == 4 ? NW / 4 : 1;
  for (int step = 0; step < h.steps; ++step) {
    for (int t = wave / share; t < tiles; t += NW / share) {
      const int i = t / S, j = t % S, part = wave % share;
      f4 acc = {0, 0, 0, 0};
      for (int k = part * 16; k < lp; k += share * 16) {
        const f4 x = *(const f4*)(X + (16 * i + c) * ld + k + 4 * g), y = *(const f4*)(X + (16 * j + c) * ld + k + 4 * g);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc = mma32(x[q], y[q], acc);
      }
      if (share == 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) A[(16 * i + 4 * g + e) * la + 16 * j + c] = acc[e];
      } else {
        *(f4*)(red + wave * 256 + lane * 4) = acc;
      }
    }
    __syncthreads();
    if (share > 1) {
      for (int q = tid; q < tiles * 256; q += kSmallThreads) {
        const int t = q >> 8, w = q & 255, i = t / S, j = t % S, ln = w >> 2;
        float v = 0.f;
        for (int p = 0; p < share; ++p) v += red[(t * share + p) * 256 + w];
        A[(16 * i + 4 * (ln >> 4) + (w & 3)) * la + 16 * j + (ln & 15)] = v;
      }
      __syncthreads();
    }
    // P = a I + b A + c A^2 (A is symmetric: its rows are its columns)
    for (int t = wave; t < tiles; t += NW) {
      const int i = t / S, j = t % S;
      f4 acc = {0, 0, 0, 0};
      for (int k = 0; k < sp; k += 16) {
        const f4 x = *(const f4*)(A + (16 * i + c) * la + k + 4 * g), y = *(const f4*)(A + (16 * j + c) * la + k + 4 * g);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc = mma32(x[q], y[q], acc);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 16 * i + 4 * g + e, k = 16 * j + c;
        P[r * la + k] = (r == k ? h.a : 0.f) + h.b * A[r * la + k] + h.c * acc[e];
      }
    }
    __syncthreads();
    // X = P X: a wavefront's 16 columns are its own
    for (int j = wave; j < lp / 16; j += NW) {
      f4 acc[kSmallSide / 16];
#pragma unroll
      for (int i = 0; i < kSmallSide / 16; ++i) acc[i] = f4{0, 0, 0, 0};
      for (int k = 0; k < sp; k += 16) {
        float y[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] = X[(k + 4 * g + q) * ld + 16 * j + c];
#pragma unroll
        for (int i = 0; i < kSmallSide / 16; ++i) {
          if (i >= S) break;
          const f4 x = *(const f4*)(P + (16 * i + c) * la + k + 4 * g);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i] = mma32(x[q], y[q], acc[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kSmallSide / 16; ++i) {
        if (i >= S) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) X[(16 * i + 4 * g + e) * ld + 16 * j + c] = acc[i][e];
      }
    }
    __syncthreads();
  }
  const float f = h.lr * T.scale;
  for (int i = tid; i < T.rows * T.cols; i += kSmallThreads) {
    const int r = i / T.cols, k = i - r * T.cols;
    const float o = X[tall ? k * ld + r : r * ld + k];
    put<BF>(T.p, at + i, fmaf(-f, o, get<BF>(T.p, at + i) * h.keep));
  }
}

// ------------------------------------------------------------------------------ large matrices
constexpr int kGroup = 40;           // tensors of one size in a launch
constexpr int kNormParts = 64;       // workgroups of a matrix's norm
// Scales of the planes: |X| <= 1.3, |A| <= 1.7 and |P| <= 3.5 stay below fp16's 65504, and small entries keep their bits
constexpr float kX = 8192.f, kA = 8192.f, kP = 8192.f;

struct MuonGroup {
  MuonTensor t[kGroup];
  int first[kGroup + 1];      // matrices before each tensor's
  int n;
  int s, l, sp, lp;           // sides, and rounded up to kBK
  double* norm;               // matrices x kNormParts
  uint16_t* X[2];             // matrices x planes x s x lp
  uint16_t* A;                // matrices x planes x s x sp
  uint16_t* P;
};

__device__ inline const MuonTensor& tensor_of(const MuonGroup& G, int mat, int64_t& at) {
  int ti = 0;
  while (ti + 1 < G.n && mat >= G.first[ti + 1]) ++ti;
  at = (int64_t)(mat - G.first[ti]) * G.s * G.l;
  return G.t[ti];
}

// m = mu m + g, and the sums of u^2.
template <bool BF>
__global__ __launch_bounds__(256) void muon_momentum_kernel(MuonGroup G, MuonHyper h) {
  __shared__ double red[4];
  int64_t at;
  const MuonTensor& T = tensor_of(G, blockIdx.y, at);
  const int64_t n = (int64_t)G.s * G.l;
  double sum = 0;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)kNormParts * 256) {
    const float gr = get<BF>(T.g, at + i);
    const float m = fmaf(h.mu, T.m[at + i], gr);
    T.m[at + i] = m;
    const float u = h.nesterov ? fmaf(h.mu, m, gr) : m;
    sum += (double)u * u;
  }
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) G.norm[(int64_t)blockIdx.y * kNormParts + blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

template <int NP>
__device__ inline void put_planes(uint16_t* p, int64_t plane, float v) {
  const _Float16 hi = (_Float16)v;
  *(_Float16*)p = hi;
  if constexpr (NP == 2) *(_Float16*)(p + plane) = (_Float16)((v - (float)hi) * kLo);
}
template <int NP>
__device__ inline void put_planes4(uint16_t* p, int64_t plane, f4 v) {
  typedef _Float16 h4 __attribute__((ext_vector_type(4)));
  h4 hi, lo;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    hi[e] = (_Float16)v[e];
    lo[e] = (_Float16)((v[e] - (float)hi[e]) * kLo);
  }
  *(h4*)p = hi;
  if constexpr (NP == 2) *(h4*)(p + plane) = lo;
}
template <int NP>
__device__ inline f4 get_planes4(const uint16_t* p, int64_t plane) {
  typedef _Float16 h4 __attribute__((ext_vector_type(4)));
  const h4 hi = *(const h4*)p;
  f4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = (float)hi[e];
  if constexpr (NP == 2) {
    const h4 lo = *(const h4*)(p + plane);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += (float)lo[e] * kLoInv;
  }
  return v;
}

// X's planes: 64 x 64 of a matrix, turned where it is tall.
template <bool BF, int NP>
__global__ __launch_bounds__(256) void muon_start_kernel(MuonGroup G, MuonHyper h, int tiles_l) {
  __shared__ float tile[64][65];
  const int tid = threadIdx.x;
  int64_t at;
  const MuonTensor& T = tensor_of(G, blockIdx.y, at);
  double sum = 0;
  for (int i = 0; i < kNormParts; ++i) sum += G.norm[(int64_t)blockIdx.y * kNormParts + i];
  const float inv = (float)((double)kX / (sqrt(sum) + (double)h.eps));
  const bool tall = T.rows > T.cols;
  const int s0 = (blockIdx.x / tiles_l) * 64, l0 = (blockIdx.x % tiles_l) * 64;
  const int r0 = tall ? l0 : s0, c0 = tall ? s0 : l0;
  for (int i = tid; i < 64 * 64; i += 256) {
    const int r = i >> 6, k = i & 63;
    float u = 0.f;
    if (r0 + r < T.rows && c0 + k < T.cols) {
      const int64_t e = at + (int64_t)(r0 + r) * T.cols + c0 + k;
      const float m = T.m[e];
      u = h.nesterov ? fmaf(h.mu, m, get<BF>(T.g, e)) : m;
    }
    tile[r][k] = u * inv;
  }
  __syncthreads();
  const int64_t plane = (int64_t)G.s * G.lp;
  uint16_t* X = G.X[0] + (int64_t)blockIdx.y * NP * plane;
  for (int i = tid; i < 64 * 64; i += 256) {
    const int r = i >> 6, k = i & 63;      // k beyond l: zeros up to lp
    if (s0 + r < G.s) put_planes<NP>(X + (int64_t)(s0 + r) * G.lp + l0 + k, plane, tall ? tile[k][r] : tile[r][k]);
  }
}

// MODE 0: A = X X^T.  1: P = a I + b A + c A A.  2: X' = P X.  3: the same, into the parameters.
template <class Pr, bool BF, int NP, int MODE>
__global__ __launch_bounds__(Pr::kThreads) void muon_product_kernel(MuonGroup G, MuonHyper h, int from, int tm, int tn) {
  extern __shared__ char smem[];
  int mt, nt;
  tile_of(blockIdx.x, gridDim.x, tm, tn, mt, nt);
  const int mat = blockIdx.y, m0 = mt * Pr::BM, n0 = nt * Pr::BN;
  const int64_t xplane = (int64_t)G.s * G.lp, aplane = (int64_t)G.s * G.sp;
  const Operand X = {G.X[from] + (int64_t)mat * NP * xplane, G.lp, xplane, G.s, G.lp};
  const Operand A = {G.A + (int64_t)mat * NP * aplane, G.sp, aplane, G.s, G.sp};
  const Operand Q = {G.P + (int64_t)mat * NP * aplane, G.sp, aplane, G.s, G.sp};
  Pr p;
  p.run(MODE == 1 ? A : X, MODE == 0 ? X : MODE == 1 ? A : Q, m0, n0, 0, MODE == 0 ? G.lp : G.sp, (lds_t*)smem);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
#pragma unroll
  for (int j = 0; j < Pr::TN; ++j) {
    const int n = n0 + (wave / Pr::WM) * Pr::TN * 16 + 16 * j + c;
    if (n >= G.s) continue;
#pragma unroll
    for (int i = 0; i < Pr::TM; ++i) {
      const int m = m0 + (wave % Pr::WM) * Pr::TM * 16 + 16 * i + 4 * g;
      f4 v = p.acc[i][j];
      if constexpr (MODE <= 1) {
        if (m >= G.sp) continue;
        const int64_t o = (int64_t)n * G.sp + m;
        if constexpr (MODE == 0) {
          v = v * (kA / (kX * kX));
        } else {
          v = v * (h.c * kP / (kA * kA)) + get_planes4<NP>(A.p + o, aplane) * (h.b * kP / kA);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (m + e == n) v[e] += h.a * kP;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (m + e >= G.s) v[e] = 0.f;      // (what pads the rows, whatever the operands' rows beyond gave)
        put_planes4<NP>((MODE == 0 ? G.A : G.P) + (int64_t)mat * NP * aplane + o, aplane, v);
      } else if constexpr (MODE == 2) {
        if (m >= G.lp) continue;
        put_planes4<NP>(G.X[from ^ 1] + (int64_t)mat * NP * xplane + (int64_t)n * G.lp + m, xplane, v * (1.f / kP));
      } else {
        int64_t at;
        const MuonTensor& T = tensor_of(G, mat, at);
        const float f = h.lr * T.scale;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (m + e < G.l) {
            const int64_t o = at + (T.rows > T.cols ? (int64_t)(m + e) * T.cols + n : (int64_t)n * T.cols + m + e);
            put<BF>(T.p, o, fmaf(-f, v[e] * (1.f / (kP * kX)), get<BF>(T.p, o) * h.keep));
          }
      }
    }
  }
}

template <class Pr, auto kernel>
hipError_t go(dim3 grid, hipStream_t s, const MuonGroup& G, const MuonHyper& h, int from, int tm, int tn) {
  const hipError_t e = allow_lds<kernel>();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, grid, dim3(Pr::kThreads), Pr::kLdsBytes, s, G, h, from, tm, tn);
  return hipGetLastError();
}

// The largest tiles that still give every CU one.
template <bool BF, int NP, int MODE>
hipError_t product(const MuonGroup& G, const MuonHyper& h, int from, int mats, hipStream_t s) {
  constexpr Side SA = MODE >= 2 ? COL : ROW;
  const int M = MODE >= 2 ? G.lp : G.sp, N = G.s;
  auto tiles = [&](int b) { return ceil_div(M, b) * ceil_div(N, b) * mats; };
#define KRON_MUON_GO(B, ...)                                                                                        \
  {                                                                                                                 \
    typedef Product<__VA_ARGS__, SA, ROW, false, NP> Pr;                                                            \
    const int tm = (int)ceil_div(M, B), tn = (int)ceil_div(N, B);                                                   \
    return go<Pr, muon_product_kernel<Pr, BF, NP, MODE>>(dim3((unsigned)(tm * tn), (unsigned)mats), s, G, h, from, tm, tn); \
  }
  if (tiles(256) >= 256) KRON_MUON_GO(256, 2, 4, 8, 4)
  if (tiles(128) >= 256) KRON_MUON_GO(128, 2, 2, 4, 4)
  KRON_MUON_GO(64, 2, 2, 2, 2)
#undef KRON_MUON_GO
}

template <bool BF>
hipError_t run_group(const MuonGroup& G, const MuonHyper& h, int mats, hipStream_t s) {
  constexpr int NP = BF ? 1 : 2;
  hipLaunchKernelGGL((muon_momentum_kernel<BF>), dim3(kNormParts, (unsigned)mats), dim3(256), 0, s, G, h);
  const int tl = G.lp / 64, ts = (int)ceil_div(G.s, 64);
  hipLaunchKernelGGL((muon_start_kernel<BF, NP>), dim3((unsigned)(tl * ts), (unsigned)mats), dim3(256), 0, s, G, h, tl);
  hipError_t e = hipGetLastError();
  for (int i = 0; i < h.steps && e == hipSuccess; ++i) {
    e = product<BF, NP, 0>(G, h, i & 1, mats, s);
    if (e == hipSuccess) e = product<BF, NP, 1>(G, h, i & 1, mats, s);
    if (e == hipSuccess) e = i + 1 < h.steps ? product<BF, NP, 2>(G, h, i & 1, mats, s) : product<BF, NP, 3>(G, h, i & 1, mats, s);
  }
  return e;
}

// What a group of `mats` matrices takes of the workspace.
size_t group_bytes(int s, int l, int64_t mats, bool bf, MuonGroup* G, char* ws) {
  const int planes = bf ? 1 : 2;
  const int sp = (int)ceil_div(s, kBK) * kBK, lp = (int)ceil_div(l, kBK) * kBK;
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t r = at; at += up256(bytes); return r; };
  const size_t norm = take(sizeof(double) * kNormParts * mats);
  const size_t x0 = take(2 * (size_t)planes * s * lp * mats), x1 = take(2 * (size_t)planes * s * lp * mats);
  const size_t a = take(2 * (size_t)planes * s * sp * mats), p = take(2 * (size_t)planes * s * sp * mats);
  if (G) {
    G->s = s, G->l = l, G->sp = sp, G->lp = lp;
    G->norm = (double*)(ws + norm);
    G->X[0] = (uint16_t*)(ws + x0), G->X[1] = (uint16_t*)(ws + x1);
    G->A = (uint16_t*)(ws + a), G->P = (uint16_t*)(ws + p);
  }
  return at;
}

// Calls f(s, l, tensors, n, matrices) for the groups of large matrices: tensors of one size, at most kGroup tensors
// and kGroupMats matrices together.  They run one after the other in the same workspace.
constexpr int kGroupMats = 64;
template <class F>
hipError_t for_groups(const MuonTensor* t, int n, const F& f) {
  std::vector<int> order;
  for (int i = 0; i < n; ++i)
    if (t[i].count > 0 && !is_small(t[i].rows, t[i].cols)) order.push_back(i);
  auto size = [&](int i) { return std::make_pair(std::min(t[i].rows, t[i].cols), std::max(t[i].rows, t[i].cols)); };
  std::stable_sort(order.begin(), order.end(), [&](int i, int j) { return size(i) < size(j); });
  MuonTensor got[kGroup];
  int k = 0;
  int64_t mats = 0;
  for (size_t o = 0; o < order.size(); ++o) {
    MuonTensor rest = t[order[o]];
    const auto sl = size(order[o]);
    const bool last = o + 1 == order.size() || size(order[o + 1]) != sl;
    while (rest.count > 0) {
      MuonTensor now = rest;
      now.count = std::min<int64_t>(rest.count, kGroupMats - mats);
      got[k++] = now;
      mats += now.count;
      const int64_t skip = now.count * rest.rows * rest.cols;
      rest.count -= now.count;
      rest.m += skip;
      rest.p = (char*)rest.p + skip * f.element();
      rest.g = (const char*)rest.g + skip * f.element();
      if (k == kGroup || mats == kGroupMats || (last && rest.count == 0)) {
        const hipError_t e = f(sl.first, sl.second, got, k, mats);
        if (e != hipSuccess) return e;
        k = 0, mats = 0;
      }
    }
  }
  return hipSuccess;
}

struct CountBytes {
  bool bf16;
  int element() const { return bf16 ? 2 : 4; }
  size_t* most;
  hipError_t operator()(int s, int l, const MuonTensor*, int, int64_t mats) const {
    *most = std::max(*most, group_bytes(s, l, mats, bf16, nullptr, nullptr));
    return hipSuccess;
  }
};

struct RunGroup {
  bool bf16;
  int element() const { return bf16 ? 2 : 4; }
  const MuonHyper* h;
  char* ws;
  hipStream_t stream;
  hipError_t operator()(int s, int l, const MuonTensor* t, int n, int64_t mats) const {
    MuonGroup G{};
    group_bytes(s, l, mats, bf16, &G, ws);
    G.n = n;
    for (int i = 0; i < n; ++i) {
      G.t[i] = t[i];
      G.first[i + 1] = G.first[i] + (int)t[i].count;
    }
    return bf16 ? run_group<true>(G, *h, (int)mats, stream) : run_group<false>(G, *h, (int)mats, stream);
  }
};

template <bool BF>
hipError_t run_small(const SmallBatch& b, int lds, const MuonHyper& h, hipStream_t s) {
  const hipError_t e = allow_lds<muon_small_kernel<BF>>();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((muon_small_kernel<BF>), dim3((unsigned)b.first[b.n]), dim3(kSmallThreads), lds, s, b, h);
  return hipGetLastError();
}

}  // namespace

size_t muon_workspace(const MuonTensor* t, int n, bool bf16) {
  size_t most = 0;
  (void)for_groups(t, n, CountBytes{bf16, &most});
  return most;
}

hipError_t launch_muon(const MuonTensor* t, int n, const MuonHyper& h, void* ws, hipStream_t s) {
  SmallBatch b{};
  size_t lds = 0;
  auto flush = [&]() {
    hipError_t e = hipSuccess;
    if (b.n) e = h.bf16 ? run_small<true>(b, (int)lds, h, s) : run_small<false>(b, (int)lds, h, s);
    b.n = 0, lds = 0;
    return e;
  };
  for (int i = 0; i < n; ++i) {
    if (t[i].count == 0 || !is_small(t[i].rows, t[i].cols)) continue;
    if (b.n == kSmallBatch || b.first[b.n] + t[i].count > (1 << 20)) {
      const hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    b.t[b.n] = t[i];
    b.first[b.n + 1] = b.first[b.n] + (int)t[i].count;
    ++b.n;
    lds = std::max(lds, small_lds(std::min(t[i].rows, t[i].cols), std::max(t[i].rows, t[i].cols)));
  }
  const hipError_t e = flush();
  if (e != hipSuccess) return e;
  return for_groups(t, n, RunGroup{h.bf16 != 0, &h, (char*)ws, s});
}

}  // namespace kron
