// Orthogonalised update of matrices (the Muon optimiser's step).  For each rows x cols matrix:
//   m = mu m + g;  u = g + mu m (Nesterov) or m;  X = u / (|u|_F + eps), its smaller side first (s x l)
//   `steps` times  A = X X^T,  X = a X + (b A + c A^2) X  (a Newton-Schulz step on the quintic a v + b v^3 + c v^5
//   of the singular values)
//   W = keep W - lr scale X
// A matrix that fits a CU's LDS is one workgroup's from the gradient to the parameters (fp32 matrix
// instruction).  Others run as tiled products over all matrices of their size; X, A and the polynomial of A
// are fp16 parts (tile_product.h): two for fp32 parameters, one for bf16 ones.
//
// What bounds it: chains.  192 matrices of 32 x 64 and 24 x 32 take 16 us, five steps of 1.8 to 2.2 us and the gradients' way in;
// 1024 x 1024 fp32 fifteen dependent products of 11.6 to 15.5 us (6.4 GFLOP of parts each for P X: 410 TFLOP/s), their tiles'
// loads out of L2 at 6 TB/s.
#include <algorithm>
#include <cmath>
#include <type_traits>
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
// N neighbouring values, i a multiple of N.
template <bool BF, int N>
__device__ inline void get_n(const void* p, int64_t i, float (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = get<BF>(p, i);
  } else if constexpr (BF) {
    const uint2 w = *(const uint2*)((const uint16_t*)p + i);
    v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
  } else {
    const f4 w = *(const f4*)((const float*)p + i);
    v[0] = w[0], v[1] = w[1], v[2] = w[2], v[3] = w[3];
  }
}
template <bool BF, int N>
__device__ inline void put_n(void* p, int64_t i, const float (&v)[N]) {
  if constexpr (N == 1) {
    if (BF) ((uint16_t*)p)[i] = (uint16_t)bf16_rne(v[0]);
    else ((float*)p)[i] = v[0];
  } else if constexpr (BF) {
    *(uint2*)((uint16_t*)p + i) = uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
  } else {
    *(f4*)((float*)p + i) = f4{v[0], v[1], v[2], v[3]};
  }
}
// u of N neighbours from the gradient and the momentum before.
template <int N>
__device__ inline void momentum(const MuonHyper& h, const float (&g)[N], float (&m)[N], float (&u)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    m[e] = fmaf(h.mu, m[e], g[e]);
    u[e] = h.nesterov ? fmaf(h.mu, m[e], g[e]) : m[e];
  }
}
// Whether fp32 holds a factor with all its bits: with the smallest eps, zeros' is infinite there, and that of gradients next
// to either end of the range is infinite or has few bits.  64 bits do then.
__device__ inline bool in_range(float v) { return v >= 0x1p-126f && v < INFINITY; }
template <bool BF>
__device__ inline void put(void* p, int64_t i, float v) {
  if (BF) ((uint16_t*)p)[i] = (uint16_t)bf16_rne(v);
  else ((float*)p)[i] = v;
}

// ------------------------------------------------------------------------------ matrices within a workgroup
constexpr int kSmallSide = 64, kSmallBatch = 40, kBatch = 4;
constexpr size_t kSmallLds = 156 * 1024;

struct SmallBatch {
  MuonTensor t[kSmallBatch];
  int first[kSmallBatch + 1];      // workgroups before each tensor's
  int n;
};

int pad16(int v) { return (v + 15) / 16 * 16; }
// LDS: X (rows of l rounded up to 16 and 4 more, so that 16 rows start in different banks), A and the polynomial, sums.
size_t small_lds(int s, int l) {
  const int sp = pad16(s), ld = pad16(l) + 4;
  return sizeof(float) * ((size_t)sp * ld + 2 * (size_t)sp * (sp + 4) + 16 * 256) + 64 * sizeof(double);
}
bool is_small(int rows, int cols) {
  const int s = std::min(rows, cols), l = std::max(rows, cols);
  return s <= kSmallSide && small_lds(s, l) <= kSmallLds;
}

__device__ inline f4 mma32(float a, float b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// c += a b^T over 16 of the contraction, two chains of sums.
__device__ inline void dot16(f4 a, f4 b, f4& c0, f4& c1) {
  c0 = mma32(a[0], b[0], c0);
  c1 = mma32(a[1], b[1], c1);
  c0 = mma32(a[2], b[2], c0);
  c1 = mma32(a[3], b[3], c1);
}

// The steps on X (16 S rows of ld = lp + 4) in LDS, by NW wavefronts; X times `inv` is the first one's.  What bounds them
// is the chain of LDS reads, products and barriers of one CU: chains are split in two, contractions among the wavefronts,
// and four of X's column blocks go together (2048 x 16: 8.3 -> 5.8 us a step, 64 x 64 5.5 -> 3.5, 32 x 64 2.2 -> 1.8).
template <int S, int NW>
__device__ __forceinline__ void small_steps(float* X, float* A, float* P, float* red, int lp, float inv, const MuonHyper& h) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;
  const int ld = lp + 4;
  constexpr int la = 16 * S + 4, T = S * (S + 1) / 2;      // tiles on and below the diagonal
  constexpr int share = NW / T > 0 ? NW / T : 1;           // wavefronts of a tile
  auto tile = [](int t, int& i, int& j) {
    i = t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0;
    j = t - i * (i + 1) / 2;
  };
  auto put = [&](float* M, int i, int j, f4 v) {      // and its mirror image
#pragma unroll
    for (int e = 0; e < 4; ++e) M[(16 * i + 4 * g + e) * la + 16 * j + c] = v[e];
    if (i != j) *(f4*)(M + (16 * j + c) * la + 16 * i + 4 * g) = v;
  };
  for (int step = 0; step < h.steps; ++step) {
    const float first = step == 0 ? inv : 1.f;
    for (int t = wave / share; t < T; t += NW / share) {
      int i, j;
      tile(t, i, j);
      f4 c0 = {0, 0, 0, 0}, c1 = {0, 0, 0, 0};
      for (int k = wave % share * 16; k < lp; k += share * 16)
        dot16(*(const f4*)(X + (16 * i + c) * ld + k + 4 * g) * first, *(const f4*)(X + (16 * j + c) * ld + k + 4 * g) * first, c0, c1);
      if (share == 1) put(A, i, j, c0 + c1);
      else *(f4*)(red + wave * 256 + lane * 4) = c0 + c1;
    }
    __syncthreads();
    if (share > 1) {
      if (wave < T) {
        int i, j;
        tile(wave, i, j);
        f4 v = {0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < share; ++p) v += *(const f4*)(red + (wave * share + p) * 256 + lane * 4);
        put(A, i, j, v);
      }
      __syncthreads();
    }
    // P = a I + b A + c A^2 (A is symmetric: its rows are its columns)
    for (int t = wave; t < T; t += NW) {
      int i, j;
      tile(t, i, j);
      f4 c0 = {0, 0, 0, 0}, c1 = {0, 0, 0, 0}, v;
#pragma unroll
      for (int k = 0; k < 16 * S; k += 16)
        dot16(*(const f4*)(A + (16 * i + c) * la + k + 4 * g), *(const f4*)(A + (16 * j + c) * la + k + 4 * g), c0, c1);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 16 * i + 4 * g + e, k = 16 * j + c;
        v[e] = (r == k ? h.a : 0.f) + h.b * A[r * la + k] + h.c * (c0[e] + c1[e]);
      }
      put(P, i, j, v);
    }
    __syncthreads();
    // X = P X: a wavefront's columns are its own
    constexpr int JB = S == 1 ? 4 : S == 2 ? 2 : 1;
    const int blocks = lp / 16;
    for (int j0 = wave; j0 < blocks; j0 += JB * NW) {
      f4 acc[JB][S];
#pragma unroll
      for (int b = 0; b < JB; ++b)
#pragma unroll
        for (int i = 0; i < S; ++i) acc[b][i] = f4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < 16 * S; k += 16) {
        f4 y[JB], x[S];
#pragma unroll
        for (int b = 0; b < JB; ++b)
#pragma unroll
          for (int q = 0; q < 4; ++q) y[b][q] = X[(k + 4 * g + q) * ld + 16 * min(j0 + b * NW, blocks - 1) + c] * first;
#pragma unroll
        for (int i = 0; i < S; ++i) x[i] = *(const f4*)(P + (16 * i + c) * la + k + 4 * g);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int b = 0; b < JB; ++b)
#pragma unroll
            for (int i = 0; i < S; ++i) acc[b][i] = mma32(x[i][q], y[b][q], acc[b][i]);
      }
#pragma unroll
      for (int b = 0; b < JB; ++b)
        if (j0 + b * NW < blocks)
#pragma unroll
          for (int i = 0; i < S; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) X[(16 * i + 4 * g + e) * ld + 16 * (j0 + b * NW) + c] = acc[b][i][e];
    }
    __syncthreads();
  }
}

template <bool BF, int NT>
__global__ __launch_bounds__(NT) void muon_small_kernel(SmallBatch batch, MuonHyper h) {
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
  float* red = P + sp * la;      // wavefronts x 256
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int NW = NT / 64;

  // what pads X's rows and columns
  for (int i = s * ld + tid; i < sp * ld; i += NT) X[i] = 0.f;
  for (int i = tid; i < s * (lp - l); i += NT) X[i / (lp - l) * ld + l + i % (lp - l)] = 0.f;
  double sum = 0;
  // kBatch groups of neighbours are in flight together (one after the other, 2048 x 16 took 45 us to come in)
  auto start = [&](auto n) {
    constexpr int N = decltype(n)::value;
    const int per = T.cols / N, all = T.rows * per;
    for (int i0 = tid; i0 < all; i0 += kBatch * NT) {
      float g[kBatch][N], m[kBatch][N], u[N];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int64_t e = at + (int64_t)min(i0 + q * NT, all - 1) * N;
        get_n<BF, N>(T.g, e, g[q]);
        get_n<false, N>(T.m, e, m[q]);
      }
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int i = i0 + q * NT;
        if (i >= all) break;
        momentum<N>(h, g[q], m[q], u);
        put_n<false, N>(T.m, at + (int64_t)i * N, m[q]);
        const int r = i / per, k = (i - r * per) * N;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          sum += (double)u[e] * u[e];
          X[tall ? (k + e) * ld + r : r * ld + k + e] = u[e];
        }
      }
    }
  };
  if (T.cols % 4 == 0) start(std::integral_constant<int, 4>{});
  else start(std::integral_constant<int, 1>{});
  sum = wave_sum(sum);
  if (lane == 0) dred[wave] = sum;
  __syncthreads();
  sum = 0;
  for (int i = 0; i < NW; ++i) sum += dred[i];
  const double inverse = 1.0 / (sqrt(sum) + (double)h.eps);
  float inv = (float)inverse;
  if (!in_range(inv)) {
    for (int i = tid; i < s * ld; i += NT) X[i] = (float)(X[i] * inverse);
    inv = 1.f;
    __syncthreads();
  }
  switch (sp / 16) {
    case 1: small_steps<1, NW>(X, A, P, red, lp, inv, h); break;
    case 2: small_steps<2, NW>(X, A, P, red, lp, inv, h); break;
    case 3: small_steps<3, NW>(X, A, P, red, lp, inv, h); break;
    default: small_steps<4, NW>(X, A, P, red, lp, inv, h); break;
  }
  const float f = h.lr * T.scale;
  auto finish = [&](auto n) {
    constexpr int N = decltype(n)::value;
    const int per = T.cols / N, all = T.rows * per;
    for (int i0 = tid; i0 < all; i0 += kBatch * NT) {
      float w[kBatch][N];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) get_n<BF, N>(T.p, at + (int64_t)min(i0 + q * NT, all - 1) * N, w[q]);
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int i = i0 + q * NT;
        if (i >= all) break;
        const int r = i / per, k = (i - r * per) * N;
#pragma unroll
        for (int e = 0; e < N; ++e) w[q][e] = fmaf(-f, X[tall ? (k + e) * ld + r : r * ld + k + e], w[q][e] * h.keep);
        put_n<BF, N>(T.p, at + (int64_t)i * N, w[q]);
      }
    }
  };
  if (T.cols % 4 == 0) finish(std::integral_constant<int, 4>{});
  else finish(std::integral_constant<int, 1>{});
}

// ------------------------------------------------------------------------------ large matrices
constexpr int kGroup = 40;           // tensors of one size in a launch
constexpr int kNormParts = 256;      // workgroups of a matrix's norm
// Scales of the parts, powers of two: what a step's X, A and P can be (muon_scales) stays below fp16's 65504, and small
// entries keep their bits.  Of the default quintic |X| <= 1.3, |A| <= 1.6 and |P| <= 3.5: all three are kScale.
constexpr float kScale = 8192.f;

struct MuonGroup {
  MuonTensor t[kGroup];
  int first[kGroup + 1];      // matrices before each tensor's
  int n;
  int s, l, sp, lp;           // sides, and rounded up to kBK
  double* norm;               // matrices x kNormParts
  uint16_t* X[2];             // matrices x s x lp, NP parts
  uint16_t* A;                // matrices x s x sp, NP parts
  uint16_t* P;
};

__device__ inline const MuonTensor& tensor_of(const MuonGroup& G, int mat, int64_t& at) {
  int ti = 0;
  while (ti + 1 < G.n && mat >= G.first[ti + 1]) ++ti;
  at = (int64_t)(mat - G.first[ti]) * G.s * G.l;
  return G.t[ti];
}

// m = mu m + g, and the sums of u^2.
template <bool BF, int N>
__global__ __launch_bounds__(256) void muon_momentum_kernel(MuonGroup G, MuonHyper h) {
  __shared__ double red[4];
  int64_t at;
  const MuonTensor& T = tensor_of(G, blockIdx.y, at);
  const int64_t n = (int64_t)G.s * G.l / N;
  double sum = 0;
#pragma unroll 2
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)kNormParts * 256) {
    float g[N], m[N], u[N];
    get_n<BF, N>(T.g, at + i * N, g);
    get_n<false, N>(T.m, at + i * N, m);
    momentum<N>(h, g, m, u);
    put_n<false, N>(T.m, at + i * N, m);
#pragma unroll
    for (int e = 0; e < N; ++e) sum += (double)u[e] * u[e];
  }
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) G.norm[(int64_t)blockIdx.y * kNormParts + blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

// Four neighbours, from column k (a multiple of four) of a row on, as NP parts.
template <int NP>
__device__ inline void put_parts(uint16_t* row, int k, f4 v) {
  uint16_t* p = NP == 2 ? row + (k / 32) * 64 + k % 32 : row + k;
  *(h4*)p = first_part(v);
  if constexpr (NP == 2) *(h4*)(p + 32) = first_part(v);
}
// The same of four rows, `ld` apart, at column k; `rows` of them are written.
template <int NP>
__device__ inline void put_parts_turned(uint16_t* first, int64_t ld, int rows, int k, f4 v) {
  uint16_t* p = NP == 2 ? first + (k / 32) * 64 + k % 32 : first + k;
#pragma unroll
  for (int q = 0; q < NP; ++q) {
    const h4 h = first_part(v);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < rows) *(_Float16*)(p + e * ld + 32 * q) = h[e];
  }
}
template <int NP>
__device__ inline f4 get_parts(const uint16_t* row, int k) {
  const uint16_t* p = NP == 2 ? row + (k / 32) * 64 + k % 32 : row + k;
  const h4 hi = *(const h4*)p;
  f4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = (float)hi[e];
  if constexpr (NP == 2) {
    const h4 lo = *(const h4*)(p + 32);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += (float)lo[e];
  }
  return v;
}
// X's parts: 64 x 64 of a matrix, turned where it is tall.
template <bool BF, int NP>
__global__ __launch_bounds__(256) void muon_start_kernel(MuonGroup G, MuonHyper h, int tiles_l) {
  __shared__ float tile[64][65];
  const int tid = threadIdx.x;
  int64_t at;
  const MuonTensor& T = tensor_of(G, blockIdx.y, at);
  __shared__ double red[4];
  const bool tall = T.rows > T.cols;
  const int s0 = (blockIdx.x / tiles_l) * 64, l0 = (blockIdx.x % tiles_l) * 64;
  const int r0 = tall ? l0 : s0, c0 = tall ? s0 : l0;
  // the tile and the norm's parts are asked for together (a branch around each load: 10 us of this kernel at any size)
  float u[16], g[16];
  const int64_t first = at + min(c0 + (tid & 63), T.cols - 1);
  auto row = [&](int q) { return first + (int64_t)min(r0 + q * 4 + (tid >> 6), T.rows - 1) * T.cols; };
#pragma unroll
  for (int q = 0; q < 16; ++q) u[q] = T.m[row(q)];
#pragma unroll
  for (int q = 0; q < 16; ++q) g[q] = h.nesterov ? get<BF>(T.g, row(q)) : 0.f;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    if (h.nesterov) u[q] = fmaf(h.mu, u[q], g[q]);
    if (r0 + q * 4 + (tid >> 6) >= T.rows || c0 + (tid & 63) >= T.cols) u[q] = 0.f;
  }
  double sum = wave_sum(G.norm[(int64_t)blockIdx.y * kNormParts + tid]);
  if ((tid & 63) == 0) red[tid >> 6] = sum;
  __syncthreads();
  sum = red[0] + red[1] + red[2] + red[3];
  const double inverse = (double)kScale / (sqrt(sum) + (double)h.eps);
  const float inv = (float)inverse;
  const bool whole = in_range(inv);
#pragma unroll
  for (int q = 0; q < 16; ++q) tile[q * 4 + (tid >> 6)][tid & 63] = whole ? u[q] * inv : (float)(u[q] * inverse);
  __syncthreads();
  uint16_t* X = G.X[0] + (int64_t)blockIdx.y * NP * G.s * G.lp;
#pragma unroll
  for (int i = tid; i < 64 * 16; i += 256) {
    const int r = i >> 4, k = (i & 15) * 4;      // k beyond l: zeros up to lp
    if (s0 + r < G.s)
      put_parts<NP>(X + (int64_t)(s0 + r) * G.lp * NP, l0 + k,
                    tall ? f4{tile[k][r], tile[k + 1][r], tile[k + 2][r], tile[k + 3][r]} : f4{tile[r][k], tile[r][k + 1], tile[r][k + 2], tile[r][k + 3]});
  }
}

// MODE 0: A = X X^T.  1: P = a I + b A + c A A.  2: X' = P X.  3: the same, into the parameters of the wide
// matrices; 4: into the tall ones' (turned: lanes hold neighbours of a row of the parameters in both).
// A and P are symmetric: their tiles on and below the diagonal are computed (tm: tiles of a side) and written twice.
template <class Pr, bool BF, int NP, int MODE>
__device__ __forceinline__ void muon_tile(const MuonGroup& G, const MuonHyper& h, const MuonScales& k, const MuonTensor& T, int64_t at, int from,
                                          int tm, int tn, char* smem) {
  int mt, nt;
  if constexpr (MODE <= 1) {
    static_assert(Pr::BM == Pr::BN, "");
    mt = (int)((sqrtf(8.f * (float)blockIdx.x + 1.f) - 1.f) * 0.5f);
    while (mt * (mt + 1) / 2 > (int)blockIdx.x) --mt;
    while ((mt + 1) * (mt + 2) / 2 <= (int)blockIdx.x) ++mt;
    nt = blockIdx.x - mt * (mt + 1) / 2;
  } else {
    tile_of(blockIdx.x, gridDim.x, tm, tn, mt, nt);
  }
  const int mat = blockIdx.y, m0 = mt * Pr::BM, n0 = nt * Pr::BN;
  const int64_t lx = (int64_t)G.lp * NP, la = (int64_t)G.sp * NP;      // rows of X, of A and P
  uint16_t* Am = G.A + (int64_t)mat * G.s * la;
  uint16_t* Pm = G.P + (int64_t)mat * G.s * la;
  const Operand X = {G.X[from] + (int64_t)mat * G.s * lx, lx, G.s, G.lp};
  const Operand A = {Am, la, G.s, G.sp}, Q = {Pm, la, G.s, G.sp};
  // what the end needs is asked for before the product
  constexpr bool early = Pr::TM * Pr::TN <= 4;
  f4 old[early ? Pr::TN : 1][early ? Pr::TM : 1];
  auto end = [&](auto f) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < Pr::TN; ++j)
#pragma unroll
      for (int i = 0; i < Pr::TM; ++i)
        f(i, j, m0 + (wave % Pr::WM) * Pr::TM * 16 + 16 * i + 4 * (lane >> 4), n0 + (wave / Pr::WM) * Pr::TN * 16 + 16 * j + (lane & 15));
  };
  if constexpr (early && MODE == 1)
    end([&](int i, int j, int m, int n) { old[j][i] = n < G.s && m < G.sp ? get_parts<NP>(Am + n * la, m) : f4{0, 0, 0, 0}; });
  Pr p;
  p.run(MODE == 4 ? Q : MODE == 1 ? A : X, MODE == 0 || MODE == 4 ? X : MODE == 1 ? A : Q, m0, n0, 0, MODE == 0 ? G.lp : G.sp, (lds_t*)smem);
  if (Pr::KG > 1 && threadIdx.x >= 64 * Pr::NW) return;
  const int rows = MODE == 4 ? G.l : G.s;
  end([&](int i, int j, int m, int n) {
    if (n >= rows) return;
    f4 v = p.acc[i][j];
    if constexpr (MODE <= 1) {
      if (m >= G.sp) return;
      if constexpr (MODE == 0) {
        v = v * (k.a / (k.x * k.x));
      } else {
        f4 a1;
        if constexpr (early) a1 = old[j][i];
        else a1 = get_parts<NP>(Am + n * la, m);
        v = v * (h.c * k.p / (k.a * k.a)) + a1 * (h.b * k.p / k.a);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (m + e == n) v[e] += h.a * k.p;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (m + e >= G.s) v[e] = 0.f;      // (what pads the rows, whatever the operands' rows beyond gave)
      uint16_t* out = MODE == 0 ? Am : Pm;
      put_parts<NP>(out + n * la, m, v);
      if (mt != nt) put_parts_turned<NP>(out + m * la, la, G.s - m, n, v);
    } else if constexpr (MODE == 2) {
      if (m >= G.lp) return;
      put_parts<NP>(G.X[from ^ 1] + ((int64_t)mat * G.s + n) * lx, m, v * (k.next / (k.p * k.x)));
    } else {
      const int cols = MODE == 4 ? G.s : G.l;
      const float f = h.lr * T.scale * (1.f / (k.p * k.x));
      const int64_t o = at + (int64_t)n * cols + m;
      if ((cols & 3) == 0) {
        float w[4];
        if (m >= cols) return;
        get_n<BF, 4>(T.p, o, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = fmaf(-f, v[e], w[e] * h.keep);
        put_n<BF, 4>(T.p, o, w);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (m + e < cols) put<BF>(T.p, o + e, fmaf(-f, v[e], get<BF>(T.p, o + e) * h.keep));
      }
    }
  });
}

// Pr; the tall matrices' last product is PrT, of as many tiles the other way round.
template <class Pr, class PrT, bool BF, int NP, int MODE>
__global__ __launch_bounds__(Pr::kThreads) void muon_product_kernel(MuonGroup G, MuonHyper h, MuonScales k, int from, int tm, int tn) {
  extern __shared__ char smem[];
  int64_t at;
  const MuonTensor& T = tensor_of(G, blockIdx.y, at);
  if (MODE == 3 && T.rows > T.cols) muon_tile<PrT, BF, NP, 4>(G, h, k, T, at, from, tn, tm, smem);
  else muon_tile<Pr, BF, NP, MODE>(G, h, k, T, at, from, tm, tn, smem);
}

template <class Pr, auto kernel>
hipError_t go(dim3 grid, hipStream_t s, const MuonGroup& G, const MuonHyper& h, const MuonScales& k, int from, int tm, int tn) {
  const hipError_t e = allow_lds<kernel>();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, grid, dim3(Pr::kThreads), Pr::kLdsBytes, s, G, h, k, from, tm, tn);
  return hipGetLastError();
}

// The largest tiles that still give every CU one.  Where there is no more than one for each, four steps' tiles are in LDS,
// else two and more workgroups on a CU (1024 x 1024 fp32, 32 steps of its symmetric products' 136 tiles: 200 us with four, 272
// with two; four 768 x 2048 bf16, 312 tiles: 283 with four, 276 with two, five 700 x 720 210 and 179).  Of P X over many steps
// four groups of wavefronts share the contraction (1024 x 1024 fp32: 21.3 -> 15.6 us; the symmetric products, of which only 136
// CUs have one, 13.0 -> 16.6, 59 x 3540 bf16 4.0 -> 5.6).
template <bool BF, int NP, int MODE>
hipError_t product(const MuonGroup& G, const MuonHyper& h, const MuonScales& k, int from, int mats, hipStream_t s) {
  constexpr Side SA = MODE >= 2 ? COL : ROW;
  const int M = MODE >= 2 ? G.lp : G.sp, N = G.s;
  auto tiles = [&](int b) {
    const int64_t m = ceil_div(M, b), n = ceil_div(N, b);
    return (MODE <= 1 ? m * (m + 1) / 2 : m * n) * mats;
  };
#define KRON_MUON_GO(B, NS, KG, ...)                                                                                \
  {                                                                                                                 \
    typedef Product<__VA_ARGS__, SA, ROW, false, NP, NS, false, KG> Pr;                                             \
    typedef Product<__VA_ARGS__, ROW, COL, false, NP, NS, false, KG> PrT;                                           \
    const int tm = (int)ceil_div(M, B), tn = (int)ceil_div(N, B);                                                   \
    return go<Pr, muon_product_kernel<Pr, PrT, BF, NP, MODE>>(dim3((unsigned)(tiles(B) / mats), (unsigned)mats), s, G, h, k, from, tm, tn); \
  }
  if (tiles(256) >= 256) KRON_MUON_GO(256, 2, 1, 2, 4, 8, 4)
  if (tiles(128) >= 256) KRON_MUON_GO(128, 2, 1, 2, 2, 4, 4)
  if (tiles(64) > 256) KRON_MUON_GO(64, 2, 1, 2, 2, 2, 2)
  if constexpr (MODE >= 2)
    if (G.sp * NP >= 1024) KRON_MUON_GO(64, 2, 4, 2, 2, 2, 2)
  KRON_MUON_GO(64, 4, 1, 2, 2, 2, 2)
#undef KRON_MUON_GO
}

template <bool BF>
hipError_t run_group(const MuonGroup& G, const MuonHyper& h, const MuonScales* k, int mats, hipStream_t s) {
  constexpr int NP = BF ? 1 : 2;
  const dim3 grid(kNormParts, (unsigned)mats);
  // (a matrix starts at a multiple of four values where all have as many)
  if ((int64_t)G.s * G.l % 4 == 0) hipLaunchKernelGGL((muon_momentum_kernel<BF, 4>), grid, dim3(256), 0, s, G, h);
  else hipLaunchKernelGGL((muon_momentum_kernel<BF, 1>), grid, dim3(256), 0, s, G, h);
  const int tl = G.lp / 64, ts = (int)ceil_div(G.s, 64);
  hipLaunchKernelGGL((muon_start_kernel<BF, NP>), dim3((unsigned)(tl * ts), (unsigned)mats), dim3(256), 0, s, G, h, tl);
  hipError_t e = hipGetLastError();
  for (int i = 0; i < h.steps && e == hipSuccess; ++i) {
    e = product<BF, NP, 0>(G, h, k[i], i & 1, mats, s);
    if (e == hipSuccess) e = product<BF, NP, 1>(G, h, k[i], i & 1, mats, s);
    if (e == hipSuccess) e = i + 1 < h.steps ? product<BF, NP, 2>(G, h, k[i], i & 1, mats, s) : product<BF, NP, 3>(G, h, k[i], i & 1, mats, s);
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
// and group_mats matrices together.  They run one after the other in the same workspace, which 2^28 values keep below 4.6 GB
// (fp32; one matrix of 16384 x 16384, sixteen of 4096 x 4096, 64 of which would take 17 GB).  By then a few fill the GPU: of
// 4096 x 4096 fp32 one takes 3.76 ms, eight 3.37 each and sixteen 3.29.
constexpr int64_t kGroupMats = 64, kGroupValues = int64_t(1) << 28;
int64_t group_mats(int64_t s, int64_t l) { return std::min(kGroupMats, std::max<int64_t>(1, kGroupValues / (s * l))); }
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
    const int64_t most = group_mats(sl.first, sl.second);
    const bool last = o + 1 == order.size() || size(order[o + 1]) != sl;
    while (rest.count > 0) {
      MuonTensor now = rest;
      now.count = std::min(rest.count, most - mats);
      got[k++] = now;
      mats += now.count;
      const int64_t skip = now.count * rest.rows * rest.cols;
      rest.count -= now.count;
      if (rest.p) {      // (sizes alone have no pointers)
        rest.m += skip;
        rest.p = (char*)rest.p + skip * f.element();
        rest.g = (const char*)rest.g + skip * f.element();
      }
      if (k == kGroup || mats == most || (last && rest.count == 0)) {
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
  const MuonScales* k;
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
    return bf16 ? run_group<true>(G, *h, k, (int)mats, stream) : run_group<false>(G, *h, k, (int)mats, stream);
  }
};

template <bool BF>
hipError_t run_small(const SmallBatch& b, size_t lds, bool large, const MuonHyper& h, hipStream_t s) {
  const dim3 grid((unsigned)b.first[b.n]);
  hipError_t e;
  if (large) {
    if ((e = allow_lds<muon_small_kernel<BF, 1024>>()) != hipSuccess) return e;
    hipLaunchKernelGGL((muon_small_kernel<BF, 1024>), grid, dim3(1024), lds, s, b, h);
  } else {
    if ((e = allow_lds<muon_small_kernel<BF, 512>>()) != hipSuccess) return e;
    hipLaunchKernelGGL((muon_small_kernel<BF, 512>), grid, dim3(512), lds, s, b, h);
  }
  return hipGetLastError();
}

}  // namespace

size_t muon_workspace(const MuonTensor* t, int n, bool bf16) {
  size_t most = 0;
  (void)for_groups(t, n, CountBytes{bf16, &most});
  return most;
}

// The singular values of X are at most 1 at first; a step takes v to v p(v^2), p(l) = a + b l + c l^2, and the values of a
// matrix are at most its largest singular value.  What 16-bit parts leave of A and P (2^-11 at most) comes on top.
bool muon_scales(const MuonHyper& h, MuonScales* k) {
  const double a = h.a, b = h.b, c = h.c;
  auto scale = [](double most) {      // (matrices that shrink from step to step keep their bits as well, down to 2^-25)
    return most >= 0.5 && most <= 6 ? kScale : (float)std::exp2(std::min(40.0, std::floor(std::log2(49152 / most))));
  };
  double x = 1;      // of X
  for (int i = 0; i < h.steps; ++i) {
    const double top = x * x * (1 + 1.0 / 64);      // of A
    const double off = (std::abs(a) + std::abs(b) * top + std::abs(c) * top * top) / 512;
    double p = 0, next = 0;
    auto at = [&](double l) {
      if (!(l >= 0 && l <= top)) return;
      const double v = std::abs(a + l * (b + l * c)) + off;
      p = std::max(p, v), next = std::max(next, std::sqrt(l) * v);
    };
    at(0), at(top);
    if (c != 0) {
      at(-b / (2 * c));      // where p and v p(v^2) turn
      const double d = 9 * b * b - 20 * a * c;
      if (d >= 0) at((-3 * b + std::sqrt(d)) / (10 * c)), at((-3 * b - std::sqrt(d)) / (10 * c));
    } else if (b != 0) {
      at(-a / (3 * b));
    }
    if (!(x <= KRON_MUON_MAX_GROWTH && p <= KRON_MUON_MAX_GROWTH)) return false;
    k[i] = MuonScales{scale(x), scale(top), scale(p), scale(next)};
    x = next;
  }
  return true;
}

hipError_t launch_muon(const MuonTensor* t, int n, const MuonHyper& h, const MuonScales* k, void* ws, hipStream_t s) {
  // Workgroups of 16 wavefronts where a matrix has over 8192 values or more than three tiles of A, of eight else, and more
  // of them on a CU.
  for (int large = 0; large < 2; ++large) {
    SmallBatch b{};
    size_t lds = 0;
    auto flush = [&]() {
      hipError_t e = hipSuccess;
      if (b.n) e = h.bf16 ? run_small<true>(b, lds, large != 0, h, s) : run_small<false>(b, lds, large != 0, h, s);
      b.n = 0, lds = 0;
      return e;
    };
    for (int i = 0; i < n; ++i) {
      if (t[i].count == 0 || !is_small(t[i].rows, t[i].cols) || (t[i].rows * t[i].cols > 8192 || std::min(t[i].rows, t[i].cols) > 32) != (large != 0)) continue;
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
  }
  return for_groups(t, n, RunGroup{h.bf16 != 0, &h, k, (char*)ws, s});
}

}  // namespace kron
