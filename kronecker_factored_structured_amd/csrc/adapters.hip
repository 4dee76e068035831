// Low-rank adapters of many requests beside a shared projection.  A request is a run of rows with one
// adapter e (or none): with D_e = down[e] (R x K) and U_e = up[e] (M x R)
//   y = base + s_e (x D_e^T) U_e^T
//   backward, t = s_e x D_e^T and g = s_e dy U_e:  dx = base + g D_e,  dD_e = g^T x,  dU_e = dy^T t
// Sixteen rows of one request are a workgroup's: their inner product stays on chip, x is read once and y written
// once.  All products run on the fp32 matrix instruction (bf16 values are exact in it): the work is bound by
// memory, and neither the inner products nor the gradients are rounded on the way.
#include <algorithm>

#include "kron_internal.h"
#include "row_tile.h"

namespace kron {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kRows = 16;            // rows of a tile
constexpr int kThreads = 256, kWaves = 4;

__device__ inline f4 mma32(float a, float b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// Four neighbouring values of a row at p + i; those from `end` on are zero.  VEC: the row and i are multiples of four.
template <bool BF, bool VEC>
__device__ inline f4 load4(const void* p, int64_t i, int left) {
  f4 v = {0, 0, 0, 0};
  if (VEC) {
    if (left <= 0) return v;
    if (BF) {
      const uint2 w = *(const uint2*)((const uint16_t*)p + i);
      return f4{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
    }
    return *(const f4*)((const float*)p + i);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) v[e] = BF ? __uint_as_float((uint32_t)((const uint16_t*)p)[i + e] << 16) : ((const float*)p)[i + e];
  return v;
}
template <bool BF, bool VEC>
__device__ inline void store4(void* p, int64_t i, int left, f4 v) {
  if (VEC) {
    if (left <= 0) return;
    if (BF) *(uint2*)((uint16_t*)p + i) = uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    else *(f4*)((float*)p + i) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) {
      if (BF) ((uint16_t*)p)[i + e] = (uint16_t)bf16_rne(v[e]);
      else ((float*)p)[i + e] = v[e];
    }
}
template <bool BF>
__device__ inline float load1(const void* p, int64_t i) {
  return BF ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}

// Segment i of B + 2: the requests, and the rows before the first and behind the last one (no adapter).
__device__ inline void segment(const Adapters& a, int i, int64_t& r0, int64_t& r1) {
  const int64_t lo = i == 0 ? 0 : a.starts[i - 1], hi = i == a.B + 1 ? a.N : a.starts[i];
  r0 = min<int64_t>(max<int64_t>(lo, 0), a.N);
  r1 = min<int64_t>(max<int64_t>(hi, r0), a.N);
}

struct Tile {
  int64_t row;       // first
  int rows, id;      // 0 rows: none
};

// The tile of workgroup `w`: the w-th block of sixteen rows, counted request by request.
__device__ inline Tile find_tile(const Adapters& a, int64_t w, int* sh) {
  if (!a.starts) return {w, w < a.N ? 1 : 0, w < a.N ? a.ids[w] : -1};
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int64_t before = 0;
  if (tid == 0) sh[5] = -1;
  for (int i0 = 0; i0 < a.B + 2; i0 += kThreads) {
    int64_t r0 = 0, r1 = 0;
    if (i0 + tid < a.B + 2) segment(a, i0 + tid, r0, r1);
    const int mine = (int)((r1 - r0 + kRows - 1) / kRows);
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int v = __shfl_up(sum, o, 64);
      if (lane >= o) sum += v;
    }
    if (lane == 63) sh[wave] = sum;
    __syncthreads();
    int64_t at = before + sum - mine;
    int64_t all = 0;
    for (int k = 0; k < kWaves; ++k) {
      if (k < wave) at += sh[k];
      all += sh[k];
    }
    if (w >= at && w < at + mine) sh[4] = (int)(w - at), sh[5] = i0 + tid;
    before += all;
    __syncthreads();
    if (w < before) break;
  }
  const int i = sh[5];
  if (i < 0) return {0, 0, -1};
  int64_t r0, r1;
  segment(a, i, r0, r1);
  r0 += (int64_t)sh[4] * kRows;
  return {r0, (int)min<int64_t>(kRows, r1 - r0), i == 0 || i == a.B + 1 ? -1 : a.ids[i - 1]};
}

// t[16][R] = f v w^T for the tile's rows of v (width n) and w (R x n): the wavefronts share the contraction.
template <bool BF, bool VEC, int RT>
__device__ inline void inner(const Adapters& a, const Tile& T, const void* v, const void* w, int n, float f, float* red, float* t) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  f4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f4{0, 0, 0, 0};
  const int64_t vrow = (T.row + min(c, T.rows - 1)) * n;
  for (int k = wave * 16; k < n; k += kWaves * 16) {
    const int at = k + 4 * g;
    const f4 x = load4<BF, VEC>(v, vrow + at, n - at);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const f4 d = load4<BF, VEC>(w, (int64_t)min(16 * i + c, a.R - 1) * n + at, n - at);
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i] = mma32(x[q], d[q], acc[i]);      // rows x rank
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) *(f4*)(red + ((wave * RT + i) * 64 + lane) * 4) = acc[i];
  __syncthreads();
  for (int e = threadIdx.x; e < RT * 256; e += kThreads) {
    const int i = e >> 8, ln = (e & 255) >> 2, q = e & 3;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) s += red[(k * RT * 64) * 4 + e];
    const int r = 16 * i + (ln & 15);
    t[(4 * (ln >> 4) + q) * (RT * 16 + 4) + r] = r < a.R ? s * f : 0.f;
  }
  __syncthreads();
}

// g[16][R] = f v w for w (n x R): w's values one by one, sixteen neighbours of a row together.
template <bool BF, bool VEC, int RT>
__device__ inline void inner_t(const Adapters& a, const Tile& T, const void* v, const void* w, int n, float f, float* red, float* t) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  f4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f4{0, 0, 0, 0};
  const int64_t vrow = (T.row + min(c, T.rows - 1)) * n;
  for (int k = wave * 16; k < n; k += kWaves * 16) {
    const int at = k + 4 * g;
    const f4 x = load4<BF, VEC>(v, vrow + at, n - at);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = min(16 * i + c, a.R - 1);
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i] = mma32(x[q], load1<BF>(w, (int64_t)min(at + q, n - 1) * a.R + r), acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) *(f4*)(red + ((wave * RT + i) * 64 + lane) * 4) = acc[i];
  __syncthreads();
  for (int e = threadIdx.x; e < RT * 256; e += kThreads) {
    const int i = e >> 8, ln = (e & 255) >> 2, q = e & 3;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) s += red[(k * RT * 64) * 4 + e];
    const int r = 16 * i + (ln & 15);
    t[(4 * (ln >> 4) + q) * (RT * 16 + 4) + r] = r < a.R ? s * f : 0.f;
  }
  __syncthreads();
}

// Rows without an adapter: out = base (zeros without one), NaN where the id is none of the table's.
template <bool BF>
__device__ inline void plain_rows(const Adapters& a, const Tile& T, const void* base, void* out, int n, int part, int parts) {
  if (T.id < 0 && base == out) return;
  for (int64_t i = (int64_t)part * kThreads + threadIdx.x; i < (int64_t)T.rows * n; i += (int64_t)parts * kThreads) {
    const int64_t at = T.row * n + i;
    if (T.id >= 0) {
      if (BF) ((uint16_t*)out)[at] = 0x7fc0;
      else ((float*)out)[at] = NAN;
    } else if (BF) {
      ((uint16_t*)out)[at] = base ? ((const uint16_t*)base)[at] : 0;
    } else {
      ((float*)out)[at] = base ? ((const float*)base)[at] : 0.f;
    }
  }
}

template <int RT>
struct Shared {
  float red[kWaves * RT * 256];
  float t[kRows * (RT * 16 + 4)];
  float g[kRows * (RT * 16 + 4)];
  int find[8];
};

template <bool BF, bool VEC, bool RVEC, int RT>
__global__ __launch_bounds__(kThreads) void adapters_fwd_kernel(Adapters a) {
  __shared__ Shared<RT> sh;
  const Tile T = find_tile(a, blockIdx.x, sh.find);
  if (T.rows == 0) return;
  if (T.id < 0 || T.id >= a.E) {
    plain_rows<BF>(a, T, a.base, a.y, a.M, blockIdx.y, gridDim.y);
    return;
  }
  const size_t es = BF ? 2 : 4;
  const float f = a.scales ? a.scales[T.id] : 1.f;
  const char* D = (const char*)a.down + (size_t)T.id * a.R * a.K * es;
  const char* U = (const char*)a.up + (size_t)T.id * a.R * a.M * es;
  inner<BF, VEC, RT>(a, T, a.x, D, a.K, f, sh.red, sh.t);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  f4 t[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) t[i] = *(const f4*)(sh.t + c * (RT * 16 + 4) + 16 * i + 4 * g);
  const int64_t row = (T.row + min(c, T.rows - 1)) * a.M;
  for (int m = (blockIdx.y * kWaves + wave) * 16; m < a.M; m += (int)gridDim.y * kWaves * 16) {
    f4 acc = {0, 0, 0, 0};
    const int64_t urow = (int64_t)min(m + c, a.M - 1) * a.R;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const f4 u = load4<BF, RVEC>(U, urow + 16 * i + 4 * g, a.R - 16 * i - 4 * g);
#pragma unroll
      for (int q = 0; q < 4; ++q) acc = mma32(u[q], t[i][q], acc);      // columns of y x rows
    }
    const int at = m + 4 * g;
    if (c < T.rows) store4<BF, VEC>(a.y, row + at, a.M - at, load4<BF, VEC>(a.base, row + at, a.M - at) + acc);
  }
}

// The rows' part of the backward: t and g of each row for the gradients' kernel, and dx.
template <bool BF, bool VEC, int RT>
__global__ __launch_bounds__(kThreads) void adapters_rows_kernel(Adapters a) {
  __shared__ Shared<RT> sh;
  const Tile T = find_tile(a, blockIdx.x, sh.find);
  if (T.rows == 0) return;
  if (T.id < 0 || T.id >= a.E) {
    if (a.y) plain_rows<BF>(a, T, a.base, a.y, a.K, 0, 1);
    return;
  }
  const size_t es = BF ? 2 : 4;
  const float f = a.scales ? a.scales[T.id] : 1.f;
  const char* D = (const char*)a.down + (size_t)T.id * a.R * a.K * es;
  const char* U = (const char*)a.up + (size_t)T.id * a.R * a.M * es;
  inner<BF, VEC, RT>(a, T, a.x, D, a.K, f, sh.red, sh.t);
  inner_t<BF, VEC, RT>(a, T, a.dy, U, a.M, f, sh.red, sh.g);
  float* keep = a.ws + T.row * 2 * (RT * 16);
  for (int e = threadIdx.x; e < T.rows * RT * 16; e += kThreads) {
    const int r = e / (RT * 16), k = e % (RT * 16);
    keep[(int64_t)r * 2 * RT * 16 + k] = sh.t[r * (RT * 16 + 4) + k];
    keep[(int64_t)r * 2 * RT * 16 + RT * 16 + k] = sh.g[r * (RT * 16 + 4) + k];
  }
  if (!a.y) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  f4 t[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) t[i] = *(const f4*)(sh.g + c * (RT * 16 + 4) + 16 * i + 4 * g);
  const int64_t row = (T.row + min(c, T.rows - 1)) * a.K;
  for (int k = wave * 16; k < a.K; k += kWaves * 16) {
    f4 acc = {0, 0, 0, 0};
    const int col = min(k + c, a.K - 1);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc = mma32(load1<BF>(D, (int64_t)min(16 * i + 4 * g + q, a.R - 1) * a.K + col), t[i][q], acc);
    const int at = k + 4 * g;
    if (c < T.rows) {
      if (a.base) acc += load4<BF, VEC>(a.base, row + at, a.K - at);
      store4<BF, VEC>(a.y, row + at, a.K - at, acc);
    }
  }
}

// The adapters' gradients: 64 columns of x (dD = g^T x) or of dy (dU = dy^T t) of one adapter, over every
// `splits`-th block of its rows.
constexpr int kCols = 64;
template <bool BF, bool VEC, int RT>
__global__ __launch_bounds__(kThreads) void adapters_params_kernel(Adapters a, int kblocks, int splits, float* part) {
  __shared__ float red[kWaves][RT * 4][256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  const int e = blockIdx.y, split = blockIdx.z;
  const bool up = (int)blockIdx.x >= kblocks;
  const int n = up ? a.M : a.K, col0 = (up ? blockIdx.x - kblocks : blockIdx.x) * kCols;
  const void* v = up ? a.dy : a.x;
  const float* tg = a.ws + (up ? 0 : RT * 16);
  f4 acc[RT][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[i][q] = f4{0, 0, 0, 0};
  const int stride = kWaves * splits, turn = split * kWaves + wave;
  int64_t seen = 0;      // blocks of four rows before
  for (int i0 = 0; i0 < a.B; i0 += 64) {
    const bool mine = i0 + lane < a.B && a.ids[min(i0 + lane, a.B - 1)] == e;
    uint64_t todo = __ballot(mine);
    while (todo) {
      const int i = i0 + __builtin_ctzll(todo);
      todo &= todo - 1;
      int64_t r0 = i, r1 = min<int64_t>(i + 1, a.N);
      if (a.starts) segment(a, i + 1, r0, r1);
      const int64_t blocks = (r1 - r0 + 3) / 4;
      int64_t b = (turn - seen % stride + stride) % stride;
      seen += blocks;
      for (; b < blocks; b += stride) {
        const int64_t row = r0 + 4 * b + g;
        const bool in = row < r1;
        const int64_t rr = in ? row : r0;
        const f4 x = load4<BF, VEC>(v, rr * n + col0 + 4 * c, n - col0 - 4 * c);
#pragma unroll
        for (int k = 0; k < RT; ++k) {
          const float w = tg[rr * 2 * RT * 16 + 16 * k + c];
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[k][q] = mma32(in ? w : 0.f, in ? x[q] : 0.f, acc[k][q]);      // rank x columns
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < RT; ++k)
#pragma unroll
    for (int q = 0; q < 4; ++q) *(f4*)&red[wave][k * 4 + q][lane * 4] = acc[k][q];
  __syncthreads();
  float* out = splits > 1 ? part + (int64_t)split * a.E * a.R * (a.K + a.M) : nullptr;
  for (int x = threadIdx.x; x < RT * 4 * 256; x += kThreads) {
    const int kq = x >> 8, w = x & 255;
    const int r = 16 * (kq >> 2) + 4 * (w >> 6) + (w & 3), col = col0 + 4 * ((w >> 2) & 15) + (kq & 3);
    if (r >= a.R || col >= n) continue;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) s += red[k][kq][w];
    if (up) (out ? out + (int64_t)a.E * a.R * a.K : a.dup)[((int64_t)e * a.M + col) * a.R + r] = s;
    else (out ? out : a.ddown)[((int64_t)e * a.R + r) * a.K + col] = s;
  }
}

__global__ __launch_bounds__(kThreads) void adapters_join_kernel(Adapters a, int splits, const float* part) {
  const int64_t nd = (int64_t)a.E * a.R * a.K, n = nd + (int64_t)a.E * a.R * a.M;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
    float s = 0.f;
    for (int k = 0; k < splits; ++k) s += part[(int64_t)k * n + i];
    (i < nd ? a.ddown[i] : a.dup[i - nd]) = s;
  }
}

// ------------------------------------------------------------------------------ host
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
int rank_blocks(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

int64_t tiles_of(const Adapters& a) { return a.starts ? ceil_div(a.N, kRows) + a.B + 1 : a.N; }

// Workgroups that share an adapter's rows, so that every CU has two.
int splits_of(const Adapters& a) {
  const int64_t groups = (ceil_div(a.K, kCols) + ceil_div(a.M, kCols)) * a.E;
  return (int)std::max<int64_t>(1, std::min({ceil_div(512, groups), ceil_div(a.N, 256), int64_t(16)}));
}

template <bool BF, bool VEC, bool RVEC, int RT>
hipError_t fwd(const Adapters& a, hipStream_t s) {
  const int64_t tiles = tiles_of(a);
  // few tiles: several workgroups share a tile's columns, each with the inner product to itself
  const int gy = (int)std::max<int64_t>(1, std::min(256 / tiles, ceil_div(a.M, kWaves * 16)));
  hipLaunchKernelGGL((adapters_fwd_kernel<BF, VEC, RVEC, RT>), dim3((unsigned)tiles, (unsigned)gy), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <bool BF, bool VEC, int RT>
hipError_t bwd(const Adapters& a, hipStream_t s) {
  if (a.N) hipLaunchKernelGGL((adapters_rows_kernel<BF, VEC, RT>), dim3((unsigned)tiles_of(a)), dim3(kThreads), 0, s, a);
  const int splits = splits_of(a), kb = (int)ceil_div(a.K, kCols), mb = (int)ceil_div(a.M, kCols);
  float* part = (float*)((char*)a.ws + up256(sizeof(float) * (size_t)a.N * 2 * RT * 16));
  hipLaunchKernelGGL((adapters_params_kernel<BF, VEC, RT>), dim3((unsigned)(kb + mb), (unsigned)a.E, (unsigned)splits), dim3(kThreads), 0, s, a,
                     kb, splits, part);
  if (splits > 1) {
    const int64_t n = (int64_t)a.E * a.R * (a.K + a.M);
    hipLaunchKernelGGL(adapters_join_kernel, dim3((unsigned)std::min<int64_t>(2048, ceil_div(n, kThreads))), dim3(kThreads), 0, s, a, splits, part);
  }
  return hipGetLastError();
}

template <bool BF, int RT>
hipError_t pick(const Adapters& a, bool backward, hipStream_t s) {
  const bool vec = a.K % 4 == 0 && a.M % 4 == 0, rvec = a.R % 4 == 0;
  if (backward) return vec ? bwd<BF, true, RT>(a, s) : bwd<BF, false, RT>(a, s);
  if (vec) return rvec ? fwd<BF, true, true, RT>(a, s) : fwd<BF, true, false, RT>(a, s);
  return rvec ? fwd<BF, false, true, RT>(a, s) : fwd<BF, false, false, RT>(a, s);
}
template <int RT>
hipError_t pick(const Adapters& a, bool backward, hipStream_t s) {
  return a.bf16 ? pick<true, RT>(a, backward, s) : pick<false, RT>(a, backward, s);
}

}  // namespace

size_t adapters_workspace(const Adapters& a, bool backward) {
  if (!backward) return 0;
  const int splits = splits_of(a);
  return up256(sizeof(float) * (size_t)a.N * 2 * rank_blocks(a.R) * 16) +
         (splits > 1 ? sizeof(float) * (size_t)splits * a.E * a.R * (a.K + a.M) : 0);
}

hipError_t launch_adapters(const Adapters& k, bool backward, void* ws, hipStream_t s) {
  Adapters a = k;
  a.ws = (float*)ws;
  switch (rank_blocks(a.R)) {
    case 1: return pick<1>(a, backward, s);
    case 2: return pick<2>(a, backward, s);
    case 4: return pick<4>(a, backward, s);
    default: return pick<8>(a, backward, s);
  }
}

}  // namespace kron
