// Low-rank adapters of many requests beside a shared projection.  A request is a run of rows with one
// adapter e (or none): with D_e = down[e] (R x K) and U_e = up[e] (M x R)
//   y = base + s_e (x D_e^T) U_e^T
//   backward, t = s_e x D_e^T and g = s_e dy U_e:  dx = base + g D_e,  dD_e = g^T x,  dU_e = dy^T t
// Sixteen rows of one request are a workgroup's: their inner product stays on chip, x is read once and y written
// once.  bf16 x and D_e are multiplied by the bf16 matrix instruction (exact products), everything else by the fp32
// one: neither the inner products nor the gradients are rounded on the way.
#include <algorithm>

#include "kron_internal.h"
#include "row_tile.h"

namespace kron {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

constexpr int kRows = 16;            // rows of a tile
constexpr int kThreads = 256, kWaves = 4;

__device__ inline f4 mma32(float a, float b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }
__device__ inline f4 mma16(u4 a, u4 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
}

// Sixteen bytes of a row (four fp32 values, eight bf16), of which `left` values are in it; the others are zero.  Rows
// may start at any element (the memory pipes take a vector at any address, once aligned to its elements).
template <bool BF>
__device__ inline u4 load16(const void* p, int64_t i, int left) {
  constexpr int N = BF ? 8 : 4;
  const char* q = (const char*)p + i * (BF ? 2 : 4);
  u4 v = {0, 0, 0, 0};
  if (left >= N) {
    __builtin_memcpy(&v, q, 16);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < left) {
        if (BF) v[e / 2] |= (uint32_t)((const uint16_t*)q)[e] << (16 * (e & 1));
        else v[e] = ((const uint32_t*)q)[e];
      }
  }
  return v;
}
// Four neighbours as fp32.
template <bool BF>
__device__ inline f4 load4(const void* p, int64_t i, int left) {
  if (!BF) return __builtin_bit_cast(f4, load16<false>(p, i, left));
  const char* q = (const char*)p + i * 2;
  uint2 w = {0, 0};
  if (left >= 4) {
    __builtin_memcpy(&w, q, 8);
  } else {
    if (left > 0) w.x = ((const uint16_t*)q)[0];
    if (left > 1) w.x |= (uint32_t)((const uint16_t*)q)[1] << 16;
    if (left > 2) w.y = ((const uint16_t*)q)[2];
  }
  return f4{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
}
template <bool BF>
__device__ inline float load1(const void* p, int64_t i) {
  return BF ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}
// Value e of what load16 gave.
template <bool BF>
__device__ inline float value(const u4& v, int e) {
  if (BF) return (e & 1) ? bf16_hi(v[e / 2]) : bf16_lo(v[e / 2]);
  return __uint_as_float(v[e & 3]);
}
// base + acc of N neighbours (fp32: 4, bf16: 8), `left` of them in the row, rounded once.
template <bool BF>
__device__ inline void store16(void* p, int64_t i, int left, const u4& base, const f4* acc) {
  constexpr int N = BF ? 8 : 4;
  float v[N];
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = value<BF>(base, e) + acc[e / 4][e & 3];
  char* q = (char*)p + i * (BF ? 2 : 4);
  u4 o;
#pragma unroll
  for (int w = 0; w < 4; ++w) o[w] = BF ? bf16_pair(v[(2 * w) % N], v[(2 * w + 1) % N]) : __float_as_uint(v[w % N]);
  if (left >= N) {
    __builtin_memcpy(q, &o, 16);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < left) {
        if (BF) ((uint16_t*)q)[e] = (uint16_t)(o[e / 2] >> (16 * (e & 1)));
        else ((uint32_t*)q)[e] = o[e & 3];
      }
  }
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

// The wavefronts' parts of a 16 x R product, joined, times f: t[16][RT * 16 + 4].
template <int RT>
__device__ inline void join(const Adapters& a, const f4* acc, float f, float* red, float* t) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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

// t = f v w^T for the tile's rows of v (width n) and w (R x n): the wavefronts share the contraction, each with
// kBatch blocks of it in flight (a block's latency after the other's, 64 tokens of 1024 -> 4096 took 13.7 us).
template <bool BF, int RT>
__device__ inline void inner(const Adapters& a, const Tile& T, const void* v, const void* w, int n, float f, float* red, float* t) {
  constexpr int KB = BF ? 32 : 16, VE = BF ? 8 : 4, kBatch = RT >= 8 ? 1 : 8 / RT;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  f4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f4{0, 0, 0, 0};
  const int64_t vrow = (T.row + min(c, T.rows - 1)) * n;
  int64_t wrow[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) wrow[i] = (int64_t)min(16 * i + c, a.R - 1) * n;
  for (int k = wave * KB; k < n; k += kBatch * kWaves * KB) {
    u4 x[kBatch], d[kBatch][RT];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int at = k + b * kWaves * KB + VE * g;
      x[b] = load16<BF>(v, vrow + at, n - at);
#pragma unroll
      for (int i = 0; i < RT; ++i) d[b][i] = load16<BF>(w, wrow[i] + at, n - at);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        if constexpr (BF) {
          acc[i] = mma16(x[b], d[b][i], acc[i]);      // rows x rank
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i] = mma32(value<false>(x[b], q), value<false>(d[b][i], q), acc[i]);
        }
      }
  }
  join<RT>(a, acc, f, red, t);
}

// g = f v w for w (n x R): w's values one by one, sixteen neighbours of a row together.
template <bool BF, int RT>
__device__ inline void inner_t(const Adapters& a, const Tile& T, const void* v, const void* w, int n, float f, float* red, float* t) {
  constexpr int KB = BF ? 32 : 16, VE = BF ? 8 : 4, kBatch = RT >= 4 ? 1 : (BF ? 4 : 8) / RT;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  f4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f4{0, 0, 0, 0};
  const int64_t vrow = (T.row + min(c, T.rows - 1)) * n;
  for (int k = wave * KB; k < n; k += kBatch * kWaves * KB) {
    u4 x[kBatch];
    float u[kBatch][RT][VE];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int at = k + b * kWaves * KB + VE * g;
      x[b] = load16<BF>(v, vrow + at, n - at);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int q = 0; q < VE; ++q) u[b][i][q] = load1<BF>(w, (int64_t)min(at + q, n - 1) * a.R + min(16 * i + c, a.R - 1));
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int q = 0; q < VE; ++q) acc[i] = mma32(value<BF>(x[b], q), u[b][i][q], acc[i]);
  }
  join<RT>(a, acc, f, red, t);
}

// Column of a row of y or dx that lane c of block h (of the two that bf16 takes together) stands for: the lane that
// holds rows 4 g .. 4 g + 3 of both results then has eight neighbours, 16 bytes.
template <bool BF>
__device__ inline int column(int c, int h) { return BF ? 8 * (c >> 2) + 4 * h + (c & 3) : c; }

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

template <bool BF, int RT>
__global__ __launch_bounds__(kThreads) void adapters_fwd_kernel(Adapters a) {
  __shared__ Shared<RT> sh;
  const Tile T = find_tile(a, blockIdx.x, sh.find);
  if (T.rows == 0) return;
  if (T.id < 0 || T.id >= a.E) {
    plain_rows<BF>(a, T, a.base, a.y, a.M, blockIdx.y, gridDim.y);
    return;
  }
  constexpr int H = BF ? 2 : 1, W = 16 * H, kBatch = RT >= 4 ? 1 : 4 / RT / H + (RT == 2 && BF);
  const size_t es = BF ? 2 : 4;
  const float f = a.scales ? a.scales[T.id] : 1.f;
  const char* D = (const char*)a.down + (size_t)T.id * a.R * a.K * es;
  const char* U = (const char*)a.up + (size_t)T.id * a.R * a.M * es;
  inner<BF, RT>(a, T, a.x, D, a.K, f, sh.red, sh.t);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  f4 t[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) t[i] = *(const f4*)(sh.t + c * (RT * 16 + 4) + 16 * i + 4 * g);
  const int64_t row = (T.row + min(c, T.rows - 1)) * a.M;
  const int stride = (int)gridDim.y * kWaves * W;
  for (int m = (blockIdx.y * kWaves + wave) * W; m < a.M; m += kBatch * stride) {
    f4 u[kBatch][H][RT];
    u4 base[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int m0 = m + b * stride, at = m0 + 4 * H * g;
      base[b] = load16<BF>(a.base, row + at, a.M - at);
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < RT; ++i)
          u[b][h][i] = load4<BF>(U, (int64_t)min(m0 + column<BF>(c, h), a.M - 1) * a.R + 16 * i + 4 * g, a.R - 16 * i - 4 * g);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      f4 acc[H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        acc[h] = f4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[h] = mma32(u[b][h][i][q], t[i][q], acc[h]);      // columns of y x rows
      }
      const int at = m + b * stride + 4 * H * g;
      if (c < T.rows) store16<BF>(a.y, row + at, a.M - at, base[b], acc);
    }
  }
}

// The rows' part of the backward: t and g of each row for the gradients' kernel, and dx.
template <bool BF, int RT>
__global__ __launch_bounds__(kThreads) void adapters_rows_kernel(Adapters a) {
  __shared__ Shared<RT> sh;
  const Tile T = find_tile(a, blockIdx.x, sh.find);
  if (T.rows == 0) return;
  if (T.id < 0 || T.id >= a.E) {
    if (a.y) plain_rows<BF>(a, T, a.base, a.y, a.K, 0, 1);
    return;
  }
  constexpr int H = BF ? 2 : 1, W = 16 * H, kBatch = RT >= 4 ? 1 : 4 / RT / H + (RT == 2 && BF);
  const size_t es = BF ? 2 : 4;
  const float f = a.scales ? a.scales[T.id] : 1.f;
  const char* D = (const char*)a.down + (size_t)T.id * a.R * a.K * es;
  const char* U = (const char*)a.up + (size_t)T.id * a.R * a.M * es;
  inner<BF, RT>(a, T, a.x, D, a.K, f, sh.red, sh.t);
  inner_t<BF, RT>(a, T, a.dy, U, a.M, f, sh.red, sh.g);
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
  for (int k = wave * W; k < a.K; k += kBatch * kWaves * W) {
    float d[kBatch][H][RT][4];
    u4 base[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int k0 = k + b * kWaves * W, at = k0 + 4 * H * g;
      base[b] = a.base ? load16<BF>(a.base, row + at, a.K - at) : u4{0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            d[b][h][i][q] = load1<BF>(D, (int64_t)min(16 * i + 4 * g + q, a.R - 1) * a.K + min(k0 + column<BF>(c, h), a.K - 1));
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      f4 acc[H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        acc[h] = f4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[h] = mma32(d[b][h][i][q], t[i][q], acc[h]);
      }
      const int at = k + b * kWaves * W + 4 * H * g;
      if (c < T.rows) store16<BF>(a.y, row + at, a.K - at, base[b], acc);
    }
  }
}

// The adapters' gradients: a block of columns of x (dD = g^T x) or of dy (dU = dy^T t) of one adapter, over every
// `splits`-th four rows of its.  A lane has NC neighbouring columns: column NC c + q is lane c's of product q.
template <bool BF, int RT>
constexpr int lane_cols() { return BF && RT <= 2 ? 8 : 4; }
template <bool BF, int RT>
__global__ __launch_bounds__(kThreads) void adapters_params_kernel(Adapters a, int kblocks, int splits, float* part) {
  constexpr int NC = lane_cols<BF, RT>(), kBatch = RT >= 4 ? 2 : 4;
  __shared__ float red[kWaves][RT * NC][256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  const int e = blockIdx.y, split = blockIdx.z;
  const bool up = (int)blockIdx.x >= kblocks;
  const int n = up ? a.M : a.K, col0 = (up ? blockIdx.x - kblocks : blockIdx.x) * 16 * NC, mine = col0 + NC * c;
  const void* v = up ? a.dy : a.x;
  const float* tg = a.ws + (up ? 0 : RT * 16);
  f4 acc[RT][NC];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int q = 0; q < NC; ++q) acc[i][q] = f4{0, 0, 0, 0};
  const int stride = kWaves * splits, turn = split * kWaves + wave;
  int64_t seen = 0;      // blocks of four rows before
  for (int i0 = 0; i0 < a.B; i0 += 64) {
    uint64_t todo = __ballot(i0 + lane < a.B && a.ids[min(i0 + lane, a.B - 1)] == e);
    while (todo) {
      const int i = i0 + __builtin_ctzll(todo);
      todo &= todo - 1;
      int64_t r0 = i, r1 = min<int64_t>(i + 1, a.N);
      if (a.starts) segment(a, i + 1, r0, r1);
      const int64_t blocks = (r1 - r0 + 3) / 4;
      int64_t b = (turn - seen % stride + stride) % stride;
      seen += blocks;
      for (; b < blocks; b += kBatch * stride) {
        u4 x[kBatch];
        float w[kBatch][RT];
#pragma unroll
        for (int t = 0; t < kBatch; ++t) {
          const int64_t row = r0 + 4 * (b + t * stride) + g;
          const bool in = row < r1;
          x[t] = u4{0, 0, 0, 0};
          if (in) {
            if (NC == 4 && BF) {
              const f4 y = load4<BF>(v, row * n + mine, n - mine);
              x[t] = __builtin_bit_cast(u4, y);
            } else {
              x[t] = load16<BF>(v, row * n + mine, n - mine);
            }
          }
#pragma unroll
          for (int k = 0; k < RT; ++k) w[t][k] = in ? tg[row * 2 * RT * 16 + 16 * k + c] : 0.f;
        }
#pragma unroll
        for (int t = 0; t < kBatch; ++t)
#pragma unroll
          for (int k = 0; k < RT; ++k)
#pragma unroll
            for (int q = 0; q < NC; ++q) acc[k][q] = mma32(w[t][k], value<NC == 8>(x[t], q), acc[k][q]);      // rank x columns
      }
    }
  }
#pragma unroll
  for (int k = 0; k < RT; ++k)
#pragma unroll
    for (int q = 0; q < NC; ++q) *(f4*)&red[wave][k * NC + q][lane * 4] = acc[k][q];
  __syncthreads();
  float* out = splits > 1 ? part + (int64_t)split * a.E * a.R * (a.K + a.M) : nullptr;
  for (int x = threadIdx.x; x < RT * NC * 256; x += kThreads) {
    // dD's neighbours along the columns, dU's along the rank
    const int k = x / (NC * 256), w = x % (NC * 256);
    const int rr = up ? w % 16 : w / (16 * NC), cc = up ? w / 16 : w % (16 * NC);
    const int r = 16 * k + rr, col = col0 + cc, kq = k * NC + cc % NC, ln = (rr >> 2) * 16 + cc / NC;
    if (r >= a.R || col >= n) continue;
    float s = 0.f;
#pragma unroll
    for (int t = 0; t < kWaves; ++t) s += red[t][kq][ln * 4 + (rr & 3)];
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

int cols_of(const Adapters& a) { return 16 * (a.bf16 && a.R <= 32 ? 8 : 4); }      // lane_cols() of sixteen lanes

// Workgroups that share an adapter's rows, so that every CU has two.
int splits_of(const Adapters& a) {
  const int64_t groups = (ceil_div(a.K, cols_of(a)) + ceil_div(a.M, cols_of(a))) * a.E;
  return (int)std::max<int64_t>(1, std::min({ceil_div(512, groups), ceil_div(a.N, 256), int64_t(16)}));
}

template <bool BF, int RT>
hipError_t fwd(const Adapters& a, hipStream_t s) {
  const int64_t tiles = tiles_of(a);
  // few tiles: several workgroups share a tile's columns, each with the inner product to itself
  const int gy = (int)std::max<int64_t>(1, std::min(256 / tiles, ceil_div(a.M, kWaves * 16)));
  hipLaunchKernelGGL((adapters_fwd_kernel<BF, RT>), dim3((unsigned)tiles, (unsigned)gy), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <bool BF, int RT>
hipError_t bwd(const Adapters& a, hipStream_t s) {
  if (a.N) hipLaunchKernelGGL((adapters_rows_kernel<BF, RT>), dim3((unsigned)tiles_of(a)), dim3(kThreads), 0, s, a);
  const int splits = splits_of(a), kb = (int)ceil_div(a.K, cols_of(a)), mb = (int)ceil_div(a.M, cols_of(a));
  float* part = (float*)((char*)a.ws + up256(sizeof(float) * (size_t)a.N * 2 * RT * 16));
  hipLaunchKernelGGL((adapters_params_kernel<BF, RT>), dim3((unsigned)(kb + mb), (unsigned)a.E, (unsigned)splits), dim3(kThreads), 0, s, a, kb,
                     splits, part);
  if (splits > 1) {
    const int64_t n = (int64_t)a.E * a.R * (a.K + a.M);
    hipLaunchKernelGGL(adapters_join_kernel, dim3((unsigned)std::min<int64_t>(2048, ceil_div(n, kThreads))), dim3(kThreads), 0, s, a, splits, part);
  }
  return hipGetLastError();
}

template <int RT>
hipError_t pick(const Adapters& a, bool backward, hipStream_t s) {
  if (backward) return a.bf16 ? bwd<true, RT>(a, s) : bwd<false, RT>(a, s);
  return a.bf16 ? fwd<true, RT>(a, s) : fwd<false, RT>(a, s);
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
