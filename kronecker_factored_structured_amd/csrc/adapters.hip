// Low-rank adapters of many requests beside a shared projection.  A request is a run of rows with one
// adapter e (or none): with D_e = down[e] (R x K) and U_e = up[e] (M x R)
//   y = base + s_e (x D_e^T) U_e^T
//   backward, t = s_e x D_e^T and g = s_e dy U_e:  dx = base + g D_e,  dD_e = g^T x,  dU_e = dy^T t
// Sixteen rows of one request are a workgroup's, or 32 and twice the wavefronts where there are many (D_e and U_e are
// read once for all of them): their inner product stays on chip, x is read once and y written once.  bf16 x and D_e are
// multiplied by the bf16 matrix instruction (exact products), everything else by the fp32 one: neither the inner products
// nor the gradients are rounded on the way.
//
// What bounds it: for few rows a chain of two dependent loads with a join between them (one token of 768 -> 2048 rank 16
// 5.1 us, 64 tokens of 1024 -> 4096 8.1), for many the reading of x and base and the writing of y in turn (8192 rows of
// 1024 -> 1024 rank 24 fp32: 39.7 us, 2.5 TB/s; matrix cores busy 0.26).  Backward of 8192 rows of 768 -> 2048 rank 16 bf16:
// the rows' kernel 23.5 us, the parameters' 27.7 (x and dy once more, in 352 workgroups of unlike many rows).
#include <algorithm>

#include "kron_internal.h"
#include "row_tile.h"

namespace kron {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;        // of a workgroup for each sixteen rows (RB of them)
constexpr int kWaves = 4;

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

// The tile of workgroup `w`: the w-th block of 16 RB rows, counted request by request.  sh: 2 + the wavefronts.
template <int RB>
__device__ inline Tile find_tile(const Adapters& a, int64_t w, int* sh) {
  constexpr int kRows = 16 * RB, NW = kWaves * RB;
  if (!a.starts) return {w, w < a.N ? 1 : 0, w < a.N ? a.ids[w] : -1};
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int64_t before = 0;
  if (tid == 0) sh[NW + 1] = -1;
  for (int i0 = 0; i0 < a.B + 2; i0 += RB * kThreads) {
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
    for (int k = 0; k < NW; ++k) {
      if (k < wave) at += sh[k];
      all += sh[k];
    }
    if (w >= at && w < at + mine) sh[NW] = (int)(w - at), sh[NW + 1] = i0 + tid;
    before += all;
    __syncthreads();
    if (w < before) break;
  }
  const int i = sh[NW + 1];
  if (i < 0) return {0, 0, -1};
  int64_t r0, r1;
  segment(a, i, r0, r1);
  r0 += (int64_t)sh[NW] * kRows;
  return {r0, (int)min<int64_t>(kRows, r1 - r0), i == 0 || i == a.B + 1 ? -1 : a.ids[i - 1]};
}

// The wavefronts' parts of a (16 RB) x R product, joined, times f: t[16 RB][RT * 16 + 4].
template <int RT, int RB>
__device__ inline void join(const Adapters& a, const f4 (*acc)[RT], float f, float* red, float* t) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int y = 0; y < RB; ++y)
#pragma unroll
    for (int i = 0; i < RT; ++i) *(f4*)(red + (((wave * RB + y) * RT + i) * 64 + lane) * 4) = acc[y][i];
  __syncthreads();
  for (int e = threadIdx.x; e < RB * RT * 256; e += RB * kThreads) {
    const int yi = e >> 8, ln = (e & 255) >> 2, q = e & 3;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves * RB; ++k) s += red[(k * RB * RT * 64) * 4 + e];
    const int r = 16 * (yi % RT) + (ln & 15);
    t[(16 * (yi / RT) + 4 * (ln >> 4) + q) * (RT * 16 + 4) + r] = r < a.R ? s * f : 0.f;
  }
  __syncthreads();
}

// t = f v w^T for the tile's rows of v (width n) and w (R x n): the wavefronts share the contraction, each with
// kBatch blocks of it in flight (a block's latency after the other's, 64 tokens of 1024 -> 4096 took 13.7 us).
template <bool BF, int RT, int RB>
__device__ inline void inner(const Adapters& a, const Tile& T, const void* v, const void* w, int n, float f, float* red, float* t) {
  constexpr int KB = BF ? 32 : 16, VE = BF ? 8 : 4, NW = kWaves * RB, kBatch = RT * RB >= 8 ? 1 : 8 / (RT * RB);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  f4 acc[RB][RT];
  int64_t vrow[RB], wrow[RT];
#pragma unroll
  for (int y = 0; y < RB; ++y) {
    vrow[y] = (T.row + min(16 * y + c, T.rows - 1)) * n;
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[y][i] = f4{0, 0, 0, 0};
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) wrow[i] = (int64_t)min(16 * i + c, a.R - 1) * n;
  for (int k = wave * KB; k < n; k += kBatch * NW * KB) {
    u4 x[kBatch][RB], d[kBatch][RT];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int at = k + b * NW * KB + VE * g;
#pragma unroll
      for (int y = 0; y < RB; ++y) x[b][y] = load16<BF>(v, vrow[y] + at, n - at);
#pragma unroll
      for (int i = 0; i < RT; ++i) d[b][i] = load16<BF>(w, wrow[i] + at, n - at);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int y = 0; y < RB; ++y)
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          if constexpr (BF) {
            acc[y][i] = mma16(x[b][y], d[b][i], acc[y][i]);      // rows x rank
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[y][i] = mma32(value<false>(x[b][y], q), value<false>(d[b][i], q), acc[y][i]);
          }
        }
  }
  join<RT, RB>(a, acc, f, red, t);
}

// Blocks of the contraction that inner_t has in flight.
template <bool BF>
constexpr int turned(int RT) { return RT >= 4 ? 1 : (BF ? 4 : 8) / RT; }

// g = f v w for w (n x R).  fp32: w's values one by one, sixteen neighbours of a row together.  bf16: 32 rows of w and
// sixteen columns go through a KB of the wavefront's LDS, whose transposing reads give the columns their rows, eight neighbours
// of the contraction as the bf16 instruction takes them (8192 rows of
// 768 -> 2048, one value a lane's load: 29.5 us of the rows' kernel, so 23).
template <bool BF, int RT, int RB>
__device__ inline void inner_t(const Adapters& a, const Tile& T, const void* v, const void* w, int n, float f, float* red, float* t) {
  constexpr int KB = BF ? 32 : 16, VE = BF ? 8 : 4, NW = kWaves * RB, kBatch = turned<BF>(RT);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  f4 acc[RB][RT];
  int64_t vrow[RB];
#pragma unroll
  for (int y = 0; y < RB; ++y) {
    vrow[y] = (T.row + min(16 * y + c, T.rows - 1)) * n;
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[y][i] = f4{0, 0, 0, 0};
  }
  for (int k = wave * KB; k < n; k += kBatch * NW * KB) {
    u4 x[kBatch][RB];
    if constexpr (BF) {
      typedef short s4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) char lds;
      typedef __attribute__((address_space(3))) s4 lds4;
      lds* mine = (lds*)(char*)red + wave * (kBatch * RT * 1024);      // (Shared's KB)
      u4 u[kBatch][RT];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int k0 = k + b * NW * KB, at = k0 + VE * g, m = k0 + (lane >> 1);
#pragma unroll
        for (int y = 0; y < RB; ++y) x[b][y] = load16<BF>(v, vrow[y] + at, n - at);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const int r = 16 * i + 8 * (lane & 1);
          u[b][i] = load16<BF>(w, (int64_t)m * a.R + r, m < n ? a.R - r : 0);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int i = 0; i < RT; ++i) *(__attribute__((address_space(3))) u4*)(mine + (b * RT + i) * 1024 + lane * 16) = u[b][i];
      asm volatile("" ::: "memory");
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          lds* q = mine + (b * RT + i) * 1024 + (8 * g + (c >> 2)) * 32 + (c & 3) * 8;
          union { s4 h[2]; u4 u; } o;
          o.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)q);
          o.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(q + 128));
#pragma unroll
          for (int y = 0; y < RB; ++y) acc[y][i] = mma16(x[b][y], o.u, acc[y][i]);
        }
      asm volatile("" ::: "memory");
    } else {
      float u[kBatch][RT][VE];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int at = k + b * NW * KB + VE * g;
#pragma unroll
        for (int y = 0; y < RB; ++y) x[b][y] = load16<BF>(v, vrow[y] + at, n - at);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int q = 0; q < VE; ++q) u[b][i][q] = load1<BF>(w, (int64_t)min(at + q, n - 1) * a.R + min(16 * i + c, a.R - 1));
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int q = 0; q < VE; ++q)
#pragma unroll
          for (int y = 0; y < RB; ++y)
#pragma unroll
            for (int i = 0; i < RT; ++i) acc[y][i] = mma32(value<BF>(x[b][y], q), u[b][i][q], acc[y][i]);
    }
  }
  // (all have read what join writes over)
  __syncthreads();
  join<RT, RB>(a, acc, f, red, t);
}

// Column of a row of y or dx that lane c of block h (of the two that bf16 takes together) stands for: the lane that
// holds rows 4 g .. 4 g + 3 of both results then has eight neighbours, 16 bytes.
template <bool BF>
__device__ inline int column(int c, int h) { return BF ? 8 * (c >> 2) + 4 * h + (c & 3) : c; }

// Rows without an adapter: out = base (zeros without one), NaN where the id is none of the table's.
template <bool BF>
__device__ inline void plain_rows(const Adapters& a, const Tile& T, const void* base, void* out, int n, int part, int parts) {
  if (T.id < 0 && base == out) return;
  for (int64_t i = (int64_t)part * blockDim.x + threadIdx.x; i < (int64_t)T.rows * n; i += (int64_t)parts * blockDim.x) {
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

// KB: of w's rows that inner_t turns, for each wavefront.
template <int RT, int RB, int KB = 0>
struct Shared {
  float red[kWaves * RB * (KB > RB * RT ? KB : RB * RT) * 256];
  float t[16 * RB * (RT * 16 + 4)];
  float g[16 * RB * (RT * 16 + 4)];
  int find[kWaves * RB + 2];
};

// out = base + t w for the tile's rows (width n), kBatch blocks of 16 or (bf16) 32 columns in flight.  factors(m, i, g): w's
// values 16 i + 4 g .. + 3 of the rank at column m.
template <bool BF, int RT, int RB, class F>
__device__ inline void outer(const Adapters& a, const Tile& T, const float* t, const void* base, void* out, int n, int part, int parts,
                             const F& factors) {
  constexpr int H = BF ? 2 : 1, W = 16 * H, NW = kWaves * RB, kBatch = RT >= 4 ? 1 : 4 / RT / H + (RT == 2 && BF);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  f4 tr[RB][RT];
  int64_t row[RB];
#pragma unroll
  for (int y = 0; y < RB; ++y) {
    row[y] = (T.row + min(16 * y + c, T.rows - 1)) * n;
#pragma unroll
    for (int i = 0; i < RT; ++i) tr[y][i] = *(const f4*)(t + (16 * y + c) * (RT * 16 + 4) + 16 * i + 4 * g);
  }
  const int stride = parts * NW * W;
  for (int m = (part * NW + wave) * W; m < n; m += kBatch * stride) {
    f4 w[kBatch][H][RT];
    u4 old[kBatch][RB];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int m0 = m + b * stride, at = m0 + 4 * H * g;
#pragma unroll
      for (int y = 0; y < RB; ++y) old[b][y] = base ? load16<BF>(base, row[y] + at, n - at) : u4{0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < RT; ++i) w[b][h][i] = factors(min(m0 + column<BF>(c, h), n - 1), i, g);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int at = m + b * stride + 4 * H * g;
#pragma unroll
      for (int y = 0; y < RB; ++y) {
        f4 acc[H];
#pragma unroll
        for (int h = 0; h < H; ++h) acc[h] = f4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int h = 0; h < H; ++h) acc[h] = mma32(w[b][h][i][q], tr[y][i][q], acc[h]);      // columns x rows
        if (16 * y + c < T.rows) store16<BF>(out, row[y] + at, n - at, old[b][y], acc);
      }
    }
  }
}

template <bool BF, int RT, int RB>
__global__ __launch_bounds__(RB * kThreads) void adapters_fwd_kernel(Adapters a) {
  __shared__ Shared<RT, RB> sh;
  const Tile T = find_tile<RB>(a, blockIdx.x, sh.find);
  if (T.rows == 0) return;
  if (T.id < 0 || T.id >= a.E) {
    plain_rows<BF>(a, T, a.base, a.y, a.M, blockIdx.y, gridDim.y);
    return;
  }
  const size_t es = BF ? 2 : 4;
  const float f = a.scales ? a.scales[T.id] : 1.f;
  const char* D = (const char*)a.down + (size_t)T.id * a.R * a.K * es;
  const char* U = (const char*)a.up + (size_t)T.id * a.R * a.M * es;
  inner<BF, RT, RB>(a, T, a.x, D, a.K, f, sh.red, sh.t);
  outer<BF, RT, RB>(a, T, sh.t, a.base, a.y, a.M, blockIdx.y, gridDim.y,
                    [&](int m, int i, int g) { return load4<BF>(U, (int64_t)m * a.R + 16 * i + 4 * g, a.R - 16 * i - 4 * g); });
}

// The rows' part of the backward: t and g of each row for the gradients' kernel, and dx.
template <bool BF, int RT, int RB>
__global__ __launch_bounds__(RB * kThreads) void adapters_rows_kernel(Adapters a) {
  __shared__ Shared<RT, RB, BF ? turned<BF>(RT) * RT : 0> sh;
  const Tile T = find_tile<RB>(a, blockIdx.x, sh.find);
  if (T.rows == 0) return;
  if (T.id < 0 || T.id >= a.E) {
    if (a.y) plain_rows<BF>(a, T, a.base, a.y, a.K, 0, 1);
    return;
  }
  const size_t es = BF ? 2 : 4;
  const float f = a.scales ? a.scales[T.id] : 1.f;
  const char* D = (const char*)a.down + (size_t)T.id * a.R * a.K * es;
  const char* U = (const char*)a.up + (size_t)T.id * a.R * a.M * es;
  inner<BF, RT, RB>(a, T, a.x, D, a.K, f, sh.red, sh.t);
  inner_t<BF, RT, RB>(a, T, a.dy, U, a.M, f, sh.red, sh.g);
  float* keep = a.ws + T.row * 2 * (RT * 16);
  for (int e = threadIdx.x; e < T.rows * RT * 16; e += RB * kThreads) {
    const int r = e / (RT * 16), k = e % (RT * 16);
    keep[(int64_t)r * 2 * RT * 16 + k] = sh.t[r * (RT * 16 + 4) + k];
    keep[(int64_t)r * 2 * RT * 16 + RT * 16 + k] = sh.g[r * (RT * 16 + 4) + k];
  }
  if (!a.y) return;
  outer<BF, RT, RB>(a, T, sh.g, a.base, a.y, a.K, 0, 1, [&](int k, int i, int g) {
    f4 d;
#pragma unroll
    for (int q = 0; q < 4; ++q) d[q] = load1<BF>(D, (int64_t)min(16 * i + 4 * g + q, a.R - 1) * a.K + k);
    return d;
  });
}

// The adapters' gradients: 64 columns of x (dD = g^T x) or of dy (dU = dy^T t) of one adapter, over every `splits`-th four
// rows of its.  A lane has four neighbouring columns: column 4 c + q is lane c's of product q.
constexpr int kCols = 64, kParamWaves = 8;
template <bool BF, int RT>
__global__ __launch_bounds__(64 * kParamWaves) void adapters_params_kernel(Adapters a, int kblocks, int splits, float* part) {
  constexpr int kBatch = 8 / RT;
  __shared__ float red[kParamWaves][4][256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  const int e = blockIdx.y, split = blockIdx.z;
  const bool up = (int)blockIdx.x >= kblocks;
  const int n = up ? a.M : a.K, col0 = (up ? blockIdx.x - kblocks : blockIdx.x) * kCols, mine = col0 + 4 * c;
  const void* v = up ? a.dy : a.x;
  const float* tg = a.ws + (up ? 0 : RT * 16);
  f4 acc[RT][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[i][q] = f4{0, 0, 0, 0};
  // The adapter's blocks of four rows, 64 requests at a time (a lane has one's rows) and numbered through them: the
  // wavefronts take turns, kBatch blocks of any requests in flight (request by request, 512 of 16 rows took 105 us).
  const int stride = kParamWaves * splits, turn = split * kParamWaves + wave;
  int64_t seen = 0;
  for (int i0 = 0; i0 < a.B; i0 += 64) {
    int r0 = 0, r1 = 0;
    if (i0 + lane < a.B && a.ids[i0 + lane] == e) {
      int64_t lo = i0 + lane, hi = min<int64_t>(i0 + lane + 1, a.N);
      if (a.starts) segment(a, i0 + lane + 1, lo, hi);
      r0 = (int)lo, r1 = (int)hi;
    }
    const int blocks = (r1 - r0 + 3) / 4;
    int upto = blocks;      // blocks of the requests up to this lane's
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int y = __shfl_up(upto, o, 64);
      if (lane >= o) upto += y;
    }
    const int total = __builtin_amdgcn_readlane(upto, 63);
    for (int b = (int)((turn - seen % stride + stride) % stride); b < total; b += kBatch * stride) {
      f4 x[kBatch];
      float w[kBatch][RT];
#pragma unroll
      for (int t = 0; t < kBatch; ++t) {
        const int at = b + t * stride;
        const int i = min(63, (int)__builtin_ctzll(__ballot(upto > at) | uint64_t(1) << 63));
        const int row = __builtin_amdgcn_readlane(r0, i) + 4 * (at - __builtin_amdgcn_readlane(upto - blocks, i)) + g;
        const bool in = at < total && row < __builtin_amdgcn_readlane(r1, i);
        x[t] = load4<BF>(v, (int64_t)row * n + mine, in ? n - mine : 0);
#pragma unroll
        for (int k = 0; k < RT; ++k) w[t][k] = in ? tg[(int64_t)row * 2 * RT * 16 + 16 * k + c] : 0.f;
      }
#pragma unroll
      for (int t = 0; t < kBatch; ++t)
#pragma unroll
        for (int k = 0; k < RT; ++k)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[k][q] = mma32(w[t][k], x[t][q], acc[k][q]);      // rank x columns
    }
    seen += total;
  }
  float* out = splits > 1 ? part + (int64_t)split * a.E * a.R * (a.K + a.M) : nullptr;
#pragma unroll
  for (int k = 0; k < RT; ++k) {
#pragma unroll
    for (int q = 0; q < 4; ++q) *(f4*)&red[wave][q][lane * 4] = acc[k][q];
    __syncthreads();
    for (int x = threadIdx.x; x < 1024; x += 64 * kParamWaves) {
      // dD's neighbours along the columns, dU's along the rank
      const int rr = up ? x % 16 : x / kCols, cc = up ? x / 16 : x % kCols;
      const int r = 16 * k + rr, col = col0 + cc, ln = (rr >> 2) * 16 + cc / 4;
      if (r >= a.R || col >= n) continue;
      float s = 0.f;
#pragma unroll
      for (int t = 0; t < kParamWaves; ++t) s += red[t][cc % 4][ln * 4 + (rr & 3)];
      if (up) (out ? out + (int64_t)a.E * a.R * a.K : a.dup)[((int64_t)e * a.M + col) * a.R + r] = s;
      else (out ? out : a.ddown)[((int64_t)e * a.R + r) * a.K + col] = s;
    }
    __syncthreads();
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

// Tiles of 32 rows where two of sixteen would be on every CU anyway, in bf16 (8192 x (768 -> 2048): rank 16 23.3 -> 21.9 us,
// rank 64 47 -> 41; else two workgroups' phases overlap better than one's: fp32 1024 -> 1024 of rank 24 39 us against 42,
// the rows' backward of rank 16 23.5 us against 28).
bool wide(const Adapters& a, bool backward) { return a.bf16 && a.N >= 8192 && a.starts && a.R <= 64 && (a.R > 16 || !backward); }
int64_t tiles_of(const Adapters& a, int RB) { return a.starts ? ceil_div(a.N, 16 * RB) + a.B + 1 : a.N; }

// Workgroups that share an adapter's rows, so that every CU has one.
int splits_of(const Adapters& a) {
  const int64_t groups = (ceil_div(a.K, kCols) + ceil_div(a.M, kCols)) * a.E;
  return (int)std::max<int64_t>(1, std::min({256 / groups, ceil_div(a.N, 256), int64_t(16)}));
}

template <bool BF, int RT, int RB>
hipError_t fwd(const Adapters& a, hipStream_t s) {
  const int64_t tiles = tiles_of(a, RB);
  // few tiles: several workgroups share a tile's columns, each with the inner product to itself
  const int gy = (int)std::max<int64_t>(1, std::min(256 / tiles, ceil_div(a.M, kWaves * 16)));
  hipLaunchKernelGGL((adapters_fwd_kernel<BF, RT, RB>), dim3((unsigned)tiles, (unsigned)gy), dim3(RB * kThreads), 0, s, a);
  return hipGetLastError();
}

template <bool BF, int RT, int RB>
hipError_t bwd(const Adapters& a, hipStream_t s) {
  if (a.N) hipLaunchKernelGGL((adapters_rows_kernel<BF, RT, RB>), dim3((unsigned)tiles_of(a, RB)), dim3(RB * kThreads), 0, s, a);
  const int splits = splits_of(a), kb = (int)ceil_div(a.K, kCols), mb = (int)ceil_div(a.M, kCols);
  float* part = (float*)((char*)a.ws + up256(sizeof(float) * (size_t)a.N * 2 * RT * 16));
  hipLaunchKernelGGL((adapters_params_kernel<BF, RT>), dim3((unsigned)(kb + mb), (unsigned)a.E, (unsigned)splits), dim3(64 * kParamWaves), 0, s, a,
                     kb, splits, part);
  if (splits > 1) {
    const int64_t n = (int64_t)a.E * a.R * (a.K + a.M);
    hipLaunchKernelGGL(adapters_join_kernel, dim3((unsigned)std::min<int64_t>(2048, ceil_div(n, kThreads))), dim3(kThreads), 0, s, a, splits, part);
  }
  return hipGetLastError();
}

template <int RT>
hipError_t pick(const Adapters& a, bool backward, hipStream_t s) {
  if (!a.bf16) return backward ? bwd<false, RT, 1>(a, s) : fwd<false, RT, 1>(a, s);
  if constexpr (RT <= 4) {      // (more would take the registers and LDS of too many)
    if (wide(a, false) && !backward) return fwd<true, RT, 2>(a, s);
  }
  if constexpr (RT == 2 || RT == 4) {
    if (wide(a, true) && backward) return bwd<true, RT, 2>(a, s);
  }
  return backward ? bwd<true, RT, 1>(a, s) : fwd<true, RT, 1>(a, s);
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
