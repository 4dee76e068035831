// Cross-entropy of a large vocabulary from the hidden states, without the logits in memory:
//   z = h W^T,  nll_n = log sum_v exp(z_nv) - z_n[label_n],  loss = sum_n w_n nll_n
//   dz_nv = w_n (softmax(z_n)_v - [v = label_n]),  dh = g dz W,  dW = g dz^T h
// The forward is one product whose epilogue keeps, for each row and tile of the vocabulary, the maximum and
// the sum of exponentials.  The backward takes the vocabulary in pieces: the logits of a piece again, their
// gradient to 16 bits, and its two products.
//
// bf16 inputs go into the products as they are (sums in fp32), and dz is rounded to bf16 once.  fp32 inputs, and
// their dz, are two fp16 planes each (tile_product.h).
#include <algorithm>
#include <cmath>

#include "row_tile.h"
#include "tile_product.h"

namespace kron {

// Rows in use, and what the scales of fp32 values come from.
struct VocabScales {
  uint32_t top_h, top_w, top_dz;      // bits of the largest finite |value|
  int count;              // rows in use
};

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
__device__ inline float expo(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// ------------------------------------------------------------------------------ rows in use and scales

__device__ inline float scale_up(uint32_t top) {
  // top 2^s in [2^14, 2^15), s within what fp32 has a normal inverse for
  const int e = (int)(top >> 23);
  const int s = top == 0 ? 0 : min(126, max(-126, 14 - (e - 127)));
  return __uint_as_float((uint32_t)(s + 127) << 23);
}
__device__ inline float scale_down(uint32_t top) { return 1.f / scale_up(top); }

// Rows of nonzero weight in order (idx), their places (pos, -1: not in use), and what the outputs of the others are.
__global__ __launch_bounds__(1024) void vocab_rows_kernel(VocabCE a) {
  __shared__ int wsum[16];
  __shared__ uint32_t wtop[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t top = 0;
  int base = 0;
  for (int64_t n0 = 0; n0 < a.N; n0 += 1024) {
    const int64_t n = n0 + tid;
    const float w = n < a.N ? (a.weights ? a.weights[n] : a.mean) : 0.f;
    const bool in = w != 0.f;      // (a NaN is in use)
    if (in && isfinite(w)) top = max(top, __float_as_uint(w) & 0x7fffffffu);
    const uint64_t m = __ballot(in);
    if (lane == 0) wsum[wave] = __popcll(m);
    __syncthreads();
    int before = base, all = 0;
    for (int i = 0; i < 16; ++i) {
      if (i < wave) before += wsum[i];
      all += wsum[i];
    }
    const int at = before + __popcll(m & ((uint64_t(1) << lane) - 1));
    if (n < a.N && a.idx) {
      a.pos[n] = in ? at : -1;
      if (in) a.idx[at] = (int)n;
      if (!in && a.nll) a.nll[n] = 0.f, a.stats[2 * n] = 0.f, a.stats[2 * n + 1] = 0.f;
    }
    base += all;
    __syncthreads();
  }
  for (int o = 32; o >= 1; o /= 2) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
  if (lane == 0) wtop[wave] = top;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < 16; ++i) top = max(top, wtop[i]);
    a.sc->top_dz = top;
    a.sc->top_h = a.sc->top_w = 0;
    a.sc->count = base;
  }
}

__device__ inline int vocab_count(const VocabCE& a) { return a.sc ? a.sc->count : (int)a.N; }

// The largest finite magnitude of h's rows in use (block.y 0) and of W (1).
__global__ __launch_bounds__(256) void vocab_top_kernel(VocabCE a) {
  const bool w = blockIdx.y == 1;
  const int rows = w ? a.V : vocab_count(a);
  const float* src = (const float*)(w ? a.W : a.h);
  uint32_t top = 0;
  for (int r = blockIdx.x; r < rows; r += gridDim.x) {
    const float* row = src + (int64_t)(!w && a.idx ? a.idx[r] : r) * a.K;
    for (int k = threadIdx.x; k < a.K; k += 256) {
      const uint32_t v = __float_as_uint(row[k]) & 0x7fffffffu;
      if (v < 0x7f800000u) top = max(top, v);
    }
  }
  for (int o = 32; o >= 1; o /= 2) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
  if ((threadIdx.x & 63) == 0 && top) atomicMax(w ? &a.sc->top_w : &a.sc->top_h, top);
}

// Rows as operands: gathered (h), padded with zeros to Kp, fp32 split into its planes.
template <bool BF>
__global__ __launch_bounds__(256) void vocab_pack_kernel(VocabCE a, int which) {
  const bool w = which == 1;
  const int rows = w ? a.V : vocab_count(a);
  const int per = a.Kp / 8;
  uint16_t* dst = w ? a.wp : a.hp;
  const int64_t plane = w ? a.wplane : a.hplane;
  float up = 1.f;
  if constexpr (!BF) up = scale_up(w ? a.sc->top_w : a.sc->top_h);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)rows * per; i += (int64_t)gridDim.x * 256) {
    const int r = (int)(i / per), k = (int)(i - (int64_t)r * per) * 8;
    const int64_t from = (int64_t)(!w && a.idx ? a.idx[r] : r) * a.K + k;
    const int64_t to = (int64_t)r * a.Kp + k;
    if constexpr (BF) {
      const uint16_t* s = (const uint16_t*)(w ? a.W : a.h) + from;
      u4 o = {0, 0, 0, 0};
      if (k + 8 <= a.K && (a.K & 7) == 0)
        o = *(const u4*)s;
      else
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (k + e < a.K) o[e / 2] |= (uint32_t)s[e] << (16 * (e & 1));
      *(u4*)(dst + to) = o;
    } else {
      const float* s = (const float*)(w ? a.W : a.h) + from;
      float v[8];
      if (k + 8 <= a.K && (a.K & 3) == 0) {
        const f4 x = *(const f4*)s, y = *(const f4*)(s + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = x[e], v[4 + e] = y[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = k + e < a.K ? s[e] : 0.f;
      }
      h8 hi, lo;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = v[e] * up;
        hi[e] = (_Float16)x;
        lo[e] = (_Float16)((x - (float)hi[e]) * kLo);
      }
      *(h8*)(dst + to) = hi;
      *(h8*)(dst + plane + to) = lo;
    }
  }
}

__device__ inline Operand h_operand(const VocabCE& a, int count) { return {a.hp, a.Kp, a.hplane, count, a.Kp}; }
__device__ inline Operand w_operand(const VocabCE& a) { return {a.wp, a.Kp, a.wplane, a.V, a.Kp}; }

// ------------------------------------------------------------------------------ forward
// Tiles of the vocabulary (m) x rows (n): each lane holds four neighbouring tokens of one row.
template <class P, bool BF>
__global__ __launch_bounds__(P::kThreads) void vocab_fwd_kernel(VocabCE a, int tm, int tn) {
  extern __shared__ char smem[];
  int mt, nt;
  tile_of(blockIdx.x, gridDim.x, tm, tn, mt, nt);
  const int count = vocab_count(a), m0 = mt * P::BM, n0 = nt * P::BN;
  if (n0 >= count) return;
  P p;
  p.run(w_operand(a), h_operand(a, count), m0, n0, 0, a.Kp, (lds_t*)smem);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  const int wm = wave % P::WM, wn = wave / P::WM;
  const float down = BF ? 1.f : scale_down(a.sc->top_h), down2 = BF ? 1.f : scale_down(a.sc->top_w);
  float* red = (float*)smem;      // (the product ended with a barrier)
#pragma unroll
  for (int j = 0; j < P::TN; ++j) {
    const int nl = wn * P::TN * 16 + 16 * j + c, n = n0 + nl;
    const int lab = n < count ? (int)min<int64_t>(max<int64_t>(a.labels[a.idx ? a.idx[n] : n], -1), a.V) : -1;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < P::TM; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int v = m0 + wm * P::TM * 16 + 16 * i + 4 * g + e;
        float z = p.acc[i][j][e];
        if constexpr (!BF) z = z * down * down2;
        if (v >= a.V) z = -INFINITY;
        if (v == lab && v < a.V) a.zlab[n] = z;
        p.acc[i][j][e] = z;
        top = z > top || z != z ? z : top;      // (a NaN stays)
      }
    float sum = 0.f;
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int i = 0; i < P::TM; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += expo(p.acc[i][j][e] - ref);
#pragma unroll
    for (int o = 16; o <= 32; o *= 2) {
      const float t2 = __shfl_xor(top, o, 64), s2 = __shfl_xor(sum, o, 64);
      const float t = t2 > top || t2 != t2 ? t2 : top, r = t == -INFINITY ? 0.f : t;
      sum = sum * expo(top - r) + s2 * expo(t2 - r);
      top = t;
    }
    if (g == 0) red[(wm * P::BN + nl) * 2] = top, red[(wm * P::BN + nl) * 2 + 1] = sum;
  }
  __syncthreads();
  for (int nl = threadIdx.x; nl < P::BN; nl += P::kThreads) {
    if (n0 + nl >= count) break;
    float t = red[nl * 2];
#pragma unroll
    for (int w = 1; w < P::WM; ++w) {
      const float t2 = red[(w * P::BN + nl) * 2];
      t = t2 > t || t2 != t2 ? t2 : t;
    }
    const float r = t == -INFINITY ? 0.f : t;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < P::WM; ++w) s += red[(w * P::BN + nl) * 2 + 1] * expo(red[(w * P::BN + nl) * 2] - r);
    ((float2*)a.part)[(int64_t)mt * a.N + n0 + nl] = float2{t, s};
  }
}

// A row's statistics from its tiles': 32 rows by 8 slices of the tiles.
__global__ __launch_bounds__(256) void vocab_join_kernel(VocabCE a, int tiles) {
  __shared__ float2 red[8][32];
  const int count = vocab_count(a), r = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int64_t i = (int64_t)blockIdx.x * 32 + r;
  const float2* part = (const float2*)a.part;
  float t = -INFINITY, s = 0.f;
  if (i < count)
    for (int m = sl; m < tiles; m += 8) {
      const float2 v = part[(int64_t)m * a.N + i];
      const float n = v.x > t || v.x != v.x ? v.x : t, ref = n == -INFINITY ? 0.f : n;
      s = s * expo(t - ref) + v.y * expo(v.x - ref);
      t = n;
    }
  red[sl][r] = float2{t, s};
  __syncthreads();
  if (sl != 0 || i >= count) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) {
    const float2 v = red[k][r];
    const float n = v.x > t || v.x != v.x ? v.x : t, ref = n == -INFINITY ? 0.f : n;
    s = s * expo(t - ref) + v.y * expo(v.x - ref);
    t = n;
  }
  const int64_t row = a.idx ? a.idx[i] : i;
  const int64_t lab = a.labels[row];
  const float nll = lab >= 0 && lab < a.V ? (t - a.zlab[i]) + logf(s) : NAN;
  a.nll[row] = nll;
  a.stats[2 * row] = t;
  a.stats[2 * row + 1] = lab >= 0 && lab < a.V ? 1.f / s : NAN;
}

// loss = sum_n w_n nll_n in 64 bits, in a fixed order.
__global__ __launch_bounds__(1024) void vocab_loss_kernel(VocabCE a) {
  __shared__ double red[16];
  double s = 0;
  for (int64_t n = threadIdx.x; n < a.N; n += 1024) {
    const float w = a.weights ? a.weights[n] : a.mean;
    if (w != 0.f) s += (double)w * (double)a.nll[n];
  }
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 16; ++i) s += red[i];
    a.loss[0] = (float)s;
  }
}

// ------------------------------------------------------------------------------ backward
// The gradient of the logits of one piece of the vocabulary, [rows][vc] in 16 bits (without the factor g).
template <class P, bool BF>
__global__ __launch_bounds__(P::kThreads) void vocab_dz_kernel(VocabCE a, int v0, int vc, int tm, int tn) {
  extern __shared__ char smem[];
  int mt, nt;
  tile_of(blockIdx.x, gridDim.x, tm, tn, mt, nt);
  const int count = vocab_count(a), m0 = mt * P::BM, n0 = nt * P::BN;
  if (n0 >= count) return;
  P p;
  p.run(w_operand(a), h_operand(a, count), v0 + m0, n0, 0, a.Kp, (lds_t*)smem);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  const int wm = wave % P::WM, wn = wave / P::WM;
  const float down = BF ? 1.f : scale_down(a.sc->top_h), down2 = BF ? 1.f : scale_down(a.sc->top_w);
  const float up = BF ? 1.f : scale_up(a.sc->top_dz);
  const int padded = (count + kBK - 1) / kBK * kBK;      // rows that the contraction over them reads
#pragma unroll
  for (int j = 0; j < P::TN; ++j) {
    const int n = n0 + wn * P::TN * 16 + 16 * j + c;
    if (n >= padded) continue;
    int lab = -1;
    float top = 0.f, inv = 0.f, w = 0.f;
    if (n < count) {
      const int64_t row = a.idx ? a.idx[n] : n;
      lab = (int)min<int64_t>(max<int64_t>(a.labels[row], -1), a.V);
      top = a.stats_in[2 * row], inv = a.stats_in[2 * row + 1];
      w = (a.weights ? a.weights[row] : a.mean) * up;
    }
#pragma unroll
    for (int i = 0; i < P::TM; ++i) {
      const int ml = m0 + wm * P::TM * 16 + 16 * i + 4 * g;
      float d[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int v = v0 + ml + e;
        float z = p.acc[i][j][e];
        if constexpr (!BF) z = z * down * down2;
        const float q = expo(z - top) * inv;
        d[e] = v >= a.V || n >= count ? 0.f : (v == lab ? q - 1.f : q) * w;
      }
      uint16_t* out = a.dz + (int64_t)n * vc + ml;
      if constexpr (BF) {
        *(uint2*)out = uint2{bf16_pair(d[0], d[1]), bf16_pair(d[2], d[3])};
      } else {
        typedef _Float16 h4 __attribute__((ext_vector_type(4)));
        h4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          hi[e] = (_Float16)d[e];
          lo[e] = (_Float16)((d[e] - (float)hi[e]) * kLo);
        }
        *(h4*)out = hi;
        *(h4*)(out + a.dzplane) = lo;
      }
    }
  }
}

// part[s] (+)= dz W over the s-th part of the piece: rows (n) x K (m).
template <class P, bool BF>
__global__ __launch_bounds__(P::kThreads) void vocab_dh_kernel(VocabCE a, int v0, int vc, int tm, int tn, int len, int add) {
  extern __shared__ char smem[];
  int mt, nt;
  tile_of(blockIdx.x, gridDim.x, tm, tn, mt, nt);
  const int count = vocab_count(a), m0 = mt * P::BM, n0 = nt * P::BN;
  if (n0 >= count) return;
  const int k0 = blockIdx.y * len, k1 = min(vc, k0 + len);
  Operand W = w_operand(a);
  W.p += (int64_t)v0 * a.Kp;
  W.rows = a.V - v0;
  const Operand dz = {a.dz, vc, a.dzplane, count, vc};
  P p;
  p.run(W, dz, m0, n0, k0, k1, (lds_t*)smem);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  float* out = a.dhpart + (int64_t)blockIdx.y * a.N * a.Kp;
#pragma unroll
  for (int j = 0; j < P::TN; ++j) {
    const int n = n0 + (wave / P::WM) * P::TN * 16 + 16 * j + c;
    if (n >= count) continue;
#pragma unroll
    for (int i = 0; i < P::TM; ++i) {
      const int m = m0 + (wave % P::WM) * P::TM * 16 + 16 * i + 4 * g;
      if (m >= a.Kp) continue;
      f4* q = (f4*)(out + (int64_t)n * a.Kp + m);
      *q = add ? *q + p.acc[i][j] : p.acc[i][j];
    }
  }
}

template <bool BF>
__global__ __launch_bounds__(256) void vocab_dh_join_kernel(VocabCE a, int splits) {
  float f = a.gout[0], f2 = 1.f;
  if constexpr (!BF) f *= scale_down(a.sc->top_dz), f2 = scale_down(a.sc->top_w);
  const int per = a.Kp / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.N * per; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per;
    const int k = (int)(i - row * per) * 4;
    if (k >= a.K) continue;
    const int64_t at = a.idx ? a.pos[row] : row;
    f4 s = {0, 0, 0, 0};
    if (at >= 0) {
      for (int t = 0; t < splits; ++t) s += *(const f4*)(a.dhpart + ((int64_t)t * a.N + at) * a.Kp + k);
      s = s * f2 * f;
    }
    if constexpr (BF) {
      uint16_t* o = (uint16_t*)a.dh + row * a.K + k;
      if ((a.K & 3) == 0)
        *(uint2*)o = uint2{bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3])};
      else
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (k + e < a.K) o[e] = (uint16_t)bf16_rne(s[e]);
    } else {
      float* o = (float*)a.dh + row * a.K + k;
      if ((a.K & 3) == 0)
        *(f4*)o = s;
      else
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (k + e < a.K) o[e] = s[e];
    }
  }
}

// dW of a piece: K (m) x vocabulary (n), the contraction over the rows.
template <class P, bool BF>
__global__ __launch_bounds__(P::kThreads) void vocab_dw_kernel(VocabCE a, int v0, int vc, int tm, int tn) {
  extern __shared__ char smem[];
  int mt, nt;
  tile_of(blockIdx.x, gridDim.x, tm, tn, mt, nt);
  const int count = vocab_count(a), m0 = mt * P::BM, n0 = nt * P::BN;
  const int padded = (count + kBK - 1) / kBK * kBK;
  const Operand dz = {a.dz, vc, a.dzplane, padded, vc};
  P p;
  p.run(h_operand(a, count), dz, m0, n0, 0, count, (lds_t*)smem);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  float f = a.gout[0], f2 = 1.f;
  if constexpr (!BF) f *= scale_down(a.sc->top_dz), f2 = scale_down(a.sc->top_h);
#pragma unroll
  for (int j = 0; j < P::TN; ++j) {
    const int v = v0 + n0 + (wave / P::WM) * P::TN * 16 + 16 * j + c;
    if (v >= a.V) continue;
#pragma unroll
    for (int i = 0; i < P::TM; ++i) {
      const int k = m0 + (wave % P::WM) * P::TM * 16 + 16 * i + 4 * g;
      if (k >= a.K) continue;
      const f4 s = p.acc[i][j] * f2 * f;
      if constexpr (BF) {
        uint16_t* o = (uint16_t*)a.dW + (int64_t)v * a.K + k;
        if ((a.K & 3) == 0)
          *(uint2*)o = uint2{bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3])};
        else
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (k + e < a.K) o[e] = (uint16_t)bf16_rne(s[e]);
      } else {
        float* o = (float*)a.dW + (int64_t)v * a.K + k;
        if ((a.K & 3) == 0)
          *(f4*)o = s;
        else
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (k + e < a.K) o[e] = s[e];
      }
    }
  }
}

// ------------------------------------------------------------------------------ host
template <bool BF, Side SA, Side SB>
using Big = Product<2, 4, 8, 4, SA, SB, BF, BF ? 1 : 2>;
template <bool BF, Side SA, Side SB>
using Few = Product<4, 1, 4, 4, SA, SB, BF, BF ? 1 : 2>;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Rows and width of a product with few rows: a tile of 64.
bool few(int64_t N) { return N <= 64; }

struct VocabPlan {
  int Kp;
  bool rows, copy_h, copy_w;      // rows in use are listed; operands that are copies
  int tiles;                      // of the vocabulary, 256 wide
  int piece, pieces, splits;      // backward
  size_t sc, idx, pos, hp, wp, part, zlab, dz, dhpart, bytes;
};

VocabPlan plan_of(int64_t N, int K, int V, bool bf, bool weights, bool backward) {
  VocabPlan p{};
  p.Kp = (int)ceil_div(K, kBK) * kBK;
  p.rows = weights;
  p.copy_h = !bf || weights || K != p.Kp;
  p.copy_w = !bf || K != p.Kp;
  p.tiles = (int)ceil_div(V, 256);
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t r = at; at += up256(bytes); return r; };
  const int planes = bf ? 1 : 2;
  const int64_t rows = ceil_div(std::max<int64_t>(N, 1), kBK) * kBK;
  p.sc = take(sizeof(VocabScales));
  p.idx = take(p.rows ? 4 * (size_t)N : 0);
  p.pos = take(p.rows ? 4 * (size_t)N : 0);
  p.hp = take(p.copy_h ? 2 * (size_t)planes * N * p.Kp : 0);
  p.wp = take(p.copy_w ? 2 * (size_t)planes * V * p.Kp : 0);
  if (!backward) {
    p.part = take(8 * (size_t)p.tiles * N);
    p.zlab = take(4 * (size_t)N);
  } else {
    // dz of a piece takes at most about 512 MB
    const int64_t most = std::max<int64_t>(1, (int64_t(512) << 20) / (rows * 256 * 2 * planes));
    p.pieces = (int)ceil_div(p.tiles, most);
    p.piece = (int)ceil_div(p.tiles, p.pieces) * 256;
    p.pieces = (int)ceil_div(V, p.piece);
    p.dz = take(2 * (size_t)planes * rows * p.piece);
    const int64_t t = ceil_div(p.Kp, 256) * ceil_div(std::max<int64_t>(N, 1), few(N) ? 64 : 256);
    p.splits = (int)std::min<int64_t>(std::max<int64_t>(1, 512 / t), std::max(1, p.piece / 512));
    p.dhpart = take(4 * (size_t)p.splits * N * p.Kp);
  }
  p.bytes = at;
  return p;
}

VocabCE bind(const VocabCE& k, const VocabPlan& p, char* ws, bool bf) {
  VocabCE a = k;
  a.Kp = p.Kp;
  a.sc = p.rows || !bf ? (VocabScales*)(ws + p.sc) : nullptr;
  a.idx = p.rows ? (int*)(ws + p.idx) : nullptr;
  a.pos = (int*)(ws + p.pos);
  a.hp = p.copy_h ? (uint16_t*)(ws + p.hp) : (uint16_t*)k.h;
  a.wp = p.copy_w ? (uint16_t*)(ws + p.wp) : (uint16_t*)k.W;
  a.hplane = k.N * p.Kp;
  a.wplane = (int64_t)k.V * p.Kp;
  a.part = (float*)(ws + p.part);
  a.zlab = (float*)(ws + p.zlab);
  a.dz = (uint16_t*)(ws + p.dz);
  a.dzplane = ceil_div(std::max<int64_t>(k.N, 1), kBK) * kBK * (int64_t)p.piece;
  a.dhpart = (float*)(ws + p.dhpart);
  return a;
}

template <class P, auto kernel, class... A>
hipError_t go(dim3 grid, hipStream_t s, A... args) {
  const hipError_t e = allow_lds<kernel>();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, grid, dim3(P::kThreads), P::kLdsBytes, s, args...);
  return hipGetLastError();
}

template <bool BF>
hipError_t prepare(const VocabCE& a, const VocabPlan& p, hipStream_t s) {
  if (p.rows || !BF) hipLaunchKernelGGL(vocab_rows_kernel, dim3(1), dim3(1024), 0, s, a);
  if (!BF) hipLaunchKernelGGL(vocab_top_kernel, dim3(1024, 2), dim3(256), 0, s, a);
  const int per = p.Kp / 8;
  auto blocks = [&](int64_t rows) { return dim3((unsigned)std::min<int64_t>(4096, std::max<int64_t>(1, ceil_div(rows * per, 256)))); };
  if (p.copy_h && a.N) hipLaunchKernelGGL((vocab_pack_kernel<BF>), blocks(a.N), dim3(256), 0, s, a, 0);
  if (p.copy_w) hipLaunchKernelGGL((vocab_pack_kernel<BF>), blocks(a.V), dim3(256), 0, s, a, 1);
  return hipGetLastError();
}

template <bool BF>
hipError_t run_fwd(const VocabCE& a, const VocabPlan& p, hipStream_t s) {
  hipError_t e = prepare<BF>(a, p, s);
  if (e != hipSuccess) return e;
  if (a.N) {
    const int tn = (int)ceil_div(a.N, few(a.N) ? 64 : 256);
    typedef Few<BF, ROW, ROW> PF;
    typedef Big<BF, ROW, ROW> PB;
    const dim3 grid((unsigned)(p.tiles * tn));
    e = few(a.N) ? go<PF, vocab_fwd_kernel<PF, BF>>(grid, s, a, p.tiles, tn) : go<PB, vocab_fwd_kernel<PB, BF>>(grid, s, a, p.tiles, tn);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(vocab_join_kernel, dim3((unsigned)ceil_div(a.N, 32)), dim3(256), 0, s, a, p.tiles);
  }
  hipLaunchKernelGGL(vocab_loss_kernel, dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}

template <bool BF>
hipError_t run_bwd(const VocabCE& a, const VocabPlan& p, hipStream_t s) {
  hipError_t e = prepare<BF>(a, p, s);
  if (e != hipSuccess) return e;
  const bool fw = few(a.N);
  const int tn = (int)ceil_div(a.N, fw ? 64 : 256), tk = (int)ceil_div(p.Kp, 256);
  for (int i = 0; i < p.pieces; ++i) {
    const int v0 = i * p.piece, vc = std::min(p.piece, (int)ceil_div(a.V - v0, 256) * 256), tm = vc / 256;
    if (a.N) {
      typedef Few<BF, ROW, ROW> PF;
      typedef Big<BF, ROW, ROW> PB;
      const dim3 grid((unsigned)(tm * tn));
      e = fw ? go<PF, vocab_dz_kernel<PF, BF>>(grid, s, a, v0, vc, tm, tn) : go<PB, vocab_dz_kernel<PB, BF>>(grid, s, a, v0, vc, tm, tn);
      if (e != hipSuccess) return e;
    }
    if (a.dh && a.N) {
      typedef Few<BF, COL, ROW> PF;
      typedef Big<BF, COL, ROW> PB;
      const int len = (int)ceil_div(ceil_div(vc, p.splits), kBK) * kBK;
      const dim3 grid((unsigned)(tk * tn), (unsigned)p.splits);
      e = fw ? go<PF, vocab_dh_kernel<PF, BF>>(grid, s, a, v0, vc, tk, tn, len, (int)(i > 0))
             : go<PB, vocab_dh_kernel<PB, BF>>(grid, s, a, v0, vc, tk, tn, len, (int)(i > 0));
      if (e != hipSuccess) return e;
    }
    if (a.dW) {
      typedef Big<BF, COL, COL> PB;
      e = go<PB, vocab_dw_kernel<PB, BF>>(dim3((unsigned)(tk * tm)), s, a, v0, vc, tk, tm);
      if (e != hipSuccess) return e;
    }
  }
  if (a.dh && a.N)
    hipLaunchKernelGGL((vocab_dh_join_kernel<BF>), dim3((unsigned)std::min<int64_t>(8192, ceil_div(a.N * (p.Kp / 4), 256))), dim3(256), 0, s, a,
                       p.splits);
  return hipGetLastError();
}

}  // namespace

size_t vocab_ce_workspace(int64_t N, int K, int V, bool bf, bool weights, bool backward) {
  return plan_of(N, K, V, bf, weights, backward).bytes;
}

hipError_t launch_vocab_ce(const VocabCE& k, bool bf, bool backward, void* ws, hipStream_t s) {
  const VocabPlan p = plan_of(k.N, k.K, k.V, bf, k.weights != nullptr, backward);
  const VocabCE a = bind(k, p, (char*)ws, bf);
  if (backward) return bf ? run_bwd<true>(a, p, s) : run_bwd<false>(a, p, s);
  return bf ? run_fwd<true>(a, p, s) : run_fwd<false>(a, p, s);
}

}  // namespace kron
