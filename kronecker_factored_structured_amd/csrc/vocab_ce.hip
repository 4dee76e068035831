// Cross-entropy of a large vocabulary from the hidden states, without the logits in memory:
//   z = h W^T,  nll_n = log sum_v exp(z_nv) - z_n[label_n],  loss = sum_n w_n nll_n
//   dz_nv = w_n (softmax(z_n)_v - [v = label_n]),  dh = g dz W,  dW = g dz^T h
// The forward is one product whose epilogue keeps, for each row and tile of the vocabulary, the maximum and
// the sum of exponentials.  The backward takes the vocabulary in pieces: the logits of a piece again, their
// gradient to 16 bits, and its two products.
//
// What bounds it: the products, and under them the clock (2.0 GHz of 2.4 by the matrix cores' power).  8192 x 768 x 50257
// bf16: forward 622 us, 1,015 TFLOP/s; with the backward 2.6 ms, 2,530 GFLOP with the recomputed logits at 970.  Few rows
// are bound by the reading of W: 37 x 768 x 50257 bf16 18 us, 4.2 TB/s.
//
// bf16 inputs go into the products as they are (sums in fp32), and dz is rounded to bf16 once.  fp32 inputs, and
// their softmax minus the label's indicator, are two fp16 parts each (tile_product.h): the rows' weights, which may
// lie far apart, then stand beside h in dW and beside the sums in dh.
#include <algorithm>
#include <cmath>

#include "row_tile.h"
#include "tile_product.h"

namespace kron {

// Rows in use, and what the scales of fp32 values come from.
struct VocabScales {
  uint32_t top_h, top_w, top_weight;      // bits of the largest finite |value|
  int count;              // rows in use
};

namespace {

// Exponentials are of the rounded log2(e): 2^(z kLog2e - t), one two-term product each, with a row's t in that scale.  It
// stretches the logits by 2^-26 of themselves and is exact otherwise, as a difference of rounded products would not be.
constexpr float kLog2e = 1.44269504088896340736f;
__device__ inline float expo2(float x) { return __builtin_amdgcn_exp2f(x); }
// Maximum and sum (of 2^(.. - maximum)) of two parts of a row.
__device__ inline float2 joined(float2 a, float2 b) {
  const float t = fmaxf(a.x, b.x), r = t == -INFINITY ? 0.f : t;
  return float2{t, a.y * expo2(a.x - r) + b.y * expo2(b.x - r)};
}

// ------------------------------------------------------------------------------ rows in use and scales

__device__ inline float scale_up(uint32_t top) {
  // top 2^s in [2^14, 2^15), s within what fp32 has a normal inverse for
  const int e = (int)(top >> 23);
  const int s = top == 0 ? 0 : min(126, max(-126, 14 - (e - 127)));
  return __uint_as_float((uint32_t)(s + 127) << 23);
}
__device__ inline float scale_down(uint32_t top) { return 1.f / scale_up(top); }
// What a product of both tensors' parts is times (a factor beyond fp32's range: its end, which takes them there as well).
__device__ inline float scale_down(uint32_t a, uint32_t b) {
  const int up = (int)(__float_as_uint(scale_up(a)) >> 23) + (int)(__float_as_uint(scale_up(b)) >> 23) - 254;
  return __uint_as_float((uint32_t)(min(127, max(-126, -up)) + 127) << 23);
}

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
    a.sc->top_weight = top;
    a.sc->top_h = a.sc->top_w = 0;
    a.sc->count = base;
  }
}

__device__ inline int vocab_count(const VocabCE& a) { return a.sc ? a.sc->count : (int)a.N; }

// The largest finite magnitude of h's rows in use (block.y 0) and of W (1): a wavefront has four rows at a time.
__global__ __launch_bounds__(1024) void vocab_top_kernel(VocabCE a) {
  const bool w = blockIdx.y == 1;
  const int rows = w ? a.V : vocab_count(a), waves = gridDim.x * 16, lane = threadIdx.x & 63;
  const float* src = (const float*)(w ? a.W : a.h);
  uint32_t top = 0;
  for (int r0 = blockIdx.x * 16 + (threadIdx.x >> 6); r0 < rows; r0 += 4 * waves) {
    const char* p[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = min(r0 + q * waves, rows - 1);
      p[q] = (const char*)(src + (int64_t)(!w && a.idx ? a.idx[r] : r) * a.K);
    }
    for (int k = lane * 4; k < a.K; k += 256) {
      u4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = row_end<true>(p[q] + k * 4, a.K - k);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t x = v[q][e] & 0x7fffffffu;
          if (x < 0x7f800000u) top = max(top, x);
        }
    }
  }
  __shared__ uint32_t red[16];
  for (int o = 32; o >= 1; o /= 2) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 16; ++i) top = max(top, red[i]);
    atomicMax(w ? &a.sc->top_w : &a.sc->top_h, top);
  }
}

// Rows as operands: gathered (h), padded with zeros to Kp, fp32 split into its parts.  which 0: h, 1: W, 2: h times the
// rows' weights.
constexpr float kOne = 32768.f;      // scale of what is at most 1
constexpr int kUp = 11;              // and of its second part beside it: fp32's dz is off by 2^-22 of itself or 2^-51 (and
                                     // its products by as much, without that of both second parts)
template <bool BF>
__global__ __launch_bounds__(256) void vocab_pack_kernel(VocabCE a, int which) {
  const bool w = which == 1;
  const int rows = w ? a.V : vocab_count(a);
  const int per = a.Kp / 8;
  uint16_t* dst = w ? a.wp : which == 2 ? a.hw : a.hp;
  float up = 1.f, up_weight = 1.f;
  if constexpr (!BF) {
    up = scale_up(w ? a.sc->top_w : a.sc->top_h);
    if (which == 2) up_weight = scale_up(a.sc->top_weight);
  }
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)rows * per; i += (int64_t)gridDim.x * 256) {
    const int r = (int)(i / per), k = (int)(i - (int64_t)r * per) * 8;
    const int64_t row = !w && a.idx ? a.idx[r] : r, from = row * a.K + k;
    if constexpr (BF) {
      const u4 o = row_end<false>((const char*)((const uint16_t*)(w ? a.W : a.h) + from), a.K - k);
      *(u4*)(dst + (int64_t)r * a.Kp + k) = o;
    } else {
      const float* s = (const float*)(w ? a.W : a.h) + from;
      const f4 v0 = __builtin_bit_cast(f4, row_end<true>((const char*)s, a.K - k));
      const f4 v1 = __builtin_bit_cast(f4, row_end<true>((const char*)(s + 4), a.K - k - 4));
      const float weight = which == 2 ? a.weights[row] * up_weight * (1.f / kOne) : 1.f;
      f4 x = v0 * up * weight, y = v1 * up * weight;
      uint16_t* d = dst + (int64_t)r * a.Kp * 2 + (k / 32) * 64 + k % 32;
      *(h4*)d = first_part(x);
      *(h4*)(d + 4) = first_part(y);
      *(h4*)(d + 32) = first_part(x);
      *(h4*)(d + 36) = first_part(y);
    }
  }
}

// The logits of a tile: tokens from v0 (m) x rows from n0 (n).  bf16 rows, and an fp32 tile's of few rows, are taken as they
// are, whatever their width.
template <class P, bool BF>
__device__ inline void vocab_logits(P& p, const VocabCE& a, int count, int v0, int n0, lds_t* lds) {
  if constexpr (BF || P::F32) {
    const Operand w = P::F32 ? Operand{(const uint16_t*)a.W, (int64_t)a.K * 2, a.V, a.K} : Operand{a.wp, a.Kw, a.V, a.Kw};
    const Operand h = P::F32 ? Operand{(const uint16_t*)a.h, (int64_t)a.K * 2, count, a.K, a.idx} : Operand{a.hp, a.Kh, count, a.Kh};
    const int whole = BF && a.Kw == a.Kp && a.Kh == a.Kp ? a.Kp : a.K / P::kStep * P::kStep;
    p.run(w, h, v0, n0, 0, whole, lds);
    if (whole < a.K)
      p.run_end([&](int m) { return (const char*)w.p + (int64_t)min(v0 + m, a.V - 1) * w.ld * 2; },
                [&](int n) {
                  const int r = min(n0 + n, count - 1);
                  return (const char*)h.p + (int64_t)(h.idx ? h.idx[r] : r) * h.ld * 2;
                },
                whole, a.K);
  } else {
    p.run(Operand{a.wp, (int64_t)a.Kp * 2, a.V, a.Kp}, Operand{a.hp, (int64_t)a.Kp * 2, count, a.Kp}, v0, n0, 0, a.Kp, lds);
  }
}

// ------------------------------------------------------------------------------ forward
// Tiles of the vocabulary (m) x rows (n): each lane holds four neighbouring tokens of one row, so that a row's statistics
// of a tile take two shuffles (rows as m would take four, for each of four rows).
template <class P, bool BF>
__global__ __launch_bounds__(P::kThreads) void vocab_fwd_kernel(VocabCE a, int tm, int tn) {
  extern __shared__ char smem[];
  int mt, nt;
  tile_of(blockIdx.x, gridDim.x, tm, tn, mt, nt);
  const int count = vocab_count(a), m0 = mt * P::BM, n0 = nt * P::BN;
  if (n0 >= count) return;
  P p;
  constexpr bool scaled = !BF && !P::F32;
  vocab_logits<P, BF>(p, a, count, m0, n0, (lds_t*)smem);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  const int wm = wave % P::WM, wn = wave / P::WM, first = m0 + wm * P::TM * 16 + 4 * g;
  const float down = scaled ? scale_down(a.sc->top_h, a.sc->top_w) : 1.f;
  float2* red = (float2*)smem;      // (the product ended with a barrier)
#pragma unroll
  for (int j = 0; j < P::TN; ++j) {
    const int nl = wn * P::TN * 16 + 16 * j + c, n = n0 + nl;
    const int64_t lab = n < count ? a.labels[a.idx ? a.idx[n] : n] : -1;
    const int64_t off = lab - first;
    const bool mine = off >= 0 && off < P::TM * 16 && (off & 15) < 4 && lab < a.V;
    float top = -INFINITY;
    if (m0 + P::BM > a.V) {      // the last tile
#pragma unroll
      for (int i = 0; i < P::TM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (first + 16 * i + e >= a.V) p.acc[i][j][e] = -INFINITY;
    }
    // (fmaxf passes over NaN: the sum has it)
#pragma unroll
    for (int i = 0; i < P::TM; ++i) {
      if constexpr (scaled) p.acc[i][j] *= down;
      top = fmaxf(fmaxf(top, fmaxf(p.acc[i][j][0], p.acc[i][j][1])), fmaxf(p.acc[i][j][2], p.acc[i][j][3]));
    }
    if (__any(mine)) {
#pragma unroll
      for (int i = 0; i < P::TM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (mine && off == 16 * i + e) a.zlab[n] = p.acc[i][j][e];
    }
    float2 s = {top * kLog2e, 0.f};
    const float ref = top == -INFINITY ? 0.f : s.x;
#pragma unroll
    for (int i = 0; i < P::TM; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s.y += expo2(fmaf(p.acc[i][j][e], kLog2e, -ref));
#pragma unroll
    for (int o = 16; o <= 32; o *= 2) s = joined(s, float2{__shfl_xor(s.x, o, 64), __shfl_xor(s.y, o, 64)});
    if (g == 0) red[wm * P::BN + nl] = s;
  }
  __syncthreads();
  for (int nl = threadIdx.x; nl < P::BN; nl += P::kThreads) {
    if (n0 + nl >= count) break;
    float2 s = red[nl];
#pragma unroll
    for (int w = 1; w < P::WM; ++w) s = joined(s, red[w * P::BN + nl]);
    ((float2*)a.part)[(int64_t)mt * a.N + n0 + nl] = s;
  }
}

// loss = sum_n w_n nll_n in 64 bits, in a fixed order (1024 threads).
__device__ inline void vocab_sum(const VocabCE& a, double* red) {
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

// A row's statistics from its tiles': R rows by SL slices of the tiles.  One workgroup alone (few rows: 64 at a time)
// takes them all, and the loss.
template <int R>
__global__ __launch_bounds__(1024) void vocab_join_kernel(VocabCE a, int tiles) {
  constexpr int SL = 1024 / R;
  __shared__ float2 red[SL][R + 1];
  __shared__ double sums[16];
  const int count = vocab_count(a), r = threadIdx.x % R, sl = threadIdx.x / R;
  const float2* part = (const float2*)a.part;
  for (int64_t row0 = (int64_t)blockIdx.x * R; row0 < count; row0 += (int64_t)gridDim.x * R) {
    float2 s = {-INFINITY, 0.f};
    if (row0 + r < count)
#pragma unroll 8
      for (int m = sl; m < tiles; m += SL) s = joined(s, part[(int64_t)m * a.N + row0 + r]);
    red[sl][r] = s;
    __syncthreads();
    // the row's slices by SL neighbouring lanes
    const int slice = threadIdx.x % SL;
    const int64_t k = row0 + threadIdx.x / SL;
    s = red[slice][threadIdx.x / SL];
#pragma unroll
    for (int o = SL / 2; o >= 1; o /= 2) s = joined(s, float2{__shfl_xor(s.x, o, SL), __shfl_xor(s.y, o, SL)});
    if (slice == 0 && k < count) {
      const int64_t row = a.idx ? a.idx[k] : k;
      const int64_t lab = a.labels[row];
      const bool token = lab >= 0 && lab < a.V;
      a.nll[row] = token ? (float)(((double)s.x + (double)log2f(s.y)) / (double)kLog2e - (double)a.zlab[k]) : NAN;
      a.stats[2 * row] = s.x;
      a.stats[2 * row + 1] = token ? 1.f / s.y : NAN;
    }
    __syncthreads();
  }
  if (gridDim.x == 1) {
    __threadfence_block();
    vocab_sum(a, sums);
  }
}

__global__ __launch_bounds__(1024) void vocab_loss_kernel(VocabCE a) {
  __shared__ double red[16];
  vocab_sum(a, red);
}

// ------------------------------------------------------------------------------ backward
// bf16's dz is without this factor, so that equal weights are 1 there and a label's entry, nearly -weight where its token is
// unlikely, is not off by the weight's rounding in every row (7252 x 1898 x 1258: gradients 0.0029 off, so 0.0020).
__device__ inline float unit_weight(const VocabCE& a) { return a.weights ? __uint_as_float(a.sc->top_weight) : a.mean; }

// The logits again (the whole of them in 16 bits would be 0.8 GB for 8192 rows of 50257) and
// the gradient of the logits of one piece of the vocabulary, [rows][vc] in 16 bits, without the factor g (fp32: and
// without the weights; bf16: over the unit weight).
template <class P, bool BF>
__global__ __launch_bounds__(P::kThreads) void vocab_dz_kernel(VocabCE a, int v0, int vc, int tm, int tn) {
  extern __shared__ char smem[];
  int mt, nt;
  tile_of(blockIdx.x, gridDim.x, tm, tn, mt, nt);
  const int count = vocab_count(a), m0 = mt * P::BM, n0 = nt * P::BN;
  if (n0 >= count || v0 + m0 >= a.V) return;      // (what is read behind V of dz lies in the tile of V - 1)
  P p;
  constexpr bool scaled = !BF && !P::F32;
  vocab_logits<P, BF>(p, a, count, v0 + m0, n0, (lds_t*)smem);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  const int wm = wave % P::WM, wn = wave / P::WM, first = v0 + m0 + wm * P::TM * 16 + 4 * g;
  const float down = scaled ? scale_down(a.sc->top_h, a.sc->top_w) : 1.f;
  const int padded = (count + kBK - 1) / kBK * kBK;      // rows that the contraction over them reads
  const bool edge = v0 + m0 + P::BM > a.V || n0 + P::BN > count;
#pragma unroll
  for (int j = 0; j < P::TN; ++j) {
    const int n = n0 + wn * P::TN * 16 + 16 * j + c;
    int64_t lab = -1;
    float top = 0.f, inv = 0.f, w = 0.f;
    if (n < count) {
      const int64_t row = a.idx ? a.idx[n] : n;
      lab = a.labels[row];
      w = !BF ? kOne : a.weights ? a.weights[row] / unit_weight(a) : 1.f;
      top = a.stats_in[2 * row], inv = a.stats_in[2 * row + 1] * w;
    }
#pragma unroll
    for (int i = 0; i < P::TM; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) p.acc[i][j][e] = expo2(fmaf(scaled ? p.acc[i][j][e] * down : p.acc[i][j][e], kLog2e, -top)) * inv;
    const int64_t off = lab - first;
    const bool mine = off >= 0 && off < P::TM * 16 && (off & 15) < 4;
    if (__any(mine)) {
#pragma unroll
      for (int i = 0; i < P::TM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (mine && off == 16 * i + e) p.acc[i][j][e] -= w;
    }
    if (edge) {
#pragma unroll
      for (int i = 0; i < P::TM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n >= count || first + 16 * i + e >= a.V) p.acc[i][j][e] = 0.f;
    }
  }
  uint16_t* out = a.dz + ((int64_t)n0 * vc + m0) * P::NP;
  if constexpr (BF) {
    store_rows<P>(smem, out, vc, padded - n0, [&](int i, int j) {
      return uint2{bf16_pair(p.acc[i][j][0], p.acc[i][j][1]), bf16_pair(p.acc[i][j][2], p.acc[i][j][3])};
    });
  } else {
    // a first part, and what it leaves, in the sum's place, as the second one
    store_rows<P>(smem, out, (int64_t)vc * 2, padded - n0, [&](int i, int j) __attribute__((always_inline)) {
      const uint2 part = __builtin_bit_cast(uint2, first_part(p.acc[i][j]));
      p.acc[i][j] *= (float)(1 << kUp);
      return part;
    });
  }
}

// part[s] (+)= dz W over the s-th part of the piece: rows (n) x K (m).  Few tiles and a long contraction: 32 x 3 tiles of
// 256 x 256 of 8192 x 768 would leave most CUs idle, 32 x 4 of 192 in two parts make a round (21760 tokens 308 us, 890 TFLOP/s).
template <class P, bool BF>
__global__ __launch_bounds__(P::kThreads) void vocab_dh_kernel(VocabCE a, int v0, int vc, int tm, int tn, int len, int add) {
  extern __shared__ char smem[];
  int mt, nt;
  tile_of(blockIdx.x, gridDim.x, tm, tn, mt, nt, 4);
  const int count = vocab_count(a), m0 = mt * P::BM, n0 = nt * P::BN;
  if (n0 >= count) return;
  const int k0 = blockIdx.y * len, k1 = min(min(vc, a.V - v0), k0 + len);
  const Operand dz = {a.dz, (int64_t)vc * P::NP, count, vc};
  P p;
  const int64_t ld = P::NP == 2 ? a.Kp * 2 : a.Kw;
  p.run(Operand{a.wp + v0 * ld, ld, a.V - v0, P::NP == 2 ? a.Kp : a.Kw}, dz, m0, n0, k0, k1, (lds_t*)smem);
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

// (64 x 1536 x 100000: 231 us, 2.7 TB/s and 85 TFLOP/s of the instruction's 157; with one step on its way 376.)
// dh's parts of few rows, of fp32's W as it is: 256 of K (four wavefronts' 64) x TN x 16 rows, the contraction over the
// tokens on the fp32 instruction.  A lane holds four neighbouring k of a token: they are rows of four products, so that row m
// of product i is k = 4 m + i.  Three steps of sixteen tokens are on their way to each wavefront's registers.
template <int TN>
__global__ __launch_bounds__(256, 2) void vocab_dh_few_kernel(VocabCE a, int v0, int vc, int tn, int len, int add) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, c = lane & 15;
  const int count = vocab_count(a), n0 = (blockIdx.x % tn) * TN * 16, k0 = (blockIdx.x / tn * 4 + wave) * 64;
  if (n0 >= count || k0 >= a.K) return;
  typedef f4 any __attribute__((aligned(4)));
  const int b0 = blockIdx.y * len, b1 = min(min(vc, b0 + len), a.V - v0);
  const float* W = (const float*)a.W + (int64_t)(v0 + b0) * a.K + k0;
  const uint16_t* dz[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) dz[j] = a.dz + (int64_t)min(n0 + 16 * j + c, count - 1) * vc * 2;
  f4 acc[4][TN];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f4{0, 0, 0, 0};
  struct Step {
    f4 w[4];
    h4 d[TN][2];
  };
  const uint32_t mine = (uint32_t)(4 * g * a.K + 4 * c);
  auto load_dz = [&](Step& s, int b) __attribute__((always_inline)) {      // (zero from V to the end of its piece)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const uint16_t* p = dz[j] + ((b + 4 * g) / 32) * 64 + (b + 4 * g) % 32;
      s.d[j][0] = *(const h4*)p, s.d[j][1] = *(const h4*)(p + 32);
    }
  };
  auto load = [&](Step& s, int b) __attribute__((always_inline)) {      // tokens b .. b + 15 of the piece, all there
#pragma unroll
    for (int e = 0; e < 4; ++e) s.w[e] = *(const any*)(W + (int64_t)(b - b0) * a.K + (mine + e * a.K));
    load_dz(s, b);
    __builtin_amdgcn_sched_barrier(0);      // (the compiler would move them behind the products)
  };
  auto multiply = [&](const Step& s) __attribute__((always_inline)) {
    f4 d[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) d[j] = __builtin_convertvector(s.d[j][0], f4) * (1 / kOne) + __builtin_convertvector(s.d[j][1], f4) * (1 / kOne / (1 << kUp));
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(s.w[e][i], d[j][e], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  int b = b0;
  if (k0 + 64 <= a.K) {
    const int steps = max(0, b1 - b0) / 16;
    Step s[3];
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < steps) load(s[i], b0 + 16 * i);
    int t = 0;
    for (; t + 6 <= steps; t += 3)
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        multiply(s[i]);
        load(s[i], b0 + 16 * (t + 3 + i));
      }
#pragma unroll
    for (int i = 0; i < 5; ++i)
      if (t + i < steps) {
        multiply(s[i % 3]);
        if (t + 3 + i < steps) load(s[i % 3], b0 + 16 * (t + 3 + i));
      }
    b += 16 * steps;
  }
  const int left = a.K - k0 - 4 * c;
  for (; b < b1; b += 16) {      // the last tokens, or the last of K
    Step s;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int v = b + 4 * g + e;
      s.w[e] = __builtin_bit_cast(f4, row_end<true>((const char*)(W + (int64_t)(v - b0) * a.K + 4 * c), v < b1 ? left : 0));
    }
    load_dz(s, b);
    multiply(s);
  }
  float* out = a.dhpart + (int64_t)blockIdx.y * a.N * a.Kp;
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int n = n0 + 16 * j + c;
    if (n >= count) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      f4* q = (f4*)(out + (int64_t)n * a.Kp + k0 + 16 * g + 4 * r);
      const f4 s = {acc[0][j][r], acc[1][j][r], acc[2][j][r], acc[3][j][r]};
      *q = add ? *q + s : s;
    }
  }
}

// What the sums of a gradient are times, in two steps: those of fp32 parts lie between 2^-20 and 2^50, whatever the tensors'
// and the weights' sizes are, and sum f is within fp32's range then where sum f f2 is.
struct Factor {
  float f, f2;
};
__device__ inline Factor factor(double v) {
  const int e = (int)((uint64_t)__double_as_longlong(v) >> 52 & 0x7ff) - 1023;
  const int near = v == 0 || e == 1024 ? e : min(60, max(-90, e)), rest = min(127, max(-126, e - near));
  return {(float)(v * __longlong_as_double((int64_t)(1023 + near - e) << 52)), __uint_as_float((uint32_t)(rest + 127) << 23)};
}

// Four gradients of a row of K in their type.
template <bool BF>
__device__ inline void put_grad(void* p, int64_t row, int k, int K, f4 s, Factor f) {
  s = s * f.f * f.f2;
  if constexpr (BF) {
    uint16_t* o = (uint16_t*)p + row * K + k;
    if ((K & 3) == 0)
      *(uint2*)o = uint2{bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3])};
    else
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (k + e < K) o[e] = (uint16_t)bf16_rne(s[e]);
  } else {
    float* o = (float*)p + row * K + k;
    if ((K & 3) == 0)
      *(f4*)o = s;
    else
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (k + e < K) o[e] = s[e];
  }
}

// Of many parts of few rows SL threads sum every SL-th, and one of them what they have (36 x 692, 170 parts: 19 -> 10 us;
// 1001 x 750, 16 parts: 8 -> 11).
template <bool BF, int SL>
__global__ __launch_bounds__(256) void vocab_dh_join_kernel(VocabCE a, int splits) {
  constexpr int G = 256 / SL;
  __shared__ f4 red[SL][G];
  // (W as it is was multiplied by dz without its scale)
  const double gout = a.gout[0], down = BF || a.wp == a.W ? 1.0 : (double)scale_down(a.sc->top_w) / kOne;
  const int per = a.Kp / 4, slice = threadIdx.x / G, mine = threadIdx.x % G;
  for (int64_t i0 = (int64_t)blockIdx.x * G; i0 < a.N * per; i0 += (int64_t)gridDim.x * G) {
    const int64_t i = i0 + mine, row = i / per;
    const int k = (int)(i - row * per) * 4;
    const bool in = row < a.N && k < a.K;
    const int64_t at = !in ? -1 : a.idx ? a.pos[row] : row;
    f4 s = {0, 0, 0, 0};
    if (at >= 0)
#pragma unroll 8
      for (int t = slice; t < splits; t += SL) s += *(const f4*)(a.dhpart + ((int64_t)t * a.N + at) * a.Kp + k);
    if constexpr (SL > 1) {
      red[slice][mine] = s;
      __syncthreads();
      if (slice == 0)
#pragma unroll
        for (int q = 1; q < SL; ++q) s += red[q][mine];
      __syncthreads();
    }
    if (in && slice == 0) {
      const double f = (BF ? unit_weight(a) : a.weights ? a.weights[row] : a.mean) * gout * down;
      put_grad<BF>(a.dh, row, k, a.K, s, at >= 0 ? factor(f) : Factor{0.f, 0.f});
    }
  }
}

// What dW's sums are times.
template <bool BF>
__device__ inline Factor dw_factor(const VocabCE& a) {
  const double gout = a.gout[0];
  if constexpr (BF) return factor(gout * unit_weight(a));
  else return factor(gout * scale_down(a.sc->top_h) * (a.weights ? (double)scale_down(a.sc->top_weight) : (double)a.mean / kOne));
}

// dW of a piece: K (m) x vocabulary (n), the contraction over the rows, in gridDim.y parts (one: into dW itself).  A piece's
// tiles fill a round (255 of 768 x 21760: 245 us over 8192 rows, 1,117 TFLOP/s); of few rows it is the writing of dW, in whole
// lines (bf16 33 x 1024 x 100000 53 us, eight bytes of each of sixteen rows at a time 80).
template <class P, bool BF>
__global__ __launch_bounds__(P::kThreads) void vocab_dw_kernel(VocabCE a, int v0, int vc, int tm, int tn) {
  extern __shared__ char smem[];
  int mt, nt;
  tile_of(blockIdx.x, gridDim.x, tm, tn, mt, nt);
  const int count = vocab_count(a), m0 = mt * P::BM, n0 = nt * P::BN;
  const int padded = (count + kBK - 1) / kBK * kBK;
  const int len = (padded / kBK + gridDim.y - 1) / gridDim.y * kBK, k0 = blockIdx.y * len;
  const Operand dz = {a.dz, (int64_t)vc * P::NP, padded, vc};
  const int wide = P::NP == 2 ? a.Kp : a.Kh;
  const Operand h = {P::NP == 2 && a.weights ? a.hw : a.hp, (int64_t)wide * P::NP, count, wide};
  P p;
  p.run(h, dz, m0, n0, k0, min(count, k0 + len), (lds_t*)smem);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  const Factor f = dw_factor<BF>(a);
  if constexpr (BF) {
    if (gridDim.y == 1 && m0 + P::BM <= a.K && a.K % 8 == 0) {      // whole lines
      store_rows<P>(smem, (uint16_t*)a.dW + (int64_t)(v0 + n0) * a.K + m0, a.K, a.V - v0 - n0, [&](int i, int j) __attribute__((always_inline)) {
        const f4 s = p.acc[i][j] * f.f * f.f2;
        return uint2{bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3])};
      });
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < P::TN; ++j) {
    const int n = n0 + (wave / P::WM) * P::TN * 16 + 16 * j + c;
    if (v0 + n >= a.V) continue;
#pragma unroll
    for (int i = 0; i < P::TM; ++i) {
      const int k = m0 + (wave % P::WM) * P::TM * 16 + 16 * i + 4 * g;
      if (gridDim.y > 1) {
        if (k < a.Kp) *(f4*)(a.dwpart + ((int64_t)blockIdx.y * vc + n) * a.Kp + k) = p.acc[i][j];
      } else if (k < a.K) {
        put_grad<BF>(a.dW, v0 + n, k, a.K, p.acc[i][j], f);
      }
    }
  }
}

template <bool BF>
__global__ __launch_bounds__(256) void vocab_dw_join_kernel(VocabCE a, int v0, int vc, int parts) {
  const Factor f = dw_factor<BF>(a);
  const int per = a.Kp / 4, rows = min(vc, a.V - v0);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)rows * per; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per;
    const int k = (int)(i - row * per) * 4;
    if (k >= a.K) continue;
    f4 s = {0, 0, 0, 0};
    for (int t = 0; t < parts; ++t) s += *(const f4*)(a.dwpart + ((int64_t)t * vc + row) * a.Kp + k);
    put_grad<BF>(a.dW, v0 + row, k, a.K, s, f);
  }
}

// ------------------------------------------------------------------------------ host
// Tiles of a product, m x n; what has a COL operand multiplies dz (B).
enum Tile { kBig, kWide, kMid, kSmall, kFew };      // 256 x 256, 192 x 256, 128 x 128, 64 x 64, 256 x 64
template <int WM, int WN, int TM, int TN, Side SA, Side SB, bool BF, int NS = 2>
using TileOf = Product<WM, WN, TM, TN, SA, SB, BF, BF ? 1 : 2, NS, false, 1, !BF && SA == COL ? kUp : 0>;
template <int T, bool BF, Side SA, Side SB>
using Tiled = std::conditional_t<T == kBig, TileOf<2, 4, 8, 4, SA, SB, BF>,
              std::conditional_t<T == kWide, TileOf<2, 4, 6, 4, SA, SB, BF>,
              std::conditional_t<T == kMid, TileOf<2, 2, 4, 4, SA, SB, BF>,
              std::conditional_t<T == kSmall, TileOf<2, 2, 2, 2, SA, SB, BF, 4>, TileOf<4, 1, 4, 4, SA, SB, BF>>>>>;
// fp32 as it is: 128 x TN 16.  The instruction's rate bounds it from about 64 rows on, W's reading below: 32 x 1024 x 60000
// 4.6 TB/s, 64 x 1024 x 32000 42 us (3.1 TB/s, 100 TFLOP/s; loads into registers, 64 bytes of sixteen rows each: 60).
template <int TN, int NS>
using Whole = Product<4, 1, 2, TN, ROW, ROW, false, 2, NS, true>;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Rows and width of a product with few rows: a tile of 64 (bf16).
bool few(int64_t N) { return N <= 64; }

// Whether fp32's products with W take it as it is, on the fp32 instruction.
bool direct_of(int64_t N, bool bf) { return !bf && N > 0 && N <= 128; }

// The tile and the parts of the contraction that cost least, with what was measured of each tile: a step of 64 where its
// workgroup has the CU to itself and where `resident` share it, and start and end; the parts' sums go through memory at
// 4.5 TB/s, `moves` times.  (362 x 424 x 6552 fp32: its products in tiles of 256 alone 33, 36, 30 and 21 us.)
struct TileCost {
  Tile tile;
  int m, n, resident;
  double alone, shared, ends;
};
constexpr TileCost kTiles[] = {{kBig, 256, 256, 1, 2.2, 2.2, 4}, {kWide, 192, 256, 1, 1.65, 1.65, 4}, {kMid, 128, 128, 2, 0.85, 0.62, 3.5},
                               {kSmall, 64, 64, 2, 0.5, 0.25, 3}, {kFew, 256, 64, 2, 0.85, 0.62, 3.5}};
struct Choice {
  Tile tile;
  int parts;
};
// tiles: a mask of the ones to choose from; steps of 64 of the contraction (fp32: of its three products).
Choice choose(int64_t m, int64_t n, int64_t steps, int most, double moves, unsigned tiles) {
  Choice best{kBig, 1};
  double least = 1e300;
  for (const TileCost& t : kTiles) {
    if (!(tiles >> t.tile & 1)) continue;
    const int64_t all = ceil_div(m, t.m) * ceil_div(n, t.n);
    for (int s = 1; s <= most && (s == 1 || steps / s >= 4); ++s) {
      const int64_t each = ceil_div(all * s, 256), rounds = each / t.resident, rest = each % t.resident, len = ceil_div(steps, s);
      auto run = [&](int64_t c) { return c ? len * std::max(t.alone, c * t.shared) + t.ends : 0.0; };
      const double us = rounds * run(t.resident) + run(rest) + (s > 1 || moves > 2 ? (double)m * n * s * moves * 8.9e-7 : 0);
      if (us < least) least = us, best = {t.tile, s};
    }
  }
  return best;
}
const TileCost& cost_of(Tile t) { return kTiles[t]; }
constexpr unsigned kSquares = 1u << kBig | 1u << kMid | 1u << kSmall;
constexpr unsigned squares_or_few(bool bf) { return kSquares | (bf ? 1u << kFew : 0); }
unsigned tiles_for(int64_t N, int planes, unsigned many) { return planes == 1 && few(N) ? 1u << kFew | 1u << kSmall : many; }

struct VocabPlan {
  int Kp;
  bool rows, copy_h, copy_w;      // rows in use are listed; operands that are copies
  bool direct;                    // W as it is
  Tile fwd;
  int tiles;                      // of the vocabulary in the forward
  int piece, pieces;              // backward
  Choice dh;
  size_t sc, idx, pos, hp, hw, wp, part, zlab, dz, dhpart, dwpart, bytes;
};

int64_t steps_of(int64_t n, int planes) { return ceil_div(n, kBK) * (planes == 2 ? 3 : 1); }
Choice logits_tile(int64_t N, int Kp, int64_t vc, int planes) {
  return choose(vc, N, steps_of(Kp, planes), 1, 2, tiles_for(N, planes, kSquares));
}
Choice dw_tile(int64_t N, int Kp, int vc, int planes) { return choose(Kp, vc, steps_of(N, planes), 8, 2, kSquares); }

VocabPlan plan_of(int64_t N, int K, int V, bool bf, bool weights, bool backward) {
  VocabPlan p{};
  p.Kp = (int)ceil_div(K, kBK) * kBK;
  p.rows = weights;
  p.direct = direct_of(N, bf);
  // bf16 rows that are not whole cache lines load slower, and are copied where a copy costs less than that: 2050 x 1000 x 32003
  // takes 175 us with copies and 194 without, 300 x 1000 x 100000 287 and 145.  (dh and dW take whole 16-byte pieces of rows.)
  const bool copies = (K % kBK && N > 512) || (backward && K % 8);
  p.copy_h = bf ? weights || copies : backward || !p.direct;
  p.copy_w = bf ? copies : !p.direct;
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t r = at; at += up256(bytes); return r; };
  const int planes = bf ? 1 : 2;
  p.fwd = logits_tile(N, p.Kp, V, planes).tile;
  p.tiles = (int)ceil_div(V, p.direct ? 128 : cost_of(p.fwd).m);
  const int64_t rows = ceil_div(std::max<int64_t>(N, 1), kBK) * kBK;
  p.sc = take(sizeof(VocabScales));
  p.idx = take(p.rows ? 4 * (size_t)N : 0);
  p.pos = take(p.rows ? 4 * (size_t)N : 0);
  p.hp = take(p.copy_h ? 2 * (size_t)planes * N * p.Kp : 0);
  p.hw = take(backward && !bf && weights ? 2 * (size_t)planes * N * p.Kp : 0);
  p.wp = take(p.copy_w ? 2 * (size_t)planes * V * p.Kp : 0);
  if (!backward) {
    p.part = take(8 * (size_t)p.tiles * N);
    p.zlab = take(4 * (size_t)N);
  } else {
    // dz of a piece takes at most about 512 MB; where a tile of dW takes long, a piece's tiles fill whole rounds
    const int64_t tk = ceil_div(p.Kp, 256), wide = ceil_div(V, 256);
    int64_t piece = std::min<int64_t>(wide, std::max<int64_t>(1, (int64_t(512) << 20) / (rows * 256 * 2 * planes)));
    if (steps_of(rows, planes) >= 16 && piece * tk >= 256) piece = piece * tk / 256 * 256 / tk;
    p.piece = (int)piece * 256;
    p.pieces = (int)ceil_div(wide, piece);
    p.dz = take(2 * (size_t)planes * rows * p.piece);
    if (p.direct) {      // (parts of 128 tokens at least)
      const int64_t groups = tk * (few(N) ? 1 : 2);
      p.dh.parts = (int)std::min<int64_t>(std::max<int64_t>(1, 512 / groups), p.piece / 128);
    } else {
      p.dh = choose(p.Kp, N, steps_of(p.piece, planes), few(N) ? 128 : 16, p.pieces > 1 ? 4 : 2, tiles_for(N, planes, kSquares | 1u << kWide));
    }
    p.dhpart = take(4 * (size_t)p.dh.parts * N * p.Kp);
    size_t most = 0;
    for (int i = 0; i < p.pieces; ++i) {
      const int vc = (int)std::min<int64_t>(p.piece, (wide - i * piece) * 256), parts = dw_tile(N, p.Kp, vc, planes).parts;
      if (parts > 1) most = std::max(most, 4 * (size_t)parts * vc * p.Kp);
    }
    p.dwpart = take(most);
  }
  p.bytes = at;
  return p;
}

VocabCE bind(const VocabCE& k, const VocabPlan& p, char* ws, bool bf) {
  VocabCE a = k;
  a.Kp = p.Kp;
  a.Kh = p.copy_h ? p.Kp : k.K;
  a.Kw = p.copy_w ? p.Kp : k.K;
  a.sc = p.rows || (p.copy_h && !bf) ? (VocabScales*)(ws + p.sc) : nullptr;
  a.idx = p.rows ? (int*)(ws + p.idx) : nullptr;
  a.pos = (int*)(ws + p.pos);
  a.hp = p.copy_h ? (uint16_t*)(ws + p.hp) : (uint16_t*)k.h;
  a.wp = p.copy_w ? (uint16_t*)(ws + p.wp) : (uint16_t*)k.W;
  a.hw = (uint16_t*)(ws + p.hw);
  a.part = (float*)(ws + p.part);
  a.zlab = (float*)(ws + p.zlab);
  a.dz = (uint16_t*)(ws + p.dz);
  a.dhpart = (float*)(ws + p.dhpart);
  a.dwpart = (float*)(ws + p.dwpart);
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
  if (a.sc) hipLaunchKernelGGL(vocab_rows_kernel, dim3(1), dim3(1024), 0, s, a);
  if (!BF && p.copy_h) {
    // (the atomics of 256 workgroups on a line take 9 us: each has 64 KB at least)
    const int64_t most = std::max<int64_t>(a.N, p.copy_w ? a.V : 0) * a.K;
    hipLaunchKernelGGL(vocab_top_kernel, dim3((unsigned)std::min<int64_t>(256, ceil_div(most, 16384)), p.copy_w ? 2 : 1), dim3(1024), 0, s, a);
  }
  const int per = p.Kp / 8;
  auto blocks = [&](int64_t rows) { return dim3((unsigned)std::min<int64_t>(4096, std::max<int64_t>(1, ceil_div(rows * per, 256)))); };
  if (p.copy_h && a.N) hipLaunchKernelGGL((vocab_pack_kernel<BF>), blocks(a.N), dim3(256), 0, s, a, 0);
  if (!BF && a.dW && a.weights && a.N) hipLaunchKernelGGL((vocab_pack_kernel<BF>), blocks(a.N), dim3(256), 0, s, a, 2);
  if (p.copy_w) hipLaunchKernelGGL((vocab_pack_kernel<BF>), blocks(a.V), dim3(256), 0, s, a, 1);
  return hipGetLastError();
}

// f(tile) with the tile as a constant, of the ones in `tiles`.
template <unsigned tiles, class F>
hipError_t with_tile(Tile t, const F& f) {
  hipError_t e = hipErrorInvalidValue;
  auto one = [&](auto tile) {
    if constexpr (tiles >> tile.value & 1)
      if (t == tile.value) e = f(tile);
  };
  one(std::integral_constant<int, kBig>{}), one(std::integral_constant<int, kWide>{}), one(std::integral_constant<int, kMid>{});
  one(std::integral_constant<int, kSmall>{}), one(std::integral_constant<int, kFew>{});
  return e;
}
// f(Product) of fp32 W as it is.
template <class F>
hipError_t with_rows(int64_t N, const F& f) {
  if (N <= 32) return f((Whole<2, 4>*)nullptr);
  if (N <= 64) return f((Whole<4, 3>*)nullptr);
  return f((Whole<8, 2>*)nullptr);
}

template <bool BF>
hipError_t run_fwd(const VocabCE& a, const VocabPlan& p, hipStream_t s) {
  hipError_t e = prepare<BF>(a, p, s);
  if (e != hipSuccess) return e;
  if (a.N) {
    if (p.direct) {
      if constexpr (!BF)
        e = with_rows(a.N, [&](auto* product) {
          typedef std::remove_pointer_t<decltype(product)> P;
          return go<P, vocab_fwd_kernel<P, BF>>(dim3((unsigned)p.tiles), s, a, p.tiles, 1);
        });
    } else {
      const int tn = (int)ceil_div(a.N, cost_of(p.fwd).n);
      e = with_tile<squares_or_few(BF)>(p.fwd, [&](auto tile) {
        typedef Tiled<tile, BF, ROW, ROW> P;
        return go<P, vocab_fwd_kernel<P, BF>>(dim3((unsigned)(p.tiles * tn)), s, a, p.tiles, tn);
      });
    }
    if (e != hipSuccess) return e;
    const bool one = a.N <= 128;      // a workgroup's few turns are shorter than another launch
    if (one) {
      hipLaunchKernelGGL((vocab_join_kernel<64>), dim3(1), dim3(1024), 0, s, a, p.tiles);
      return hipGetLastError();
    }
    hipLaunchKernelGGL((vocab_join_kernel<32>), dim3((unsigned)ceil_div(a.N, 32)), dim3(1024), 0, s, a, p.tiles);
  }
  hipLaunchKernelGGL(vocab_loss_kernel, dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}

template <bool BF>
hipError_t run_dz(const VocabCE& a, const VocabPlan& p, int v0, int vc, hipStream_t s) {
  if (p.direct) {
    if constexpr (!BF)
      return with_rows(a.N, [&](auto* product) {
        typedef std::remove_pointer_t<decltype(product)> P;
        return go<P, vocab_dz_kernel<P, BF>>(dim3((unsigned)(vc / P::BM)), s, a, v0, vc, vc / P::BM, 1);
      });
  }
  return with_tile<squares_or_few(BF)>(logits_tile(a.N, p.Kp, vc, BF ? 1 : 2).tile, [&](auto tile) {
    typedef Tiled<tile, BF, ROW, ROW> P;
    const int tm = vc / P::BM, tn = (int)ceil_div(a.N, P::BN);
    return go<P, vocab_dz_kernel<P, BF>>(dim3((unsigned)(tm * tn)), s, a, v0, vc, tm, tn);
  });
}

template <bool BF>
hipError_t run_dh(const VocabCE& a, const VocabPlan& p, int v0, int vc, hipStream_t s) {
  const int len = (int)ceil_div(ceil_div(vc, p.dh.parts), kBK) * kBK, add = v0 > 0;
  if (p.direct) {
    const int tn = few(a.N) ? 1 : 2;
    const dim3 grid((unsigned)(ceil_div(p.Kp, 256) * tn), (unsigned)p.dh.parts);
    if (a.N <= 32) hipLaunchKernelGGL((vocab_dh_few_kernel<2>), grid, dim3(256), 0, s, a, v0, vc, tn, len, add);
    else hipLaunchKernelGGL((vocab_dh_few_kernel<4>), grid, dim3(256), 0, s, a, v0, vc, tn, len, add);
    return hipGetLastError();
  }
  return with_tile<squares_or_few(BF) | 1u << kWide>(p.dh.tile, [&](auto tile) {
    typedef Tiled<tile, BF, COL, ROW> P;
    const int tm = (int)ceil_div(p.Kp, P::BM), tn = (int)ceil_div(a.N, P::BN);
    return go<P, vocab_dh_kernel<P, BF>>(dim3((unsigned)(tm * tn), (unsigned)p.dh.parts), s, a, v0, vc, tm, tn, len, add);
  });
}

template <bool BF>
hipError_t run_dw(const VocabCE& a, const VocabPlan& p, int v0, int vc, hipStream_t s) {
  const Choice w = dw_tile(a.N, p.Kp, vc, BF ? 1 : 2);
  const hipError_t e = with_tile<kSquares>(w.tile, [&](auto tile) {
    typedef Tiled<tile, BF, COL, COL> P;
    const int tm = (int)ceil_div(p.Kp, P::BM), tn = vc / P::BN;
    return go<P, vocab_dw_kernel<P, BF>>(dim3((unsigned)(tm * tn), (unsigned)w.parts), s, a, v0, vc, tm, tn);
  });
  if (e != hipSuccess || w.parts == 1) return e;
  hipLaunchKernelGGL((vocab_dw_join_kernel<BF>), dim3((unsigned)std::min<int64_t>(4096, ceil_div((int64_t)vc * (p.Kp / 4), 256))), dim3(256), 0, s,
                     a, v0, vc, w.parts);
  return hipGetLastError();
}

template <bool BF>
hipError_t run_bwd(const VocabCE& a, const VocabPlan& p, hipStream_t s) {
  hipError_t e = prepare<BF>(a, p, s);
  for (int i = 0; i < p.pieces && e == hipSuccess; ++i) {
    const int v0 = i * p.piece, vc = std::min(p.piece, (int)ceil_div(a.V - v0, 256) * 256);
    if (a.N) e = run_dz<BF>(a, p, v0, vc, s);
    if (a.dh && a.N && e == hipSuccess) e = run_dh<BF>(a, p, v0, vc, s);
    if (a.dW && e == hipSuccess) e = run_dw<BF>(a, p, v0, vc, s);
  }
  if (e == hipSuccess && a.dh && a.N) {
    auto join = [&](auto kernel, int each) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(8192, ceil_div(a.N * (p.Kp / 4), each))), dim3(256), 0, s, a, p.dh.parts);
    };
    if (p.dh.parts >= 16 && a.N * (p.Kp / 4) <= 65536) join(vocab_dh_join_kernel<BF, 8>, 32);
    else join(vocab_dh_join_kernel<BF, 1>, 256);
    e = hipGetLastError();
  }
  return e;
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
