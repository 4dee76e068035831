// The gated Kronecker block, forward and backward:
//   g = x Wg + bg,  u = x Wu + bu,  y = act(g) o u,   W_f = sum_i kron(S_f o A_fi, B_fi)
// Row n of x is a p x m matrix X, and with C_fi = S_f o A_fi (the layer's formulas, twice)
//   Z_fi = X B_fi (p x n),   g, u = sum_i C_fi^T Z_fi (q x n)
//   dg = dy u act'(g),  du = dy act(g);   dX = sum_fi C_fi (d_f B_fi^T)
//   dC_fi = sum_rows Z_fi d_f^T,  dB_fi = sum_rows X^T (C_fi d_f),  dA = S o dC,  dS = sum_i A_i o dC_i
// The products are in glu_rows.hip (forward, gradients of both projections, dX) and glu_param.hip (the
// factors' gradients); here are the layout of the factors, the last sums and the order of the launches.
//
// Small calls are bound by their launches and the latency in them: one token through 768 -> 2048 takes 13 to 15 us, 4.4
// of them the layout of the factors and 5.5 the products (on four workgroups); a backward of 61 rows 31 us in five
// launches of 4 to 13 under the profiler.  The layout is made in each call, from the plain factors that the
// calls take: training changes them with every step, serving pays the 4.4 us for each token.
#include "glu_parts.h"

namespace kron {
namespace {

// ---------------------------------------------------------------------------------
// The factors as operand blocks.  A table holds, for projection f and rank i, the blocks
// [tile of 16 columns][step of 32 k][part], 64 lanes x 16 bytes each.
// ---------------------------------------------------------------------------------
struct PackArgs {
  int p, q, m, n, r;
  int bf16, parts_b, parts_c;
  int tables;             // 2: the forward's, 4: the backward's too
  const void* S;
  const void* A;
  const void* B;
  u4* t[4];               // see GluTables
  int lanes[4];           // lanes of each table (all f, i): tile x step x 64, without parts
};

__device__ inline float raw(const void* t, int64_t i, int bf16) {
  return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)t)[i] << 16) : ((const float*)t)[i];
}
__device__ inline int chained(int g, int e) { return e < 4 ? 4 * g + e : 12 + 4 * g + e; }

__global__ __launch_bounds__(256) void glu_pack_kernel(PackArgs a) {
  int id = blockIdx.x * 256 + threadIdx.x;      // (32 bits throughout: divisions are most of this kernel's time)
  int w = 0;
  while (w < a.tables && id >= a.lanes[w]) id -= a.lanes[w++];
  if (w >= a.tables) return;
  // table 0: B, k = m, columns n; 1: C, k = p, columns q; 2: B^T, k = n, columns m; 3: C^T, k = q, columns p
  const int kd = w == 0 ? a.m : w == 1 ? a.p : w == 2 ? a.n : a.q;
  const int cd = w == 0 ? a.n : w == 1 ? a.q : w == 2 ? a.m : a.p;
  const int steps = (kd + 31) / 32, tiles = (cd + 15) / 16;
  const int lane = id & 63, g = lane >> 4, c = lane & 15;
  const int b = id >> 6, ks = b & (steps - 1), bt = steps == 2 ? b >> 1 : b;      // (a side of at most 64 has one step or two)
  const int fi = bt / tiles, tile = bt % tiles, f = fi >= a.r;
  const bool isb = (w & 1) == 0;
  const int col = 16 * tile + c;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int k = 32 * ks + (isb ? 8 * g + e : chained(g, e));
    float x = 0.f;
    if (k < kd && col < cd) {
      if (isb) {
        const int mi = w == 0 ? k : col, ni = w == 0 ? col : k;
        x = raw(a.B, (fi * a.m + mi) * a.n + ni, a.bf16);
      } else {
        const int pi = w == 1 ? k : col, qi = w == 1 ? col : k;
        x = raw(a.A, (fi * a.p + pi) * a.q + qi, a.bf16);
        // the product of two bf16 values has 16 bits: exact in fp32 and in two parts
        if (a.S) x *= raw(a.S, (f * a.p + pi) * a.q + qi, a.bf16);
      }
    }
    v[e] = x;
  }
  Op o[3];
  split<3>(f4{v[0], v[1], v[2], v[3]}, f4{v[4], v[5], v[6], v[7]}, o);
  const int parts = isb ? a.parts_b : a.parts_c;
  u4* dst = a.t[w] + b * parts * 64 + lane;
  for (int s = 0; s < parts; ++s) dst[s * 64] = s == 0 ? o[0].u : s == 1 ? o[1].u : o[2].u;
}

// ---------------------------------------------------------------------------------
// The partial rows summed in 64 bits in a fixed order, and dA = S o dC, dS = sum_i A_i o dC_i from dC.  A
// workgroup has a block of 32 columns (part_index): of dB, of dbias, or with S of dC's e-th elements of
// every rank.  32 rows of threads, four loads each on their way: 5.2 us for 18432 columns of 128 rows (with
// eight rows of threads and a barrier for each rank 12).
// ---------------------------------------------------------------------------------
struct ReduceArgs {
  const float* part[2];
  int rows[2];             // partial rows of each kind
  int nB, nC, nbias;       // columns: dB, dC, dbias
  int pq, r, bf16;
  const void* S;
  const void* A;
  float* dB;
  float* dA;
  float* dS;
  float* dbias;
};

// 32 rows of threads: thread y's share of a column's sum over `rows` (rows y, y + 32, ...; four loads on their way).
constexpr int kRedY = 32;
__device__ inline double column_part(const float* part, int rows, int64_t column, bool in, int y) {
  double s = 0.0;
  if (in) {
    const float* src = part + part_index(rows, 0, column);
    int g = y;
    for (; g + 3 * kRedY < rows; g += 4 * kRedY) {
      float u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = src[(int64_t)(g + kRedY * i) * kRedCols];
      s += ((double)u[0] + (double)u[1]) + ((double)u[2] + (double)u[3]);
    }
    for (; g < rows; g += kRedY) s += (double)src[(int64_t)g * kRedCols];
  }
  return s + __shfl_xor(s, 32, 64);      // (y and y + 1 stand in one wavefront)
}

__global__ __launch_bounds__(32 * kRedY) void glu_reduce_kernel(ReduceArgs a) {
  __shared__ double red[KRON_GLU_MAX_RANK][kRedY / 2][32];
  const int col = threadIdx.x & 31, y = threadIdx.x >> 5;
  auto total = [&](int i) {
    double t = 0.0;
#pragma unroll
    for (int k = 0; k < kRedY / 2; ++k) t += red[i][k][col];
    return t;
  };
  int b = blockIdx.x;
  const int bB = (a.nB + 31) / 32, bb = a.dbias ? (a.nbias + 31) / 32 : 0;
  if (b < bB + bb || !a.S) {
    // dB; then dbias, dA
    const int kind = b < bB ? 1 : 0, at = b < bB ? 0 : b < bB + bb ? a.nC : 0;
    const int c = 32 * (b < bB ? b : b < bB + bb ? b - bB : b - bB - bb) + col;
    const bool in = c < (b < bB ? a.nB : b < bB + bb ? a.nbias : a.nC);
    float* out = b < bB ? a.dB : b < bB + bb ? a.dbias : a.dA;
    red[0][y / 2][col] = column_part(a.part[kind], a.rows[kind], at + c, in, y);
    __syncthreads();
    if (y == 0 && in) out[c] = (float)total(0);
    return;
  }
  b -= bB + bb;
  const int per = (a.pq + 31) / 32, f = b / per, e = 32 * (b % per) + col;
  const bool in = e < a.pq;
  for (int i = 0; i < a.r; ++i)
    red[i][y / 2][col] = column_part(a.part[0], a.rows[0], ((int64_t)f * a.r + i) * a.pq + e, in, y);
  __syncthreads();
  double t = 0.0;      // thread y < r has rank y's dC; then its part of dS
  if (y < a.r && in) {
    const int64_t c = ((int64_t)f * a.r + y) * a.pq + e;
    t = total(y);
    a.dA[c] = (float)((double)raw(a.S, (int64_t)f * a.pq + e, a.bf16) * t);
    t *= (double)raw(a.A, c, a.bf16);
  }
  __syncthreads();
  if (y < a.r) red[y][0][col] = t;
  __syncthreads();
  if (!in || y != 0) return;
  double ds = 0.0;
  for (int i = 0; i < a.r; ++i) ds += red[i][0][col];
  a.dS[(int64_t)f * a.pq + e] = (float)ds;
}

struct Sizes {
  int parts_b, parts_c;
  int64_t lanes[4], bytes[4];
  int n4, groups[2], waves, share, pair_groups;
  int64_t off_d, off_part[2], fwd_bytes, bwd_bytes;
};

Sizes sizes_of(const GluArgs& a) {
  Sizes z{};
  z.parts_b = a.bf16 ? 1 : 3;
  z.parts_c = a.bf16 ? (a.S ? 2 : 1) : 3;
  const int dims[4][2] = {{a.m, a.n}, {a.p, a.q}, {a.n, a.m}, {a.q, a.p}};
  int64_t off = 0;
  for (int t = 0; t < 4; ++t) {
    z.lanes[t] = (int64_t)2 * a.r * ceil_div(dims[t][0], 32) * ceil_div(dims[t][1], 16) * 64;
    z.bytes[t] = z.lanes[t] * 16 * ((t & 1) ? z.parts_c : z.parts_b);
    off += z.bytes[t];
    if (t == 1) z.fwd_bytes = off;
  }
  z.n4 = (a.n + 3) & ~3;
  z.off_d = (off + 255) & ~int64_t(255);
  z.off_part[0] = z.off_d + ((2 * a.N * a.q * z.n4 * 4 + 255) & ~int64_t(255));
  // The parameters' kernel: one workgroup a CU, each with at least four rows where there are that many.  The
  // kinds get numbers of them by their products for a row and pair, and what staging and splitting it costs
  // either kind: as much as 150 products (by the products alone 8192 x (768 -> 2048) bf16 took 292 us and 8192 x
  // (1024 -> 2048) 546, so 274 and 515; half each 276 and 509, but r = 6 of 64 x 32 and 16 x 64 308, so 297).
  z.waves = param_waves(a.bf16, a.p > 32, a.n > 32, std::max(a.q, a.m) > 32);
  z.share = 1;
  while (2 * z.share * 2 * a.r <= z.waves) z.share *= 2;
  z.pair_groups = ceil_div(2 * a.r, z.waves / z.share);
  const int PT = ceil_div(a.p, 16), QT = ceil_div(a.q, 16), MT = ceil_div(a.m, 16), NT = ceil_div(a.n, 16);
  const int PK = ceil_div(a.p, 32), QK = ceil_div(a.q, 32), MK = ceil_div(a.m, 32), NK = ceil_div(a.n, 32);
  const int tb = a.bf16 ? 1 : 6, tc = a.bf16 ? (a.S ? 5 : 3) : 6, tx = a.bf16 ? 3 : 6;      // instructions of a product
  const double w0 = 150 + PT * 2 * NK * MK * tb + PT * QT * NK * 6, w1 = 150 + 2 * PK * NT * QK * tc + MT * NT * PK * tx;
  const int total = std::max(2, 256 / z.pair_groups);
  const int64_t most = (a.N + 3) / 4;
  z.groups[0] = std::min(std::max((int)(total * w0 / (w0 + w1) + 0.5), 1), total - 1);
  z.groups[1] = total - z.groups[0];
  for (int k = 0; k < 2; ++k) z.groups[k] = (int)std::max<int64_t>(1, std::min<int64_t>(z.groups[k], most));
  const int64_t PW0 = (int64_t)2 * a.r * a.p * a.q + 2 * a.q * a.n, PW1 = (int64_t)2 * a.r * a.m * a.n;
  z.off_part[1] = z.off_part[0] + ((part_floats(z.groups[0] * z.share, PW0) * 4 + 255) & ~int64_t(255));
  z.bwd_bytes = z.off_part[1] + part_floats(z.groups[1] * z.share, PW1) * 4;
  return z;
}

hipError_t launch_pack(const GluArgs& a, const Sizes& z, int tables, u4* const t[4], hipStream_t s) {
  PackArgs k{a.p, a.q, a.m, a.n, a.r, a.bf16, z.parts_b, z.parts_c, tables, a.S, a.A, a.B, {}, {}};
  int64_t total = 0;
  for (int i = 0; i < tables; ++i) {
    k.t[i] = t[i];
    k.lanes[i] = (int)z.lanes[i];
    total += z.lanes[i];
  }
  hipLaunchKernelGGL(glu_pack_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, s, k);
  return hipGetLastError();
}

}  // namespace

size_t glu_workspace_bytes(const GluArgs& a, bool backward) {
  const Sizes z = sizes_of(a);
  return (size_t)(backward ? z.bwd_bytes : z.fwd_bytes);
}

hipError_t launch_glu_fwd(const GluArgs& a, void* ws, hipStream_t s) {
  const Sizes z = sizes_of(a);
  u4* t[4] = {(u4*)ws, (u4*)((char*)ws + z.bytes[0]), nullptr, nullptr};
  hipError_t e = launch_pack(a, z, 2, t, s);
  if (e != hipSuccess) return e;
  GluRows k{};
  k.N = a.N; k.p = a.p; k.q = a.q; k.m = a.m; k.n = a.n; k.r = a.r;
  k.ldm = a.m; k.ldx = (int64_t)a.p * a.m; k.act = a.act;
  k.x[0] = k.x[1] = a.x; k.tb = t[0]; k.tc = t[1]; k.bias = a.bias; k.y = a.y; k.n4 = z.n4;
  return launch_glu_rows0(k, a.bf16, a.S != nullptr, s);
}

hipError_t launch_glu_bwd(const GluArgs& a, void* ws, hipStream_t s) {
  const Sizes z = sizes_of(a);
  char* w = (char*)ws;
  u4* t[4];
  for (int i = 0; i < 4; ++i) {
    t[i] = (u4*)w;
    w += z.bytes[i];
  }
  float* d = (float*)((char*)ws + z.off_d);
  hipError_t e = launch_pack(a, z, 4, t, s);
  if (e != hipSuccess) return e;
  float* d2 = d + a.N * a.q * z.n4;
  if (a.N > 0) {
    GluRows k{};
    k.N = a.N; k.p = a.p; k.q = a.q; k.m = a.m; k.n = a.n; k.r = a.r;
    k.ldm = a.m; k.ldx = (int64_t)a.p * a.m; k.act = a.act;
    k.x[0] = k.x[1] = a.x; k.tb = t[0]; k.tc = t[1]; k.bias = a.bias; k.dy = a.dy;
    k.d[0] = d; k.d[1] = d2; k.n4 = z.n4;
    e = launch_glu_rows1(k, a.bf16, a.S != nullptr, s);
    if (e != hipSuccess) return e;
    if (a.dx) {
      GluRows x{};
      x.N = a.N; x.p = a.q; x.q = a.p; x.m = a.n; x.n = a.m; x.r = a.r;
      x.ldm = z.n4; x.ldx = (int64_t)a.q * z.n4; x.n4 = (a.m + 3) & ~3;
      x.x[0] = d; x.x[1] = d2; x.tb = t[2]; x.tc = t[3]; x.y = a.dx;
      e = launch_glu_rows2(x, a.bf16, a.S != nullptr, s);
      if (e != hipSuccess) return e;
    }
  }
  GluParam k{};
  k.N = a.N; k.p = a.p; k.q = a.q; k.m = a.m; k.n = a.n; k.r = a.r; k.n4 = z.n4;
  k.x = a.x; k.d[0] = d; k.d[1] = d2; k.tb = t[0]; k.tc = t[3];
  for (int i = 0; i < 2; ++i) k.part[i] = (float*)((char*)ws + z.off_part[i]);
  k.share = z.share;
  k.pair_groups = z.pair_groups;
  for (int i = 0; i < 2; ++i) k.groups[i] = z.groups[i];
  e = !a.bf16 ? launch_glu_param_f32(k, s) : a.S ? launch_glu_param_bf16_S(k, s) : launch_glu_param_bf16(k, s);
  if (e != hipSuccess) return e;
  ReduceArgs ra{};
  for (int i = 0; i < 2; ++i) {
    ra.part[i] = k.part[i];
    ra.rows[i] = z.groups[i] * z.share;
  }
  ra.pq = a.p * a.q; ra.r = a.r; ra.bf16 = a.bf16;
  ra.nB = 2 * a.r * a.m * a.n; ra.nC = 2 * a.r * ra.pq; ra.nbias = 2 * a.q * a.n;
  ra.S = a.S; ra.A = a.A; ra.dB = a.dB; ra.dA = a.dA; ra.dS = a.dS; ra.dbias = a.dbias;
  const int blocks = ceil_div(ra.nB, 32) + (a.dbias ? ceil_div(ra.nbias, 32) : 0) +
                     (a.S ? 2 * ceil_div(ra.pq, 32) : ceil_div(ra.nC, 32));
  hipLaunchKernelGGL(glu_reduce_kernel, dim3((unsigned)blocks), dim3(32 * kRedY), 0, s, ra);
  return hipGetLastError();
}

}  // namespace kron
