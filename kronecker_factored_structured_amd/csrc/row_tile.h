// A row of logits as 16-byte vectors, shared by the kernels over a vocabulary (distill.hip,
// topk_logits.hip).
//
// A vocabulary is rarely a multiple of eight and rows may be padded, so a row starts at any
// element.  The row is covered by the 16-byte aligned vectors that overlap it: vector j holds
// the elements [j*VE - off, (j+1)*VE - off), off = elements from the last 16-byte boundary to
// the row's start.  Vectors wholly inside the row move as one 16-byte access; the (at most two)
// vectors that cross an end of the row move element by element, so nothing outside the row is
// read or written.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace kron {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ inline float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// fp32 -> bf16, nearest even; a NaN stays a NaN
__device__ inline uint32_t bf16_rne(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
// two of them, a in the low half (one conversion instruction)
__device__ inline uint32_t bf16_pair(float a, float b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, b2{(__bf16)a, (__bf16)b});
}

// float or bf16 (a 16-bit pattern) as stored.
template <bool BF>
struct RowTile {
  static constexpr int VE = BF ? 8 : 4;       // elements of a vector
  static constexpr int ES = BF ? 2 : 4;       // bytes of an element
  char* base;      // address of vector 0 (16-byte aligned, at or before the row's start)
  int off;         // elements of vector 0 before the row
  int V;

  __device__ RowTile(const void* p, int64_t row, int64_t ld, int V_) : V(V_) {
    const uint64_t a = (uint64_t)p + (uint64_t)row * (uint64_t)ld * ES;
    base = (char*)(a & ~uint64_t(15));
    off = (int)(a & 15) / ES;
  }
  __device__ int vectors() const { return (V + off + VE - 1) / VE; }
  __device__ int first(int j) const { return j * VE - off; }   // element index of vector j's first value
  __device__ bool inside(int j) const {
    const int e = first(j);
    return e >= 0 && e + VE <= V;
  }
  static __device__ u32x4 empty() {      // -infinity in every element
    u32x4 r;
#pragma unroll
    for (int w = 0; w < 4; ++w) r[w] = BF ? 0xff80ff80u : 0xff800000u;
    return r;
  }
  // Vector j if it is wholly inside the row, else -infinity throughout.  Loads and stores of whole vectors are
  // non-temporal: rows stream through once (loss and gradient of 8192 x 50257 bf16 446 -> 415 us, of 2050 x 32003
  // fp32 207 -> 184, its gradient alone 163 -> 149; stores alone 436, 201 and 174; the top of 8192 x 50257 275 -> 250).
  __device__ u32x4 whole(int j) const {
    return inside(j) ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(base + (uint32_t)(j * 16))) : empty();
  }
  __device__ void store(int j, const u32x4& v) const {      // inside the row
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(base + (uint32_t)(j * 16)));
  }
  // Vector j; elements outside the row are -infinity.  (An ordinary load: what is read again.)
  __device__ u32x4 load(int j) const {
    if (inside(j)) return *reinterpret_cast<const u32x4*>(base + (uint32_t)(j * 16));
    u32x4 r = empty();
    const int e = first(j);
    if (e >= V || e + VE <= 0) return r;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      if (e + i >= 0 && e + i < V) {
        if (BF) {
          const uint32_t h = *reinterpret_cast<const uint16_t*>(base + (uint32_t)(j * 16) + 2 * i);
          r[i / 2] = (i & 1) ? ((r[i / 2] & 0xffffu) | (h << 16)) : ((r[i / 2] & 0xffff0000u) | h);
        } else {
          r[i & 3] = *reinterpret_cast<const uint32_t*>(base + (uint32_t)(j * 16) + 4 * i);
        }
      }
    }
    return r;
  }
  // Vectors [j0, j1) of the row into the registers of NT threads, vector j0 + tid + i NT in reg[i]
  // (-infinity from j1 on).  Only the row's first and last vector can be partial: they are loaded
  // apart, once, not in every step of the loop.
  template <int NT, int NV>
  __device__ void fetch(u32x4 (&reg)[NV], int tid, int j0, int j1) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = j0 + tid + i * NT;
      reg[i] = j < j1 ? whole(j) : empty();
    }
    const int last = vectors() - 1;
    if (j0 == 0 && off != 0 && tid == 0) reg[0] = load(0);
    if (!inside(last) && last >= j0 && last < j1) {
      const int il = (last - j0) / NT, tl = (last - j0) % NT;
      u32x4 v = empty();
      if (tid == tl) v = load(last);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i == il && tid == tl) reg[i] = v;
    }
  }
  static __device__ float value(const u32x4& v, int i) {
    if (BF) return (i & 1) ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]);
    return __uint_as_float(v[i & 3]);
  }
  static __device__ void values(const u32x4& v, float (&x)[VE]) {
#pragma unroll
    for (int i = 0; i < VE; ++i) x[i] = value(v, i);
  }
  static __device__ u32x4 packed(const float (&x)[VE]) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = BF ? bf16_pair(x[(2 * i) % VE], x[(2 * i + 1) % VE]) : __float_as_uint(x[i % VE]);
    return r;
  }
  // One value of the row.
  __device__ float at(int e) const {
    if (BF) return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(base + (uint32_t)((e + off) * 2)) << 16);
    return *reinterpret_cast<const float*>(base + (uint32_t)((e + off) * 4));
  }
  __device__ void put(int e, float f) const {
    if (BF)
      *reinterpret_cast<uint16_t*>(base + (uint32_t)((e + off) * 2)) = (uint16_t)bf16_rne(f);
    else
      *reinterpret_cast<float*>(base + (uint32_t)((e + off) * 4)) = f;
  }
};

// The packed row as new values: what one pass unpacked is not kept for the next (it would take
// twice the row's registers or more).
template <int NV>
__device__ inline void fresh(u32x4 (&reg)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) asm volatile("" : "+v"(reg[i]));
}

// Reductions over a workgroup of NW wavefronts; every thread gets the result.  `red` holds NW
// values and may be used again after the next barrier.
__device__ inline float wave_max(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o /= 2) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o /= 2) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ inline double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o /= 2) v += __shfl_xor(v, o, 64);
  return v;
}

}  // namespace kron
