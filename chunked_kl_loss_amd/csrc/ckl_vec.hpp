// What the kernels on rows of vectors share: loads and stores of eight or four
// elements as floats, sums over a wave or a workgroup, rows cut into units, and
// the 8-bit form of 32 columns.
#pragma once

#include <type_traits>

#include "ckl_common.hpp"

namespace ckl {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Eight consecutive elements (16-byte aligned) as floats, and back with one
// rounding.
__device__ __forceinline__ void load8(const bf16_t* p, float* f) {
  const u32x4 v = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* f) {
  const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = a[i];
    f[4 + i] = b[i];
  }
}
__device__ __forceinline__ void store8(bf16_t* p, const float* f) {
  *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                       pack_bf16x2(f[6], f[7])};
}
__device__ __forceinline__ void store8(float* p, const float* f) {
  reinterpret_cast<f32x4*>(p)[0] = f32x4{f[0], f[1], f[2], f[3]};
  reinterpret_cast<f32x4*>(p)[1] = f32x4{f[4], f[5], f[6], f[7]};
}
__device__ __forceinline__ void store4(bf16_t* p, f32x4 v) {
  *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}
__device__ __forceinline__ void store4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
// The same without a place in the caches for what is written: for outputs larger
// than they are (embedding of 32768 x 2880: 71 -> 56 us).
__device__ __forceinline__ void stream8(bf16_t* p, const float* f) {
  const u32x4 v = {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
}
__device__ __forceinline__ void stream8(float* p, const float* f) {
  __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f32x4*>(p));
  __builtin_nontemporal_store(f32x4{f[4], f[5], f[6], f[7]}, reinterpret_cast<f32x4*>(p) + 1);
}
// Four elements.
__device__ __forceinline__ void load4(const bf16_t* p, float* f) {
  const u32x2 v = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load4(const float* p, float* f) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = a[i];
}
// Four elements that nothing else will read.
__device__ __forceinline__ void load4_once(const bf16_t* p, float* f) {
  const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load4_once(const float* p, float* f) {
  const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = a[i];
}
// A weight of either type, eight columns.
__device__ __forceinline__ void load8_any(const void* p, int is_bf16, int64_t at, float* f) {
  if (is_bf16)
    load8(reinterpret_cast<const bf16_t*>(p) + at, f);
  else
    load8(reinterpret_cast<const float*>(p) + at, f);
}

__device__ __forceinline__ float wave_sum_f(float x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

// Inclusive sums over the wave, lane by lane.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);  // from 1, 2, 4, 8 lanes below in the row of 16
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row ends into rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // lane 31 into rows 2 and 3
  return x;
}

// Rows of n units each, cut into runs of consecutive units: the row and column
// of unit base + off, for off below a few thousand and base below 2^40.
struct Units {
  uint32_t n;
  uint64_t m64;  // 2^64 / n rounded up (n > 1): base / n is the high word of base m64
  uint32_t m32;  // the same for 32 bits
};
__device__ __forceinline__ void unit_at(const Units& q, int64_t base, uint32_t off, int64_t* row, uint32_t* col) {
  if (q.n == 1) {
    *row = base + off;
    *col = 0;
    return;
  }
  const uint64_t r0 = __umul64hi((uint64_t)base, q.m64);
  const uint32_t u = (uint32_t)((uint64_t)base - r0 * q.n) + off;
  const uint32_t r = __umulhi(u, q.m32);
  *row = (int64_t)(r0 + r);
  *col = u - r * q.n;
}
inline Units units(int64_t n) {
  Units q{(uint32_t)n, 0, 0};
  if (n > 1) {
    q.m64 = ~(uint64_t)0 / (uint64_t)n + 1;
    q.m32 = (uint32_t)((((uint64_t)1 << 32) / (uint64_t)n) + 1);
  }
  return q;
}

// Sum over the workgroup, in every thread.  `slots` holds one float per wave.
__device__ __forceinline__ float group_sum(float x, float* slots) {
  x = wave_sum_f(x);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return x;
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = x;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < waves; ++w) s += slots[w];
  __syncthreads();
  return s;
}

// ------------------------------------------------------- 8 bits a value --
// Blocks of 32 columns of a row share a power of two 2^(E - 127), the smallest
// that brings the block's largest magnitude below 127.5, kept within 2^-126 and
// 2^121 (127 steps of a larger one are no float); a code is the value divided
// by it, rounded to the nearest whole number, ties to even, at most 127.
// Multiplying by powers of two is exact, so a code depends on nothing but its
// block, and a restored value (7 bits and a sign) is exact in bf16.
// E = 255 marks a block that holds an infinity or a NaN: all of it restores to
// NaN.
__device__ __forceinline__ uint32_t top_bits(const float* f) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(f[i]) & 0x7fffffffu;  // as integers, NaN > inf > finite
    a = b > a ? b : a;
  }
  return a;
}
__device__ __forceinline__ uint32_t block_exponent(uint32_t top) {
  uint32_t o = __shfl_xor(top, 1);
  top = o > top ? o : top;
  o = __shfl_xor(top, 2);
  top = o > top ? o : top;
  if (top >= 0x7f800000u) return 255;
  // adding 2^16 carries into the exponent exactly when top >= 127.5 / 64 of its power of two
  const int e = (int)((top + 0x10000u) >> 23) - 6;
  return e < 1 ? 1u : e > 248 ? 248u : (uint32_t)e;
}
__device__ __forceinline__ u32x2 encode8(const float* f, uint32_t e) {
  if (e == 255) return u32x2{0, 0};
  const float inv = __uint_as_float((254u - e) << 23);
  u32x2 c = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int v = (int)fminf(fmaxf(rintf(f[i] * inv), -127.f), 127.f);  // past 127 only at E = 248
    c[i >> 2] |= ((uint32_t)v & 255u) << (8 * (i & 3));
  }
  return c;
}
__device__ __forceinline__ float block_step(uint32_t e) {
  return e == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(e << 23);
}
__device__ __forceinline__ void decode8(u32x2 c, float step, float* f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = (float)(int)(int8_t)(c[i >> 2] >> (8 * (i & 3))) * step;
}

}  // namespace ckl
