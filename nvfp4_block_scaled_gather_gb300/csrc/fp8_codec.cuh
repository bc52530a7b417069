// The codec of 8-bit rows (moe_dense.h): e4m3 codes under a power of two for
// each 128 values.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "moe_dense.h"

namespace moe {

constexpr uint32_t kNoScale = 127;  // the byte of 2^0, for scales past the last block

// Two values of a 16-bit type, the first in the low half.
template <int kType>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (kType == MOE_BF16) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  } else {
    __half2 h;
    *reinterpret_cast<uint32_t*>(&h) = v;
    return __half22float2(h);
  }
}
template <int kType>
__device__ __forceinline__ uint32_t pack16x2(float a, float b) {
  if constexpr (kType == MOE_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// A value's part in its block's largest magnitude: infinities and NaN have none.
__device__ __forceinline__ float finite_size(float v) {
  const float a = fabsf(v);
  return a < INFINITY ? a : 0.0f;
}

// The scale's byte: the smallest power of two, from 2^-127 on, times 448 =
// 1.75 * 2^8 that holds amax = 1.m * 2^(E - 127).
__device__ __forceinline__ uint32_t e8m0_of(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e > 0 ? (uint32_t)e : 0u;
}
// One over the scale, exactly (a byte of e8m0_of is at most 247).
__device__ __forceinline__ float e8m0_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Codes of two and four values, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) { return e4m3x2(a.x, a.y) | (e4m3x2(b.x, b.y) << 16); }
// The same over a scale. The product is exact up to fp32's smallest values, so
// a code is rounded once. (An infinity would become the largest code: times 0
// first it is NaN.)
__device__ __forceinline__ uint32_t e4m3x2_of(float a, float b, float inverse) {
  return e4m3x2(fmaf(a, inverse, a * 0.0f), fmaf(b, inverse, b * 0.0f));
}
__device__ __forceinline__ uint32_t e4m3x4_of(float a, float b, float c, float d, float inverse) {
  return e4m3x2_of(a, b, inverse) | (e4m3x2_of(c, d, inverse) << 16);
}

// The largest finite magnitude of 2 kWords 16-bit values each of kWidth threads next to each other, as fp32. By whole
// warps.
template <int kType, int kWidth, int kWords>
__device__ __forceinline__ float finite_block_max(const uint32_t (&w)[kWords]) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    const float2 v = unpack2<kType>(w[i]);
    amax = fmaxf(amax, fmaxf(finite_size(v.x), finite_size(v.y)));
  }
#pragma unroll
  for (int o = 1; o < kWidth; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  return amax;
}
// The same with infinities and NaN counted: then it is one of them. Magnitudes are compared as whole numbers, two at a
// time.
template <int kType, int kWidth, int kWords>
__device__ __forceinline__ uint32_t block_max_bits(const uint32_t (&w)[kWords]) {
  constexpr uint32_t kMagnitude = 0x7fff7fffu;
  uint32_t m = w[0] & kMagnitude;
#pragma unroll
  for (int i = 1; i < kWords; ++i) m = __vmaxu2(m, w[i] & kMagnitude);
#pragma unroll
  for (int o = 1; o < kWidth; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(~0u, m, o));
  return max(m & 0xffffu, m >> 16);
}
template <int kType>
constexpr uint32_t kInfinityBits = kType == MOE_BF16 ? 0x7f80u : 0x7c00u;

// The codes of four 16-bit values over a scale.
template <int kType>
__device__ __forceinline__ uint32_t e4m3x4_of(uint32_t lo, uint32_t hi, float inverse) {
  const float2 a = unpack2<kType>(lo), b = unpack2<kType>(hi);
  return e4m3x4_of(a.x, a.y, b.x, b.y, inverse);
}

}  // namespace moe
