// e4m3 codes of blocks of 32 elements under a power of two.
//
// The scale byte of a block is c = max(E - 7, 1), E the biased fp32 exponent of
// its largest finite magnitude, and stands for 2^(c - 127): scaled values stay
// below 256, so that rounding to nearest never leaves e4m3 (448), and scaling is
// exact.  A value that is not finite becomes NaN and leaves its block alone; with kSpecial
// infinities take the largest codes, which no finite value has, a finite value's code never
// stands for 2^128, and one that is not zero never has zero's.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace muon {

// The bits of |v| where v is finite, else 0: their maximum gives the scale.
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
__device__ __forceinline__ uint32_t scale_byte(uint32_t most) {
  const int e = (int)(most >> 23) - 7;
  return (uint32_t)(e > 1 ? e : 1);
}
// 2^(127 - c) of a scale byte that scale_byte gave (1 .. 247)
__device__ __forceinline__ float scale_up(uint32_t c) { return __uint_as_float((254u - c) << 23); }
// 2^(c - 127) of any scale byte; 255 stands for NaN
__device__ __forceinline__ float scale_down(uint32_t c) {
  return c == 0u ? __uint_as_float(0x00400000u) : c == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(c << 23);
}

// What the conversion gets for v if its code is to be of v's kind.
__device__ __forceinline__ float of_its_kind(float v, float up) {
  const float a = v * up, m = fabsf(a);
  if (m < 0.001953125f && v != 0.f) return copysignf(0.001953125f, v);   // 2^-9, the smallest code
  if (up == scale_up(247u) && m > 240.f && m < 256.f) return copysignf(240.f, v);
  return a;
}

// Codes of two values, lo in the lower byte.  The conversion takes infinities to
// the largest codes: without kSpecial they are made NaN first.
template <bool kSpecial = false> __device__ __forceinline__ uint32_t encode2(float lo, float hi, float up) {
  const float nan = __uint_as_float(0x7fc00000u);
  const float a = kSpecial ? of_its_kind(lo, up) : fabsf(lo) < __uint_as_float(0x7f800000u) ? lo * up : nan;
  const float b = kSpecial ? of_its_kind(hi, up) : fabsf(hi) < __uint_as_float(0x7f800000u) ? hi * up : nan;
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// Values of two codes before their scale: every e4m3 number is an fp16 number.
template <bool kSpecial = false> __device__ __forceinline__ float2 decode2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  if constexpr (kSpecial) {
    const float inf = __uint_as_float(0x7f800000u);
    if (fabsf(f.x) == 448.f) f.x = copysignf(inf, f.x);
    if (fabsf(f.y) == 448.f) f.y = copysignf(inf, f.y);
  }
  return f;
}

// ---- the same in 16 bits: fp16 numbers under c = max(E - 14, 1), so that the block's
// largest lies in [2^14, 2^15]: eight times as exact as bf16 in as many bytes, over
// fp32's range.  Infinities stay what they are.
__device__ __forceinline__ uint32_t scale_byte16(uint32_t most) {
  const int e = (int)(most >> 23) - 14;
  return (uint32_t)(e > 1 ? e : 1);
}
__device__ __forceinline__ uint32_t encode16(float lo, float hi, float up) {
  const __half2 h = __floats2half2_rn(lo * up, hi * up);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 decode16(uint32_t codes) { return __half22float2(*reinterpret_cast<const __half2*>(&codes)); }

}  // namespace muon
