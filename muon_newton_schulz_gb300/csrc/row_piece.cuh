// How the kernels that move rows take them: 16 bytes at a time, or less where
// the rows are no multiple of that.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "train_internal.h"

namespace muon {

// What a thread moves at once: 16 bytes where the row length and all addresses
// are multiples of 16 bytes; else kMost units, a row of threads apart, of 4
// bytes or of one element of an odd row of bf16.  Four in flight are faster than
// one or eight for dispatch and combine (16384 x 4 rows of 2047 bf16: combine
// 108 us against 130 and 126; 2048 wide 60), one for the backward pass, which
// has more rows in flight anyway (169 us against 184 and 223; 2048 wide 97).
// A thread starts at first() and goes on kStep * tx elements later.
template <typename T, int kBytes, int kMost = kRowUnits> struct Piece {
  static constexpr int kUnit = kBytes / sizeof(T), kUnits = kBytes == 16 ? 1 : kMost;
  static constexpr int N = kUnit * kUnits, kStep = N;
  static constexpr int kWords = kBytes == 16 ? 4 : 1;   // registers of a unit
  uint32_t raw[kUnits][kWords];
  static __device__ __forceinline__ int64_t first(int thread) { return (int64_t)thread * kUnit; }
  __device__ __forceinline__ void load(const T* row, int64_t c, int64_t end, int tx) {
    if constexpr (kBytes == 16) {
      const uint4 t = *reinterpret_cast<const uint4*>(row + c);
      raw[0][0] = t.x; raw[0][1] = t.y; raw[0][2] = t.z; raw[0][3] = t.w;
    } else {
#pragma unroll
      for (int q = 0; q < kUnits; ++q) {
        const int64_t e = c + q * (tx * kUnit);
        raw[q][0] = 0u;
        if (kUnits == 1 || e < end) {   // the caller has looked at the first
          if constexpr (kBytes == 4) raw[q][0] = *reinterpret_cast<const uint32_t*>(row + e);
          else raw[q][0] = *reinterpret_cast<const uint16_t*>(row + e);
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* row, int64_t c, int64_t end, int tx) const {
    if constexpr (kBytes == 16) {
      *reinterpret_cast<uint4*>(row + c) = make_uint4(raw[0][0], raw[0][1], raw[0][2], raw[0][3]);
    } else {
#pragma unroll
      for (int q = 0; q < kUnits; ++q) {
        const int64_t e = c + q * (tx * kUnit);
        if (kUnits == 1 || e < end) {   // the caller has looked at the first
          if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(row + e) = raw[q][0];
          else *reinterpret_cast<uint16_t*>(row + e) = (uint16_t)raw[q][0];
        }
      }
    }
  }
  __device__ __forceinline__ void get(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < kUnits * kWords; ++i) {
      const uint32_t w = raw[i / kWords][i % kWords];
      if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w);
      else if constexpr (kBytes == 2) v[i] = __uint_as_float(w << 16);
      else {
        v[2 * i] = __uint_as_float(w << 16);
        v[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void set(const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < kUnits * kWords; ++i) {
      uint32_t& w = raw[i / kWords][i % kWords];
      if constexpr (sizeof(T) == 4) w = __float_as_uint(v[i]);
      else if constexpr (kBytes == 2) w = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
      else {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w = *reinterpret_cast<const uint32_t*>(&t);
      }
    }
  }
};

// Calls f with the element type and the bytes that a thread moves at once.
template <typename T, int kBytes> struct Kind {
  using Type = T;
  static constexpr int bytes = kBytes;
};
template <typename F>
int with_kind(bool bf16, int bytes, F f) {
  if (!bf16) return bytes == 16 ? f(Kind<float, 16>()) : f(Kind<float, 4>());
  if (bytes == 16) return f(Kind<__nv_bfloat16, 16>());
  return bytes == 4 ? f(Kind<__nv_bfloat16, 4>()) : f(Kind<__nv_bfloat16, 2>());
}

}  // namespace muon
