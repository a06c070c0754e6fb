// Activations kept in 8 bits between the forward and the backward pass: e4m3
// codes, with a power of two for each 32 elements of a row (see code8.cuh).
// One pass over the data each way, bound by HBM: 16384 x 16384 bf16 there and back 245 us,
// 99 % of a plain copy's rate.  1003 x 1001 fp32 (rows off their boundaries): 5.9 and 5.2 us.
#include <cuda_runtime.h>

#include <type_traits>

#include "code8.cuh"
#include "launch_util.cuh"
#include "layer_internal.h"

namespace muon {

namespace {

// Eight consecutive elements, 16 or 32 bytes.
template <typename T> struct Eight {
  uint4 raw[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* x) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) raw[i] = reinterpret_cast<const uint4*>(x)[i];
  }
  __device__ __forceinline__ void store(T* x) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(x)[i] = raw[i];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
      else v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    uint32_t* w = reinterpret_cast<uint32_t*>(raw);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      if constexpr (sizeof(T) == 4) {
        w[i] = __float_as_uint(v[i]);
        w[i + 1] = __float_as_uint(v[i + 1]);
      } else {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[i], v[i + 1]);
        w[i / 2] = *reinterpret_cast<const uint32_t*>(&t);
      }
    }
  }
};

constexpr int kAhead = 4;   // groups of eight that a thread has in flight

// Where group i of eight elements begins.
__device__ __forceinline__ int64_t begin_of(const Saved8Params& p, int64_t i) {
  if (p.rows == 1) return i * 8;
  const int64_t per_row = p.cols / 8;
  return i / per_row * p.ldx + i % per_row * 8;
}

// Rows of a multiple of 32 elements on 16-byte boundaries: four lanes share a
// block, eight elements each.
template <typename T, bool kSpecial>
__global__ void __launch_bounds__(kThreads256) k_pack8(const __grid_constant__ Saved8Params p) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t n = p.rows * (p.cols / 8);
  const int64_t step = (int64_t)gridDim.x * (kThreads256 * kAhead);
  for (int64_t i0 = (int64_t)blockIdx.x * (kThreads256 * kAhead) + threadIdx.x; i0 - threadIdx.x < n; i0 += step) {
    Eight<T> r[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int64_t i = i0 + q * kThreads256;
      if (i < n) r[q].load(static_cast<const T*>(p.x) + begin_of(p, i));
      else r[q] = Eight<T>{};
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int64_t i = i0 + q * kThreads256;
      float v[8];
      r[q].get(v);
      uint32_t most = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) most = max(most, finite_bits(v[j]));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
      if (i >= n) continue;
      const uint32_t c = scale_byte(most);
      const float up = scale_up(c);
      uint2 w;
      w.x = encode2<kSpecial>(v[0], v[1], up) | encode2<kSpecial>(v[2], v[3], up) << 16;
      w.y = encode2<kSpecial>(v[4], v[5], up) | encode2<kSpecial>(v[6], v[7], up) << 16;
      reinterpret_cast<uint2*>(p.codes)[i] = w;
      if ((threadIdx.x & 3) == 0) p.scales[i / 4] = (uint8_t)c;
    }
  }
}

template <typename T, bool kSpecial>
__global__ void __launch_bounds__(kThreads256) k_unpack8(const __grid_constant__ Saved8Params p) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t n = p.rows * (p.cols / 8);
  const int64_t step = (int64_t)gridDim.x * (kThreads256 * kAhead);
  for (int64_t i0 = (int64_t)blockIdx.x * (kThreads256 * kAhead) + threadIdx.x; i0 < n; i0 += step) {
    uint2 w[kAhead];
    uint32_t c[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int64_t i = i0 + q * kThreads256;
      if (i >= n) break;
      w[q] = reinterpret_cast<const uint2*>(p.codes)[i];
      c[q] = p.scales[i / 4];
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int64_t i = i0 + q * kThreads256;
      if (i >= n) break;
      const float s = scale_down(c[q]);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = decode2<kSpecial>((j < 2 ? w[q].x : w[q].y) >> (j & 1 ? 16 : 0));
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
      }
      Eight<T> r;
      r.set(v);
      r.store(static_cast<T*>(p.x) + begin_of(p, i));
    }
  }
}

// Any other rows: a warp for each block, a lane for each element.
template <typename T, bool kSpecial>
__global__ void __launch_bounds__(kThreads256) k_pack8_any(const __grid_constant__ Saved8Params p) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const int64_t blocks = (p.cols + kSaved8Block - 1) / kSaved8Block, n = p.rows * blocks;
  const int64_t warps = (int64_t)gridDim.x * (kThreads256 / 32);
  for (int64_t b0 = ((int64_t)blockIdx.x * (kThreads256 / 32) + (threadIdx.x >> 5)) * kAhead; b0 < n; b0 += warps * kAhead) {
    float v[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int64_t b = b0 + q, row = b / blocks, col = b % blocks * kSaved8Block + lane;
      v[q] = b < n && col < p.cols ? (float)static_cast<const T*>(p.x)[row * p.ldx + col] : 0.f;
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int64_t b = b0 + q, row = b / blocks, col = b % blocks * kSaved8Block + lane;
      if (b >= n) break;
      const uint32_t c = scale_byte(__reduce_max_sync(0xffffffffu, finite_bits(v[q])));
      if (col < p.cols) p.codes[row * p.cols + col] = (uint8_t)encode2<kSpecial>(v[q], 0.f, scale_up(c));
      if (lane == 0) p.scales[b] = (uint8_t)c;
    }
  }
}

template <typename T, bool kSpecial>
__global__ void __launch_bounds__(kThreads256) k_unpack8_any(const __grid_constant__ Saved8Params p) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const int64_t blocks = (p.cols + kSaved8Block - 1) / kSaved8Block, n = p.rows * blocks;
  const int64_t warps = (int64_t)gridDim.x * (kThreads256 / 32);
  for (int64_t b0 = ((int64_t)blockIdx.x * (kThreads256 / 32) + (threadIdx.x >> 5)) * kAhead; b0 < n; b0 += warps * kAhead) {
    uint32_t w[kAhead], c[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int64_t b = b0 + q, row = b / blocks, col = b % blocks * kSaved8Block + lane;
      const bool has = b < n && col < p.cols;
      w[q] = has ? p.codes[row * p.cols + col] : 0u;
      c[q] = has ? p.scales[b] : 0u;
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int64_t b = b0 + q, row = b / blocks, col = b % blocks * kSaved8Block + lane;
      if (b < n && col < p.cols) static_cast<T*>(p.x)[row * p.ldx + col] = (T)(decode2<kSpecial>(w[q]).x * scale_down(c[q]));
    }
  }
}

// The form of a call: rows that follow one another without a gap and end with a
// block are one long row; `vec` where all accesses fall on their boundaries.
struct Form {
  Saved8Params p;
  bool vec;
  dim3 grid;
};

Form form_of(Saved8Params p, int64_t es) {
  if (p.rows == 1) p.ldx = p.cols;
  if (p.ldx == p.cols && p.cols % kSaved8Block == 0) {
    p.cols = p.ldx = p.rows * p.cols;
    p.rows = 1;
  }
  auto on = [](const void* at, int64_t bytes) { return reinterpret_cast<uintptr_t>(at) % (uintptr_t)bytes == 0; };
  const bool vec = p.cols % kSaved8Block == 0 && on(p.x, 16) && (p.rows == 1 || p.ldx * es % 16 == 0) && on(p.codes, 8);
  const int64_t per = vec ? 8 * kAhead * kThreads256 : kAhead * kThreads256 / 32;   // elements, or blocks, of a CTA
  const int64_t n = vec ? p.rows * p.cols : p.rows * ((p.cols + kSaved8Block - 1) / kSaved8Block);
  const int64_t ctas = (n + per - 1) / per, most = 152 * 32;
  return {p, vec, dim3((unsigned)(ctas < most ? ctas : most))};
}

}  // namespace

int launch_pack8(const Saved8Params& p, bool bf16, void* stream, bool pdl) {
  const Form f = form_of(p, bf16 ? 2 : 4);
  auto launch = [&](auto* k) { return launch_kernel(k, f.grid, dim3(kThreads256), 0, stream, pdl, f.p); };
  auto kind = [&](auto special) {
    constexpr bool kSpecial = decltype(special)::value;
    return launch(f.vec ? bf16 ? k_pack8<__nv_bfloat16, kSpecial> : k_pack8<float, kSpecial> : bf16 ? k_pack8_any<__nv_bfloat16, kSpecial> : k_pack8_any<float, kSpecial>);
  };
  return p.special ? kind(std::true_type()) : kind(std::false_type());
}

int launch_unpack8(const Saved8Params& p, bool bf16, void* stream, bool pdl) {
  const Form f = form_of(p, bf16 ? 2 : 4);
  auto launch = [&](auto* k) { return launch_kernel(k, f.grid, dim3(kThreads256), 0, stream, pdl, f.p); };
  auto kind = [&](auto special) {
    constexpr bool kSpecial = decltype(special)::value;
    return launch(f.vec ? bf16 ? k_unpack8<__nv_bfloat16, kSpecial> : k_unpack8<float, kSpecial> : bf16 ? k_unpack8_any<__nv_bfloat16, kSpecial> : k_unpack8_any<float, kSpecial>);
  };
  return p.special ? kind(std::true_type()) : kind(std::false_type());
}

}  // namespace muon
