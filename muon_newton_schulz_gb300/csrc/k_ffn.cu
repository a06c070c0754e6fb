// Gated feed-forward products on fp32 arithmetic, for every type, size and
// stride.
//
// The tokens of an expert are consecutive rows.  A CTA computes 64 x 64 elements
// of a product: both operands pass through shared memory 16 deep, each of 256
// threads sums 4 x 4.  The products over rows take their tiles from the counts on
// the device; a weight's gradient sums over the rows of its expert.
#include <cuda_runtime.h>

#include "code8.cuh"
#include "ffn_act.cuh"
#include "launch_util.cuh"
#include "train_internal.h"

namespace muon {

namespace {

constexpr int kTile = 64, kDeep = 16, kPer = 4;

template <typename T> __device__ __forceinline__ float at(const FfnStack& s, int64_t e, int64_t i, int64_t j) {
  return (float)static_cast<const T*>(s.p)[e * s.se + i * s.si + j * s.sj];
}

// The expert and the first of its rows that row tile t covers; false behind the last.
__device__ bool find_tile(const FfnRows& r, int64_t t, int& expert, int& first, int& count, int& offset) {
  if (!r.offsets) {
    expert = 0;
    offset = 0;
    count = r.rows;
    first = (int)(t * kTile);
    return t * kTile < r.rows;
  }
  const int lane = threadIdx.x & 31;
  for (int e0 = 0; e0 < r.experts; e0 += 32) {
    const int e = e0 + lane;
    int begin = 0, n = 0;
    if (e < r.experts) {
      begin = max(r.offsets[e], 0);
      n = min(r.counts[e], r.rows - begin);   // rows that a route names outside the buffer are left out
    }
    const int tiles = n > 0 ? (n + kTile - 1) / kTile : 0;
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const unsigned has = __ballot_sync(0xffffffffu, t < upto);
    if (has) {
      const int src = __ffs(has) - 1;
      expert = e0 + src;
      offset = __shfl_sync(0xffffffffu, begin, src);
      count = __shfl_sync(0xffffffffu, n, src);
      first = (int)(t - __shfl_sync(0xffffffffu, upto - tiles, src)) * kTile;
      return true;
    }
    t -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

// 64 x 16 elements of an operand into shared memory, [k][row]; threads follow the
// direction in which it is contiguous.
template <typename T>
__device__ __forceinline__ void fill(float (&to)[kDeep][kTile + 4], const FfnStack& s, int64_t e, int64_t i0, int64_t in,
                                     int64_t k0, int64_t kn) {
  const bool along_k = s.sj == 1;
#pragma unroll
  for (int q = 0; q < kTile * kDeep / kThreads256; ++q) {
    const int x = threadIdx.x + q * kThreads256;
    const int i = along_k ? x / kDeep : x % kTile, k = along_k ? x % kDeep : x / kTile;
    to[k][i] = i0 + i < in && k0 + k < kn ? at<T>(s, e, i0 + i, k0 + k) : 0.f;
  }
}

// Keeps four values of a row, columns c .. c + 3 of 32 that eight neighbouring lanes share.
template <typename T>
__device__ __forceinline__ void keep(void* to, uint8_t* scales, const float (&v)[kPer], int64_t row, int64_t c, int64_t n,
                                     int64_t ldf, bool valid) {
  if (!scales) {
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (valid && c + q < n) static_cast<T*>(to)[row * ldf + c + q] = (T)v[q];
    return;
  }
  uint32_t most = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) most = max(most, c + q < n ? finite_bits(v[q]) : 0u);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  const uint32_t s = scale_byte(most);
  if (!valid) return;
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (c + q < n) static_cast<uint8_t*>(to)[row * ldf + c + q] = (uint8_t)encode2(v[q], 0.f, scale_up(s));
  if (c % 32 == 0 && c < n) scales[row * (ldf / 32) + c / 32] = (uint8_t)s;
}

template <typename T>
__device__ __forceinline__ float kept(const void* from, const uint8_t* scales, int64_t row, int64_t c, int64_t ldf) {
  if (!scales) return (float)static_cast<const T*>(from)[row * ldf + c];
  return decode2(static_cast<const uint8_t*>(from)[row * ldf + c]).x * scale_down(scales[row * (ldf / 32) + c / 32]);
}

template <typename T, FfnProduct kWhat>
__global__ void __launch_bounds__(kThreads256) k_ffn_simt(const __grid_constant__ FfnSimtParams p) {
  __shared__ float as[kDeep][kTile + 4], bs[2][kDeep][kTile + 4];
  grid_dependency_wait();
  allow_dependent_launch();
  constexpr bool kTwo = kWhat == FfnProduct::kGated, kSegments = kWhat == FfnProduct::kInput;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t n0 = (int64_t)blockIdx.y * kTile;
  int e = 0, first = 0, count = 0, offset = 0;
  int64_t m0, mn, k_end = p.k;
  if constexpr (kWhat == FfnProduct::kWeight) {
    e = blockIdx.z;
    m0 = (int64_t)blockIdx.x * kTile;
    mn = p.m;
    count = p.r.rows;
    if (p.r.offsets) {
      offset = max(p.r.offsets[e], 0);
      count = max(0, min(p.r.counts[e], p.r.rows - offset));
    }
    k_end = count;
  } else {
    if (!find_tile(p.r, blockIdx.x, e, first, count, offset)) return;
    m0 = first;
    mn = count;
  }
  float acc[kTwo ? 2 : 1][kPer][kPer] = {};
#pragma unroll 1
  for (int seg = 0; seg < (kSegments ? 2 : 1); ++seg) {
    FfnStack a = p.a[seg], b = p.b[seg];
    // operands over the sorted rows begin at the expert's
    if constexpr (kWhat == FfnProduct::kWeight) {
      a.p = static_cast<T*>(a.p) + offset * a.sj;
      b.p = static_cast<T*>(b.p) + offset * b.sj;
    } else {
      a.p = static_cast<T*>(a.p) + offset * a.si;
    }
    for (int64_t k0 = 0; k0 < k_end; k0 += kDeep) {
      __syncthreads();
      fill<T>(as, a, 0, m0, mn, k0, k_end);
      fill<T>(bs[0], b, kWhat == FfnProduct::kWeight ? 0 : e, n0, p.n, k0, k_end);
      if constexpr (kTwo) fill<T>(bs[1], p.b[1], e, n0, p.n, k0, k_end);
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(&as[k][ty * kPer]);
        const float xv[kPer] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int w = 0; w < (kTwo ? 2 : 1); ++w) {
          const float4 y = *reinterpret_cast<const float4*>(&bs[w][k][tx * kPer]);
          const float yv[kPer] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int j = 0; j < kPer; ++j) acc[w][i][j] = fmaf(xv[i], yv[j], acc[w][i][j]);
        }
      }
    }
  }
  const int64_t c0 = n0 + tx * kPer;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t m = m0 + ty * kPer + i, row = offset + m;
    const bool valid = m < mn;
    if constexpr (kWhat == FfnProduct::kGated) {
      if (p.saved.gate) {
        keep<T>(p.saved.gate, p.saved.gate_scales, acc[0][i], row, c0, p.n, p.ldf, valid);
        keep<T>(p.saved.up, p.saved.up_scales, acc[1][i], row, c0, p.n, p.ldf, valid);
      }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int64_t c = c0 + j;
      if (!valid || c >= p.n) continue;
      if constexpr (kWhat == FfnProduct::kGated) {
        static_cast<T*>(p.act)[row * p.ldf + c] = (T)(ffn_act<sizeof(T) == 2>(acc[0][i][j], p.activation).act * acc[1][i][j]);
      } else if constexpr (kWhat == FfnProduct::kSlope) {
        const float g = kept<T>(p.saved.gate, p.saved.gate_scales, row, c, p.ldf);
        const float u = kept<T>(p.saved.up, p.saved.up_scales, row, c, p.ldf);
        const FfnSlope s = ffn_act<sizeof(T) == 2>(g, p.activation);
        const float dh = acc[0][i][j];
        static_cast<T*>(p.dgate)[row * p.ldf + c] = (T)(dh * u * s.slope);
        static_cast<T*>(p.dup)[row * p.ldf + c] = (T)(dh * s.act);
        if (p.act) static_cast<T*>(p.act)[row * p.ldf + c] = (T)(s.act * u);
      } else if constexpr (kWhat == FfnProduct::kWeight) {
        static_cast<T*>(p.out.p)[e * p.out.se + m * p.out.si + c * p.out.sj] = (T)acc[0][i][j];
      } else {
        static_cast<T*>(p.out.p)[row * p.out.si + c] = (T)acc[0][i][j];
      }
    }
  }
}

// Sets the rows that hold no token to zero: after each expert's last token up to
// the next expert, and after the last expert.  Warps share them, row by row.
template <typename T>
__global__ void __launch_bounds__(kThreads256) k_ffn_clear(const __grid_constant__ FfnClearParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const uint32_t nw = gridDim.x * (kThreads256 / 32);
  const uint32_t me = blockIdx.x * (kThreads256 / 32) + (threadIdx.x >> 5);
  for (int e0 = 0; e0 <= p.r.experts; e0 += 32) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < p.r.experts) {
      lo = max(p.r.offsets[e], 0) + max(p.r.counts[e], 0);
      hi = p.r.offsets[e + 1];
    } else if (e == p.r.experts) {
      lo = p.r.offsets[e];
      hi = p.r.rows;
    }
    lo = max(lo, 0);
    hi = min(hi, p.r.rows);
    const uint32_t first = (uint32_t)lo + (me + nw - (uint32_t)lo % nw) % nw;   // this warp's first row of the expert
    unsigned some = __ballot_sync(0xffffffffu, lo < hi && first < (uint32_t)hi);
    while (some) {
      const int src = __ffs(some) - 1;
      some &= some - 1;
      const uint32_t a = __shfl_sync(0xffffffffu, first, src), b = __shfl_sync(0xffffffffu, (uint32_t)hi, src);
      for (uint32_t r = a; r < b; r += nw) {
        T* to = static_cast<T*>(p.out) + (int64_t)r * p.ld;
        const int64_t bytes = p.cols * (int64_t)sizeof(T);
        if ((reinterpret_cast<uintptr_t>(to) | (uintptr_t)bytes) % 16 == 0) {
          for (int64_t c = lane; c < bytes / 16; c += 32) reinterpret_cast<uint4*>(to)[c] = make_uint4(0u, 0u, 0u, 0u);
        } else {
          for (int64_t c = lane; c < p.cols; c += 32) to[c] = (T)0.f;
        }
      }
    }
  }
}

template <typename T>
int launch_simt(FfnProduct what, const FfnSimtParams& p, void* stream, bool pdl) {
  const unsigned nt = (unsigned)((p.n + kTile - 1) / kTile);
  if (what == FfnProduct::kWeight)
    return launch_kernel(k_ffn_simt<T, FfnProduct::kWeight>, dim3((unsigned)((p.m + kTile - 1) / kTile), nt, (unsigned)p.r.experts),
                         dim3(kThreads256), 0, stream, pdl, p);
  // an expert's last tile may be short: at most one more for each
  const unsigned mt = (unsigned)(p.r.rows / kTile + (p.r.offsets ? p.r.experts : 1));
  const dim3 grid(mt, nt), block(kThreads256);
  switch (what) {
    case FfnProduct::kGated: return launch_kernel(k_ffn_simt<T, FfnProduct::kGated>, grid, block, 0, stream, pdl, p);
    case FfnProduct::kDown: return launch_kernel(k_ffn_simt<T, FfnProduct::kDown>, grid, block, 0, stream, pdl, p);
    case FfnProduct::kSlope: return launch_kernel(k_ffn_simt<T, FfnProduct::kSlope>, grid, block, 0, stream, pdl, p);
    default: return launch_kernel(k_ffn_simt<T, FfnProduct::kInput>, grid, block, 0, stream, pdl, p);
  }
}

}  // namespace

int launch_ffn_simt(FfnProduct what, const FfnSimtParams& p, bool bf16, void* stream, bool pdl) {
  return bf16 ? launch_simt<__nv_bfloat16>(what, p, stream, pdl) : launch_simt<float>(what, p, stream, pdl);
}

int launch_ffn_clear(const FfnClearParams& p, bool bf16, void* stream, bool pdl) {
  const int64_t warps = p.r.rows < 8 * 304 ? p.r.rows : 8 * 304;
  const dim3 grid((unsigned)((warps + 7) / 8));
  if (bf16) return launch_kernel(k_ffn_clear<__nv_bfloat16>, grid, dim3(kThreads256), 0, stream, pdl, p);
  return launch_kernel(k_ffn_clear<float>, grid, dim3(kThreads256), 0, stream, pdl, p);
}

}  // namespace muon
