// Tokens sorted by expert, and back.
//
// The sort is a stable counting sort of the slots (token, choice): a slot's
// row is its expert's first row plus the number of earlier slots of the same
// expert.  The row kernels go through the tokens, not through the sorted rows:
// a token's row is then read once however many experts it goes to, and a sum
// over its choices stays in one thread.  All of them are bound by HBM on
// batches and by launch latency on a few tokens.
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "launch_util.cuh"
#include "train_internal.h"

namespace muon {

namespace {

// ---------------------------------------------------------------- sort

__device__ __forceinline__ int expert_of(const SortParams& p, int64_t i) {
  // -1 for a slot that goes to no expert
  if (p.ids64) {
    const int64_t e = static_cast<const int64_t*>(p.ids)[i];
    return e >= 0 && e < p.experts ? (int)e : -1;
  }
  const int e = static_cast<const int32_t*>(p.ids)[i];
  return e >= 0 && e < p.experts ? e : -1;
}

// Counts each CTA's slots by expert.
__global__ void __launch_bounds__(kSortThreads) k_moe_count(const __grid_constant__ SortParams p) {
  extern __shared__ int32_t sm[];
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x) sm[e] = 0;
  __syncthreads();
  allow_dependent_launch();
  const int64_t i0 = (int64_t)blockIdx.x * p.per_cta;
  const int64_t i1 = min(i0 + p.per_cta, (int64_t)p.slots);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += blockDim.x) {
    const int e = expert_of(p, i);
    if (e >= 0) atomicAdd(&sm[e], 1);   // integer sums: the order does not matter
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x) p.hist[(int64_t)blockIdx.x * p.experts + e] = sm[e];
}

// Places each CTA's slots.  Each warp has a run of consecutive slots: the
// warps' counts, summed in their order, give the rank at which each warp
// starts in every expert; within 32 slots the rank is the number of lower
// lanes with the same expert.
__global__ void __launch_bounds__(kSortThreads) k_moe_place(const __grid_constant__ SortParams p) {
  extern __shared__ int32_t sm[];
  constexpr int kWarps = kSortThreads / 32;
  const int E = p.experts, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t* first = sm;              // [E] first row of each expert
  int32_t* start = sm + E;          // [kWarps][E] next rank of each warp in each expert
  __shared__ int32_t wsum[kWarps];
  for (int i = threadIdx.x; i < kWarps * E; i += kSortThreads) start[i] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * p.per_cta;
  const int64_t i1 = min(i0 + p.per_cta, (int64_t)p.slots);
  const int64_t per_warp = ((i1 - i0 + kSortThreads - 1) / kSortThreads) * 32;
  const int64_t w0 = min(i0 + warp * per_warp, i1), w1 = min(w0 + per_warp, i1);
  for (int64_t i = w0 + lane; i < w1; i += 32) {
    const int e = expert_of(p, i);
    if (e >= 0) atomicAdd(&start[warp * E + e], 1);
  }
  __syncthreads();
  grid_dependency_wait();
  // thread e: rank at which this CTA and each of its warps start in expert e,
  // and the expert's slots in all CTAs
  const int e = threadIdx.x;
  int total = 0, before = 0;
  if (e < E) {
    if (p.hist) {
      for (int c = 0; c < p.ctas; ++c) {
        const int n = p.hist[(int64_t)c * E + e];
        before = c < (int)blockIdx.x ? before + n : before;
        total += n;
      }
    }
    int run = before;
    for (int w = 0; w < kWarps; ++w) {
      const int n = start[w * E + e];
      start[w * E + e] = run;
      run += n;
    }
    if (!p.hist) total = run;
  }
  // first rows: a sum over the experts before, each rounded up
  const int kept = p.capacity > 0 ? min(total, p.capacity) : total;
  const int room = e >= E ? 0 : p.capacity > 0 ? p.capacity : (total + p.align - 1) / p.align * p.align;
  int incl = room;
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < warp; ++w) base += wsum[w];
  if (e < E) {
    first[e] = base + incl - room;
    if (blockIdx.x == 0) {
      p.offsets[e] = base + incl - room;
      p.counts[e] = kept;
      if (e == E - 1) p.offsets[E] = base + incl;
    }
  }
  __syncthreads();
  for (int64_t i = w0; i < w1; i += 32) {
    const int x = i + lane < w1 ? expert_of(p, i + lane) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, x);
    int rank = 0;
    if (x >= 0) rank = start[warp * E + x] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (x >= 0 && (same >> lane) == 1u) start[warp * E + x] = rank + 1;   // the highest of its lanes
    __syncwarp();
    if (i + lane < w1)
      p.row[i + lane] = x >= 0 && (p.capacity == 0 || rank < p.capacity) ? first[x] + rank : -1;
  }
}

// ---------------------------------------------------------------- rows

// Vec: what a thread moves at once: 16 bytes, or one element where addresses
// or the row length are not multiples of 16 bytes.
template <typename T, bool kVec> struct Piece;
template <> struct Piece<float, true> {
  static constexpr int N = 4;
  using Raw = float4;
};
template <> struct Piece<float, false> {
  static constexpr int N = 1;
  using Raw = float;
};
template <> struct Piece<__nv_bfloat16, true> {
  static constexpr int N = 8;
  using Raw = uint4;
};
template <> struct Piece<__nv_bfloat16, false> {
  static constexpr int N = 1;
  using Raw = __nv_bfloat16;
};

__device__ __forceinline__ void unpack(const float4& r, float (&v)[4]) { v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w; }
__device__ __forceinline__ void unpack(const float& r, float (&v)[1]) { v[0] = r; }
__device__ __forceinline__ void unpack(const __nv_bfloat16& r, float (&v)[1]) { v[0] = __bfloat162float(r); }
__device__ __forceinline__ void unpack(const uint4& r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void pack(float4& r, const float (&v)[4]) { r = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void pack(float& r, const float (&v)[1]) { r = v[0]; }
__device__ __forceinline__ void pack(__nv_bfloat16& r, const float (&v)[1]) { r = __float2bfloat16_rn(v[0]); }
__device__ __forceinline__ void pack(uint4& r, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
  r = make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename Raw> __device__ __forceinline__ Raw zero_raw();
template <> __device__ __forceinline__ float4 zero_raw<float4>() { return make_float4(0.f, 0.f, 0.f, 0.f); }
template <> __device__ __forceinline__ float zero_raw<float>() { return 0.f; }
template <> __device__ __forceinline__ uint4 zero_raw<uint4>() { return make_uint4(0u, 0u, 0u, 0u); }
template <> __device__ __forceinline__ __nv_bfloat16 zero_raw<__nv_bfloat16>() { return __float2bfloat16_rn(0.f); }

__device__ __forceinline__ float weight(const RowsParams& p, int64_t slot) {
  return p.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.w)[slot]) : static_cast<const float*>(p.w)[slot];
}

// Sets the rows of the sorted buffer that hold no token to zero: after each
// expert's last token up to the next expert, and after the last expert.  The
// warps of the launch's last CTAs share them, row by row.
template <typename T, bool kVec>
__device__ __forceinline__ void clear_rows(const RowsParams& p) {
  using Raw = typename Piece<T, kVec>::Raw;
  constexpr int N = Piece<T, kVec>::N;
  const int lane = threadIdx.x & 31;
  const int64_t nw = (int64_t)(gridDim.x - p.token_ctas) * (kThreads256 / 32);
  const int64_t me = (int64_t)(blockIdx.x - p.token_ctas) * (kThreads256 / 32) + (threadIdx.x >> 5);
  T* out = static_cast<T*>(p.out);
  for (int e0 = 0; e0 <= p.experts; e0 += 32) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < p.experts) {
      lo = p.offsets[e] + p.counts[e];
      hi = p.offsets[e + 1];
    } else if (e == p.experts) {
      lo = p.offsets[e];
      hi = p.rows;
    }
    lo = max(lo, 0);
    hi = min(hi, p.rows);
    unsigned some = __ballot_sync(0xffffffffu, lo < hi);
    while (some) {
      const int src = __ffs(some) - 1;
      some &= some - 1;
      const int a = __shfl_sync(0xffffffffu, lo, src), b = __shfl_sync(0xffffffffu, hi, src);
      for (int64_t r = a + (me - a % nw + nw) % nw; r < b; r += nw) {
        T* to = out + r * p.ldo;
        for (int64_t c = (int64_t)lane * N; c < p.hidden; c += 32 * N) *reinterpret_cast<Raw*>(to + c) = zero_raw<Raw>();
      }
    }
  }
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads256) k_moe_dispatch(const __grid_constant__ RowsParams p) {
  using Raw = typename Piece<T, kVec>::Raw;
  constexpr int N = Piece<T, kVec>::N;
  if ((int)blockIdx.x >= p.token_ctas) {
    clear_rows<T, kVec>(p);
    return;
  }
  const int ty = kThreads256 / p.tx;
  const int64_t t = (int64_t)blockIdx.x * ty + threadIdx.x / p.tx;
  if (t >= p.tokens) return;
  const T* x = static_cast<const T*>(p.x) + t * p.ldx;
  T* out = static_cast<T*>(p.out);
  const int32_t* row = p.row + t * p.topk;
  for (int64_t c = (int64_t)(threadIdx.x % p.tx) * N; c < p.hidden; c += (int64_t)p.tx * N) {
    const Raw v = *reinterpret_cast<const Raw*>(x + c);
    for (int k = 0; k < p.topk; ++k) {
      const int r = row[k];
      if ((uint32_t)r < (uint32_t)p.rows) *reinterpret_cast<Raw*>(out + r * p.ldo + c) = v;
    }
  }
}

// Choices are taken kK at a time so that their rows are loaded together.
template <typename T, bool kVec, int kK>
__global__ void __launch_bounds__(kThreads256) k_moe_combine(const __grid_constant__ RowsParams p) {
  using Raw = typename Piece<T, kVec>::Raw;
  constexpr int N = Piece<T, kVec>::N;
  const int ty = kThreads256 / p.tx;
  const int64_t t = (int64_t)blockIdx.x * ty + threadIdx.x / p.tx;
  if (t >= p.tokens) return;
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out) + t * p.ldo;
  const int64_t slot = t * p.topk;
  for (int64_t c = (int64_t)(threadIdx.x % p.tx) * N; c < p.hidden; c += (int64_t)p.tx * N) {
    float acc[N];
#pragma unroll
    for (int q = 0; q < N; ++q) acc[q] = 0.f;
    for (int k0 = 0; k0 < p.topk; k0 += kK) {
      Raw v[kK];
      float w[kK];
      bool has[kK];
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        const int r = k0 + k < p.topk ? p.row[slot + k0 + k] : -1;
        has[k] = (uint32_t)r < (uint32_t)p.rows;
        if (has[k]) {
          v[k] = *reinterpret_cast<const Raw*>(x + r * p.ldx + c);
          w[k] = p.w ? weight(p, slot + k0 + k) : 1.f;
        }
      }
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        if (!has[k]) continue;
        float f[N];
        unpack(v[k], f);
#pragma unroll
        for (int q = 0; q < N; ++q) acc[q] = fmaf(w[k], f[q], acc[q]);
      }
    }
    Raw o;
    pack(o, acc);
    *reinterpret_cast<Raw*>(out + c) = o;
  }
}

template <typename T, bool kVec, int kK>
__global__ void __launch_bounds__(kThreads256) k_moe_backward(const __grid_constant__ RowsParams p) {
  using Raw = typename Piece<T, kVec>::Raw;
  constexpr int N = Piece<T, kVec>::N;
  __shared__ float red[kThreads256 / 32][kK];
  if ((int)blockIdx.x >= p.token_ctas) {
    clear_rows<T, kVec>(p);
    return;
  }
  // tx is at least 32: a warp works on one token
  const int ty = kThreads256 / p.tx, y0 = threadIdx.x / p.tx;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = p.tx >> 5;
  const int64_t t = (int64_t)blockIdx.x * ty + y0;
  const bool live = t < p.tokens;
  const T* dout = static_cast<const T*>(p.x) + t * p.ldx;
  const T* y = static_cast<const T*>(p.y);
  T* out = static_cast<T*>(p.out);
  const int64_t slot = t * p.topk;
  for (int k0 = 0; k0 < p.topk; k0 += kK) {
    float dot[kK], w[kK];
    int r[kK];
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      dot[k] = 0.f;
      r[k] = live && k0 + k < p.topk ? p.row[slot + k0 + k] : -1;
      if ((uint32_t)r[k] >= (uint32_t)p.rows) r[k] = -1;
      w[k] = r[k] >= 0 ? weight(p, slot + k0 + k) : 0.f;
    }
    for (int64_t c = (int64_t)(threadIdx.x % p.tx) * N; live && c < p.hidden; c += (int64_t)p.tx * N) {
      const Raw draw = *reinterpret_cast<const Raw*>(dout + c);
      Raw v[kK];
#pragma unroll
      for (int k = 0; k < kK; ++k)
        if (r[k] >= 0) v[k] = *reinterpret_cast<const Raw*>(y + r[k] * p.ldy + c);
      float d[N];
      unpack(draw, d);
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        if (r[k] < 0) continue;
        float f[N], o[N];
        unpack(v[k], f);
#pragma unroll
        for (int q = 0; q < N; ++q) {
          dot[k] = fmaf(d[q], f[q], dot[k]);
          o[q] = w[k] * d[q];
        }
        Raw ro;
        pack(ro, o);
        *reinterpret_cast<Raw*>(out + r[k] * p.ldo + c) = ro;
      }
    }
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      for (int o = 16; o > 0; o >>= 1) dot[k] += __shfl_xor_sync(0xffffffffu, dot[k], o);
      if (lane == 0) red[warp][k] = dot[k];
    }
    __syncthreads();
    const int k = threadIdx.x % p.tx;
    if (live && k < kK && k0 + k < p.topk) {
      float s = 0.f;
      for (int i = 0; i < warps; ++i) s += red[y0 * warps + i][k];
      if (p.w_bf16) static_cast<__nv_bfloat16*>(p.dw)[slot + k0 + k] = __float2bfloat16_rn(s);
      else static_cast<float*>(p.dw)[slot + k0 + k] = s;
    }
    __syncthreads();
  }
}

template <typename F>
int opt_in_smem(F* kernel, size_t bytes) {
  return bytes <= 48 * 1024 ? 0 : (int)cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, bool kVec>
int launch_combine_k(const RowsParams& p, int grid, void* stream) {
  const dim3 g((unsigned)grid), b(kThreads256);
  if (p.topk == 1) return launch_kernel(k_moe_combine<T, kVec, 1>, g, b, 0, stream, false, p);
  if (p.topk == 2) return launch_kernel(k_moe_combine<T, kVec, 2>, g, b, 0, stream, false, p);
  if (p.topk <= 4) return launch_kernel(k_moe_combine<T, kVec, 4>, g, b, 0, stream, false, p);
  return launch_kernel(k_moe_combine<T, kVec, 8>, g, b, 0, stream, false, p);
}

template <typename T, bool kVec>
int launch_backward_k(const RowsParams& p, int grid, void* stream) {
  const dim3 g((unsigned)grid), b(kThreads256);
  if (p.topk == 1) return launch_kernel(k_moe_backward<T, kVec, 1>, g, b, 0, stream, false, p);
  if (p.topk == 2) return launch_kernel(k_moe_backward<T, kVec, 2>, g, b, 0, stream, false, p);
  if (p.topk <= 4) return launch_kernel(k_moe_backward<T, kVec, 4>, g, b, 0, stream, false, p);
  return launch_kernel(k_moe_backward<T, kVec, 8>, g, b, 0, stream, false, p);
}

}  // namespace

int launch_moe_sort_count(const SortParams& p, void* stream) {
  return launch_kernel(k_moe_count, dim3((unsigned)p.ctas), dim3(kSortThreads), (size_t)p.experts * 4, stream, false, p);
}

int launch_moe_sort_place(const SortParams& p, void* stream, bool pdl) {
  const size_t smem = (size_t)p.experts * (kSortThreads / 32 + 1) * 4;
  const int e = opt_in_smem(k_moe_place, smem);
  if (e) return e;
  return launch_kernel(k_moe_place, dim3((unsigned)p.ctas), dim3(kSortThreads), smem, stream, pdl, p);
}

int launch_moe_dispatch(const RowsParams& p, bool bf16, bool vec, int grid, void* stream) {
  const dim3 g((unsigned)grid), b(kThreads256);
  if (bf16)
    return vec ? launch_kernel(k_moe_dispatch<__nv_bfloat16, true>, g, b, 0, stream, false, p)
               : launch_kernel(k_moe_dispatch<__nv_bfloat16, false>, g, b, 0, stream, false, p);
  return vec ? launch_kernel(k_moe_dispatch<float, true>, g, b, 0, stream, false, p)
             : launch_kernel(k_moe_dispatch<float, false>, g, b, 0, stream, false, p);
}

int launch_moe_combine(const RowsParams& p, bool bf16, bool vec, int grid, void* stream) {
  if (bf16) return vec ? launch_combine_k<__nv_bfloat16, true>(p, grid, stream) : launch_combine_k<__nv_bfloat16, false>(p, grid, stream);
  return vec ? launch_combine_k<float, true>(p, grid, stream) : launch_combine_k<float, false>(p, grid, stream);
}

int launch_moe_backward(const RowsParams& p, bool bf16, bool vec, int grid, void* stream) {
  if (bf16) return vec ? launch_backward_k<__nv_bfloat16, true>(p, grid, stream) : launch_backward_k<__nv_bfloat16, false>(p, grid, stream);
  return vec ? launch_backward_k<float, true>(p, grid, stream) : launch_backward_k<float, false>(p, grid, stream);
}

}  // namespace muon
