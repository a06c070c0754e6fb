// AdamW over many tensors, with states in 32 or in 8 bits.
//
//   m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2,
//   p <- p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// All tensors of a call go through one launch (two when both kinds of state
// occur): a CTA takes one chunk of kAdamChunk elements and finds its tensor by
// a binary search of the parameter block.  Nothing is reused, so HBM bounds
// both kernels.
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "launch_util.cuh"
#include "train_internal.h"

namespace muon {

namespace {

constexpr int kThreads = kThreads256;

__device__ __forceinline__ const AdamTensor& find_tensor(const AdamParams& p, uint32_t chunk) {
  int lo = 0, hi = p.n - 1;
  while (lo < hi) {  // last tensor whose chunk_begin <= chunk
    const int mid = (lo + hi + 1) >> 1;
    if (p.t[mid].chunk_begin <= chunk) lo = mid; else hi = mid - 1;
  }
  return p.t[lo];
}

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 t = *reinterpret_cast<const float4*>(p);
  v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 t = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(t.x << 16); v[1] = __uint_as_float(t.x & 0xffff0000u);
  v[2] = __uint_as_float(t.y << 16); v[3] = __uint_as_float(t.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The update of one parameter from its new m and v.  The root and the quotient
// are the approximate ones (a few units in the last place of the update, which
// itself is a small part of p); their exact forms would cost several times the
// instructions.
__device__ __forceinline__ float updated(float p, float m, float v, const AdamTensor& t, float eps) {
  const float denom = fmaf(sqrt_approx(v), t.inv_sqrt_bc2, eps);
  return fmaf(-t.step_size, __fdividef(m, denom), p * t.decay);
}

// ---------------------------------------------------------------- 32-bit states

template <typename P, typename G>
__device__ __forceinline__ void adamw32_body(const AdamParams& a, const AdamTensor& t, uint32_t chunk) {
  // Groups of four elements, aligned to vector boundaries: element 0 lies
  // `shift` elements past one.
  const int64_t base = (int64_t)(chunk - t.chunk_begin) * kAdamChunk - t.shift;
  P* p = static_cast<P*>(t.P);
  const G* g = static_cast<const G*>(t.G);
  float* m = static_cast<float*>(t.M);
  float* v = static_cast<float*>(t.V);
  constexpr int U = 2;
  if (t.vec && base >= 0 && base + kAdamChunk <= t.n) {
#pragma unroll 1
    for (int it = 0; it < kAdamChunk / (kThreads * 4 * U); ++it) {
      const int64_t e0 = base + it * (kThreads * 4 * U) + threadIdx.x * 4;
      float pv[U][4], gv[U][4], mv[U][4], vv[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t e = e0 + u * (kThreads * 4);
        load4(p + e, pv[u]);
        load4(g + e, gv[u]);
        load4(m + e, mv[u]);
        load4(v + e, vv[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t e = e0 + u * (kThreads * 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          mv[u][q] = fmaf(a.beta1, mv[u][q], a.one_minus_beta1 * gv[u][q]);
          vv[u][q] = fmaf(a.beta2, vv[u][q], a.one_minus_beta2 * (gv[u][q] * gv[u][q]));
          pv[u][q] = updated(pv[u][q], mv[u][q], vv[u][q], t, a.eps);
        }
        store4(m + e, mv[u]);
        store4(v + e, vv[u]);
        store4(p + e, pv[u]);
      }
    }
    return;
  }
  // a tensor's ends, and tensors whose pointers differ in their alignment
  const int64_t end = base + kAdamChunk < t.n ? base + kAdamChunk : t.n;
  for (int64_t e = (base < 0 ? 0 : base) + threadIdx.x; e < end; e += kThreads) {
    const float gv = load1(g + e);
    const float mv = fmaf(a.beta1, m[e], a.one_minus_beta1 * gv);
    const float vv = fmaf(a.beta2, v[e], a.one_minus_beta2 * (gv * gv));
    m[e] = mv;
    v[e] = vv;
    store1(p + e, updated(load1(p + e), mv, vv, t, a.eps));
  }
}

__global__ void __launch_bounds__(kThreads) k_adamw32(const __grid_constant__ AdamParams a) {
  const AdamTensor& t = find_tensor(a, blockIdx.x);
  if (t.p_bf16) {
    if (t.g_bf16) adamw32_body<__nv_bfloat16, __nv_bfloat16>(a, t, blockIdx.x);
    else adamw32_body<__nv_bfloat16, float>(a, t, blockIdx.x);
  } else {
    if (t.g_bf16) adamw32_body<float, __nv_bfloat16>(a, t, blockIdx.x);
    else adamw32_body<float, float>(a, t, blockIdx.x);
  }
}

// ---------------------------------------------------------------- 8-bit states
//
// A warp takes one block of 256 elements, 8 per lane, so that the block's two
// scales are one warp-wide maximum each.  m and v are formed with separately
// rounded products and sums (no fused multiply-add): the stored codes then
// follow from the stated fp32 arithmetic bit for bit.

__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  x ^= x >> 16;
  return x;
}

// Two e4m3 / e5m2 codes to fp32, exactly.
__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
  float2 r;
  asm("{\n.reg .f16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}" : "=f"(r.x), "=f"(r.y) : "r"(h));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
  uint32_t h;
  asm("{\n.reg .b16 t;\ncvt.u16.u32 t, %1;\ncvt.rn.f16x2.e4m3x2 %0, t;\n}" : "=r"(h) : "r"(two));
  return half2_to_float2(h);
}
// e5m2 is the upper byte of an fp16 number
__device__ __forceinline__ float2 e5m2x2_to_float2(uint32_t two) {
  return half2_to_float2(__byte_perm(two, 0, 0x1404));
}
// fp32 values that are e4m3 / e5m2 numbers to their codes (the first in the low byte)
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint32_t r;
  asm("{\n.reg .b16 t;\ncvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\ncvt.u32.u16 %0, t;\n}" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint32_t to_e5m2x2(float lo, float hi) {
  uint32_t r;
  asm("{\n.reg .b16 t;\ncvt.rn.satfinite.e5m2x2.f32 t, %2, %1;\ncvt.u32.u16 %0, t;\n}" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// y >= 0 rounded to a grid of numbers with `23 - kDrop` mantissa bits, whose
// numbers below kLow are spaced like those just above it; `bits` is uniform in
// [0, 2^kDrop).  Adding kLow to a number below it brings it into a binade
// whose grid has the right spacing.
template <int kDrop>
__device__ __forceinline__ float round_up_by(float y, uint32_t bits, float kLow) {
  const float off = y < kLow ? kLow : 0.f;
  const uint32_t t = (__float_as_uint(__fadd_rn(y, off)) + bits) & ~((1u << kDrop) - 1u);
  return __fadd_rn(__uint_as_float(t), -off);
}

constexpr uint32_t kInfBits = 0x7f800000u;

template <typename P, typename G>
__device__ __forceinline__ void adamw8_block(const AdamParams& a, const AdamTensor& t, int64_t b) {
  const int lane = threadIdx.x & 31;
  P* p = static_cast<P*>(t.P);
  const G* g = static_cast<const G*>(t.G);
  uint8_t* m8 = static_cast<uint8_t*>(t.M);
  uint8_t* v8 = static_cast<uint8_t*>(t.V);
  const int64_t e0 = b * kStateBlock;
  // whole blocks on vector boundaries: lane l has elements 8 l .. 8 l + 7;
  // else elements l, l + 32, ...: single accesses that are still coalesced
  const bool vec = t.vec && e0 + kStateBlock <= t.n;
  const uint32_t first = vec ? lane * 8 : lane, stride = vec ? 1 : 32;

  float pv[8], gv[8];
  uint32_t mc[4], vc[4];   // codes, two in each
  if (vec) {
    const int64_t e = e0 + lane * 8;
    float x[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load4(p + e + 4 * h, x);
#pragma unroll
      for (int q = 0; q < 4; ++q) pv[4 * h + q] = x[q];
      load4(g + e + 4 * h, x);
#pragma unroll
      for (int q = 0; q < 4; ++q) gv[4 * h + q] = x[q];
    }
    const uint2 mu = *reinterpret_cast<const uint2*>(m8 + e);
    const uint2 vu = *reinterpret_cast<const uint2*>(v8 + e);
    mc[0] = mu.x & 0xffffu; mc[1] = mu.x >> 16; mc[2] = mu.y & 0xffffu; mc[3] = mu.y >> 16;
    vc[0] = vu.x & 0xffffu; vc[1] = vu.x >> 16; vc[2] = vu.y & 0xffffu; vc[3] = vu.y >> 16;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) mc[j] = vc[j] = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t e = e0 + lane + 32 * j;
      pv[j] = gv[j] = 0.f;
      if (e < t.n) {
        pv[j] = load1(p + e);
        gv[j] = load1(g + e);
        mc[j >> 1] |= (uint32_t)m8[e] << (8 * (j & 1));
        vc[j >> 1] |= (uint32_t)v8[e] << (8 * (j & 1));
      }
    }
  }
  const uint32_t sc = *reinterpret_cast<const uint16_t*>(t.scales + 2 * b);
  const float ms = __uint_as_float((sc & 0xffu) << 23), vs = __uint_as_float((sc >> 8) << 23);

  float m[8], v[8];
  uint32_t mmax = 0, vmax = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 m2 = e4m3x2_to_float2(mc[j]), v2 = e5m2x2_to_float2(vc[j]);
    m[2 * j] = m2.x * ms; m[2 * j + 1] = m2.y * ms;
    v[2 * j] = v2.x * vs; v[2 * j + 1] = v2.y * vs;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    m[j] = __fadd_rn(__fmul_rn(a.beta1, m[j]), __fmul_rn(a.one_minus_beta1, gv[j]));
    v[j] = __fadd_rn(__fmul_rn(a.beta2, v[j]), __fmul_rn(a.one_minus_beta2, __fmul_rn(gv[j], gv[j])));
    pv[j] = updated(pv[j], m[j], v[j], t, a.eps);
    mmax = max(mmax, __float_as_uint(m[j]) & 0x7fffffffu);
    vmax = max(vmax, __float_as_uint(v[j]) & 0x7fffffffu);
  }
  mmax = __reduce_max_sync(0xffffffffu, mmax);
  vmax = __reduce_max_sync(0xffffffffu, vmax);
  const bool broken = mmax >= kInfBits || vmax >= kInfBits;   // the same for the whole warp
  if (broken) {
    // scales from the finite elements
    mmax = vmax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t mb = __float_as_uint(m[j]) & 0x7fffffffu, vb = __float_as_uint(v[j]) & 0x7fffffffu;
      if (mb < kInfBits) mmax = max(mmax, mb);
      if (vb < kInfBits) vmax = max(vmax, vb);
    }
    mmax = __reduce_max_sync(0xffffffffu, mmax);
    vmax = __reduce_max_sync(0xffffffffu, vmax);
  }
  const int cm = max((int)(mmax >> 23) - 7, 1), cv = max((int)(vmax >> 23) - 14, 1);
  const float mup = __uint_as_float((uint32_t)(254 - cm) << 23), vup = __uint_as_float((uint32_t)(254 - cv) << 23);

  const uint32_t seed = mix32((uint32_t)b + t.key_lo) ^ t.key_hi;
  float mq[8], vq[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t h = mix32(seed + (first + j * stride) * 0x9E3779B9u);
    const float ym = fabsf(m[j]) * mup, yv = v[j] * vup;
    mq[j] = copysignf(round_up_by<20>(ym, (h & 0xffffu) << 4, 0x1p-6f), m[j]);
    vq[j] = round_up_by<21>(yv, (h >> 16) << 5, 0x1p-14f);
    if (v[j] > 0.f && vq[j] == 0.f) vq[j] = 0x1p-16f;
    if (broken) {
      if ((__float_as_uint(m[j]) & 0x7fffffffu) >= kInfBits) mq[j] = __uint_as_float(0x7fffffffu);
      if ((__float_as_uint(v[j]) & 0x7fffffffu) >= kInfBits) vq[j] = __uint_as_float(0x7fffffffu);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    mc[j] = to_e4m3x2(mq[2 * j], mq[2 * j + 1]);
    vc[j] = to_e5m2x2(vq[2 * j], vq[2 * j + 1]);
  }
  if (vec) {
    const int64_t e = e0 + lane * 8;
    *reinterpret_cast<uint2*>(m8 + e) = make_uint2(mc[0] | mc[1] << 16, mc[2] | mc[3] << 16);
    *reinterpret_cast<uint2*>(v8 + e) = make_uint2(vc[0] | vc[1] << 16, vc[2] | vc[3] << 16);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float x[4] = {pv[4 * h], pv[4 * h + 1], pv[4 * h + 2], pv[4 * h + 3]};
      store4(p + e + 4 * h, x);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t e = e0 + lane + 32 * j;
      if (e < t.n) {
        m8[e] = (uint8_t)(mc[j >> 1] >> (8 * (j & 1)));
        v8[e] = (uint8_t)(vc[j >> 1] >> (8 * (j & 1)));
        store1(p + e, pv[j]);
      }
    }
  }
  if (lane == 0) *reinterpret_cast<uint16_t*>(t.scales + 2 * b) = (uint16_t)(cm | cv << 8);
}

template <typename P, typename G>
__device__ __forceinline__ void adamw8_body(const AdamParams& a, const AdamTensor& t, uint32_t chunk) {
  constexpr int kBlocks = kAdamChunk / kStateBlock, kWarps = kThreads / 32;
  const int64_t b0 = (int64_t)(chunk - t.chunk_begin) * kBlocks + (threadIdx.x >> 5);
#pragma unroll 1
  for (int i = 0; i < kBlocks / kWarps; ++i) {
    const int64_t b = b0 + i * kWarps;
    if (b * kStateBlock < t.n) adamw8_block<P, G>(a, t, b);
  }
}

__global__ void __launch_bounds__(kThreads) k_adamw8(const __grid_constant__ AdamParams a) {
  const AdamTensor& t = find_tensor(a, blockIdx.x);
  if (t.p_bf16) {
    if (t.g_bf16) adamw8_body<__nv_bfloat16, __nv_bfloat16>(a, t, blockIdx.x);
    else adamw8_body<__nv_bfloat16, float>(a, t, blockIdx.x);
  } else {
    if (t.g_bf16) adamw8_body<float, __nv_bfloat16>(a, t, blockIdx.x);
    else adamw8_body<float, float>(a, t, blockIdx.x);
  }
}

// ---------------------------------------------------------------- gradient clipping

// One chunk of a tensor: seg columns of rows_per_chunk rows.
struct ClipChunk {
  int64_t r0, c0;
  int nr, nc;
};

__device__ __forceinline__ ClipChunk clip_chunk(const ClipTensor& t, uint32_t local) {
  ClipChunk k;
  const int64_t rb = local / t.segs_per_row;
  k.r0 = rb * t.rows_per_chunk;
  k.c0 = (local - rb * t.segs_per_row) * t.seg - t.shift;
  k.nr = (int)min((int64_t)t.rows_per_chunk, t.rows - k.r0);
  k.nc = (int)min((int64_t)t.seg, t.cols - k.c0);
  return k;
}

__device__ __forceinline__ const ClipTensor& find_tensor(const ClipParams& p, uint32_t chunk) {
  int lo = 0, hi = p.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.t[mid].chunk_begin <= chunk) lo = mid; else hi = mid - 1;
  }
  return p.t[lo];
}

// Calls f(gradient address, row, column, elements) for this thread's groups of
// up to four elements of the chunk; `full` groups lie on a vector boundary.
template <typename F>
__device__ __forceinline__ void for_groups(const ClipTensor& t, const ClipChunk& k, F f) {
  const int groups = (k.nc + 3) >> 2;
  const int items = groups * k.nr;
  for (int i = threadIdx.x; i < items; i += kThreads) {
    const int r = k.nr == 1 ? 0 : i / groups;
    const int64_t c = k.c0 + (int64_t)(i - r * groups) * 4;
    const int64_t c1 = min(c + 4, k.c0 + k.nc);
    f(k.r0 + r, c, c1, t.vec && c >= 0 && c1 - c == 4);
  }
}

template <typename G>
__device__ __forceinline__ float sum_squares(const ClipTensor& t, const ClipChunk& k) {
  const G* g = static_cast<const G*>(t.G);
  float s = 0.f;
  for_groups(t, k, [&](int64_t r, int64_t c, int64_t c1, bool full) {
    const G* at = g + r * t.ldg;
    if (full) {
      float x[4];
      load4(at + c, x);
#pragma unroll
      for (int q = 0; q < 4; ++q) s = fmaf(x[q], x[q], s);
    } else {
      for (int64_t e = c < 0 ? 0 : c; e < c1; ++e) {
        const float x = load1(at + e);
        s = fmaf(x, x, s);
      }
    }
  });
  return s;
}

__device__ __forceinline__ double block_sum(double v, double* red) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  for (int i = 0; i < kThreads / 32; ++i) s += red[i];  // fixed order
  return s;
}

__global__ void __launch_bounds__(kThreads) k_clip_sumsq(const __grid_constant__ ClipParams p) {
  __shared__ double red[kThreads / 32];
  grid_dependency_wait();
  allow_dependent_launch();
  double s = 0.0;
  for (uint32_t chunk = blockIdx.x; chunk < p.chunks; chunk += gridDim.x) {
    const ClipTensor& t = find_tensor(p, chunk);
    const ClipChunk k = clip_chunk(t, chunk - t.chunk_begin);
    s += t.g_bf16 ? sum_squares<__nv_bfloat16>(t, k) : sum_squares<float>(t, k);
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) p.partial[p.partial_begin + blockIdx.x] = s;
}

template <typename G, typename O>
__device__ __forceinline__ void scale_chunk(const ClipTensor& t, const ClipChunk& k, float f) {
  const G* g = static_cast<const G*>(t.G);
  O* out = static_cast<O*>(t.out);
  for_groups(t, k, [&](int64_t r, int64_t c, int64_t c1, bool full) {
    const G* at = g + r * t.ldg;
    O* to = out + r * t.ldo;
    if (full) {
      float x[4];
      load4(at + c, x);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[q] *= f;
      store4(to + c, x);
    } else {
      for (int64_t e = c < 0 ? 0 : c; e < c1; ++e) store1(to + e, load1(at + e) * f);
    }
  });
}

// Every CTA sums the partials for itself, in the same order.
__global__ void __launch_bounds__(kThreads) k_clip_scale(const __grid_constant__ ClipParams p) {
  __shared__ double red[kThreads / 32];
  grid_dependency_wait();
  allow_dependent_launch();
  double s = 0.0;
  for (int i = threadIdx.x; i < p.partials; i += kThreads) s += p.partial[i];
  s = block_sum(s, red);
  const float norm = (float)sqrt(s);
  if (p.write_norm && blockIdx.x == 0 && threadIdx.x == 0) *p.norm = norm;
  // min(1, max_norm / (norm + 1e-6)), a NaN kept
  const float q = p.max_norm / (norm + 1e-6f);
  const float f = q >= 1.f ? 1.f : q;
  for (uint32_t chunk = blockIdx.x; chunk < p.chunks; chunk += gridDim.x) {
    const ClipTensor& t = find_tensor(p, chunk);
    if (f == 1.f && t.out == t.G) continue;   // in place: unchanged
    const ClipChunk k = clip_chunk(t, chunk - t.chunk_begin);
    if (t.g_bf16) {
      if (t.o_bf16) scale_chunk<__nv_bfloat16, __nv_bfloat16>(t, k, f);
      else scale_chunk<__nv_bfloat16, float>(t, k, f);
    } else {
      if (t.o_bf16) scale_chunk<float, __nv_bfloat16>(t, k, f);
      else scale_chunk<float, float>(t, k, f);
    }
  }
}

}  // namespace

int launch_adamw32(const AdamParams& p, void* stream) {
  return launch_kernel(k_adamw32, dim3(p.chunks), dim3(kThreads), 0, stream, false, p);
}

int launch_adamw8(const AdamParams& p, void* stream) {
  return launch_kernel(k_adamw8, dim3(p.chunks), dim3(kThreads), 0, stream, false, p);
}

int launch_clip_sumsq(const ClipParams& p, int grid, void* stream, bool pdl) {
  return launch_kernel(k_clip_sumsq, dim3((unsigned)grid), dim3(kThreads), 0, stream, pdl, p);
}

int launch_clip_scale(const ClipParams& p, int grid, void* stream, bool pdl) {
  return launch_kernel(k_clip_scale, dim3((unsigned)grid), dim3(kThreads), 0, stream, pdl, p);
}

}  // namespace muon
