// AdamW over many tensors, with states in 32 or in 8 bits, and gradient
// clipping by the global norm.
//
//   m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2,
//   p <- p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// All tensors of a call go through one launch (two when both kinds of state
// occur): a CTA takes one chunk of a tensor, which it finds by a binary search
// of the parameter block.  Nothing is reused, so HBM bounds the step with
// 32-bit states: 134 M bf16 elements (22 bytes each) take 422 us, 7.0 TB/s, the
// rate of a plain copy.  A short call (49 vectors of 2048) takes 4 us.
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "launch_util.cuh"
#include "train_internal.h"

namespace muon {

namespace {

constexpr int kThreads = kThreads256;

template <typename Block>
__device__ __forceinline__ const auto& find_tensor(const Block& p, uint32_t chunk) {
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
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 t = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Four elements at once where `vec` says that they lie on a vector boundary,
// else one by one.
template <typename T> __device__ __forceinline__ void load4(const T* p, float (&v)[4], bool vec) {
  if (vec) load4(p, v);
  else
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = load1(p + q);
}
template <typename T> __device__ __forceinline__ void store4(T* p, const float (&v)[4], bool vec) {
  if (vec) store4(p, v);
  else
#pragma unroll
    for (int q = 0; q < 4; ++q) store1(p + q, v[q]);
}

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
__device__ __forceinline__ void adamw32_one(const AdamHead& a, const AdamTensor& t, P* p, const G* g, float* m, float* v,
                                            int64_t e) {
  const float gv = load1(g + e);
  const float mv = fmaf(a.beta1, m[e], a.one_minus_beta1 * gv);
  const float vv = fmaf(a.beta2, v[e], a.one_minus_beta2 * (gv * gv));
  m[e] = mv;
  v[e] = vv;
  store1(p + e, updated(load1(p + e), mv, vv, t, a.eps));
}

// kAll: p, g, m and v all lie alike, as they nearly always do; else each of p, g
// and v is looked at, which costs a tenth.
template <typename P, typename G, bool kAll>
__device__ __forceinline__ void adamw32_body(const AdamHead& a, const AdamTensor& t, uint32_t chunk) {
  // Groups of four elements on m's vector boundaries: element 0 lies `shift`
  // elements past one.
  const int64_t base = (int64_t)(chunk - t.chunk_begin) * kAdamChunk - t.shift;
  P* p = static_cast<P*>(t.P);
  const G* g = static_cast<const G*>(t.G);
  float* m = static_cast<float*>(t.M);
  float* v = static_cast<float*>(t.V);
  constexpr int U = 2;
  const bool vp = kAll || (t.vec & kVecP), vg = kAll || (t.vec & kVecG), vv4 = kAll || (t.vec & kVecV);
#pragma unroll 1
  for (int it = 0; it < kAdamChunk / (kThreads * 4 * U); ++it) {
    const int64_t e0 = base + it * (kThreads * 4 * U) + threadIdx.x * 4;
    float pv[U][4], gv[U][4], mv[U][4], vv[U][4];
    bool full[U];   // a whole group inside the tensor
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t e = e0 + u * (kThreads * 4);
      full[u] = e >= 0 && e + 4 <= t.n;
      if (full[u]) {
        load4(p + e, pv[u], vp);
        load4(g + e, gv[u], vg);
        load4(m + e, mv[u]);
        load4(v + e, vv[u], vv4);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t e = e0 + u * (kThreads * 4);
      if (full[u]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          mv[u][q] = fmaf(a.beta1, mv[u][q], a.one_minus_beta1 * gv[u][q]);
          vv[u][q] = fmaf(a.beta2, vv[u][q], a.one_minus_beta2 * (gv[u][q] * gv[u][q]));
          pv[u][q] = updated(pv[u][q], mv[u][q], vv[u][q], t, a.eps);
        }
        store4(m + e, mv[u]);
        store4(v + e, vv[u], vv4);
        store4(p + e, pv[u], vp);
      } else {
        for (int64_t i = e < 0 ? 0 : e; i < e + 4 && i < t.n; ++i) adamw32_one(a, t, p, g, m, v, i);
      }
    }
  }
}

template <bool kAll>
__device__ __forceinline__ void adamw32_body(const AdamHead& a, const AdamTensor& t, uint32_t chunk) {
  if (t.p_bf16) {
    if (t.g_bf16) adamw32_body<__nv_bfloat16, __nv_bfloat16, kAll>(a, t, chunk);
    else adamw32_body<__nv_bfloat16, float, kAll>(a, t, chunk);
  } else {
    if (t.g_bf16) adamw32_body<float, __nv_bfloat16, kAll>(a, t, chunk);
    else adamw32_body<float, float, kAll>(a, t, chunk);
  }
}

template <int kTensors>
__global__ void __launch_bounds__(kThreads) k_adamw32(const __grid_constant__ AdamBlock<kTensors> a) {
  grid_dependency_wait();
  allow_dependent_launch();
  const AdamTensor& t = find_tensor(a, blockIdx.x);
  if (t.vec == (kVecP | kVecG | kVecV)) adamw32_body<true>(a, t, blockIdx.x);
  else adamw32_body<false>(a, t, blockIdx.x);
}

// ---------------------------------------------------------------- 8-bit states
//
// A warp takes one block of 256 elements, 8 per lane, so that the block's two
// scales are one warp-wide maximum each.  m and v are formed with separately
// rounded products and sums (no fused multiply-add): the stored codes then
// follow from the stated fp32 arithmetic bit for bit.
//
// Why these formats.  e4m3 and e5m2 under a power-of-two scale span 2^17 and
// 2^30 below a block's largest m and v (sqrt(v): 2^15), and scaling is exact.
// Rounding is stochastic because v changes by 1 - b2 (0.1 to 5 %) a step and
// e5m2 numbers are 12 to 25 % apart: rounded to nearest, v would never move.
//
// What bounds it.  268 M bf16 elements (10.02 bytes each) take 420 us, 6.4 TB/s
// or 94 % of a plain copy's rate; the issue slots are 85 % busy with some 53
// instructions per element, 9 of them for the random bits.  The first form of
// this kernel (one element at a time, loads straight to registers) took 748 us.

// A block's part of the random numbers of its elements.
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  x ^= x >> 16;
  return x;
}

// The two 16-bit halves of mix32(x): its last step leaves the upper half alone.
__device__ __forceinline__ void mix32_halves(uint32_t x, uint32_t& low, uint32_t& high) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  high = x >> 16;
  low = (x ^ high) & 0xffffu;
}

// Codes to fp32, exactly: two fp16 numbers, four e4m3 codes, four e5m2 codes.
__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
  float2 r;
  asm("{\n.reg .f16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}" : "=f"(r.x), "=f"(r.y) : "r"(h));
  return r;
}
__device__ __forceinline__ void e4m3x4_to_float2(uint32_t four, float2& lo, float2& hi) {
  uint32_t a, b;
  asm("{\n.reg .b16 s, t;\nmov.b32 {s, t}, %2;\ncvt.rn.f16x2.e4m3x2 %0, s;\ncvt.rn.f16x2.e4m3x2 %1, t;\n}" : "=r"(a), "=r"(b) : "r"(four));
  lo = half2_to_float2(a);
  hi = half2_to_float2(b);
}
// e5m2 is the upper byte of an fp16 number
__device__ __forceinline__ void e5m2x4_to_float2(uint32_t four, float2& lo, float2& hi) {
  lo = half2_to_float2(__byte_perm(four, 0, 0x1404));
  hi = half2_to_float2(__byte_perm(four, 0, 0x3424));
}

// The largest magnitude of three numbers, NaN if one of them is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

constexpr uint32_t kInfBits = 0x7f800000u;

// What the blocks of one tensor have in common, in registers.
struct Adam8 {
  float beta1, one_minus_beta1, beta2, one_minus_beta2, eps;
  float decay, step_size, inv_sqrt_bc2;
  float zero;   // -0
};

__device__ __forceinline__ Adam8 adam8(const AdamHead& p, const AdamTensor& t) {
  return {p.beta1, p.one_minus_beta1, p.beta2, p.one_minus_beta2, p.eps, t.decay, t.step_size, t.inv_sqrt_bc2, p.minus_zero};
}

// With an eps this large the root may take subnormal numbers for 0 (it is then
// below 2^-24 eps / 5), which saves the scaling that they need (67 M bf16 elements:
// 125 us against 139).
constexpr float kFlushEps = 1e-11f;

// Two sums or fused products at once, each rounded as by itself.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nadd.rn.f32x2 z, x, y;\nmov.b64 {%0, %1}, z;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n.reg .b64 x, y, z, w;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmov.b64 w, {%6, %7};\nfma.rn.f32x2 z, x, y, w;\n"
      "mov.b64 {%0, %1}, z;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// Two products rounded by themselves: `zero` is -0, which changes no sum, in a
// register whose value the assembler does not know: it fuses a plain packed
// product with the sum that follows (measured: codes that differ).
__device__ __forceinline__ float2 mul2(float2 a, float2 b, float zero) { return fma2(a, b, both(zero)); }

// Four numbers 0 <= y < 2^15 to four bytes, fp16 numbers without their last
// bits: kDrop = 21 leaves 5 exponent and 2 mantissa bits, the e5m2 codes;
// kDrop = 20 leaves, y being at most 1, 4 exponent and 3 mantissa bits, the
// e4m3 codes of 2^8 y.  Rounded stochastically: `random`, uniform in [0, 2^16),
// is added below the last bit that is kept.  Numbers below 2^-14 (fp16's, and
// the codes', subnormal ones) have 2^-14 added first, which gives them the
// spacing of the numbers just above it; their code is then one binade too
// high.  Taking the binade off the finished byte and not off the number makes
// the carry into the next binade come out right without another step.
template <int kDrop>
__device__ __forceinline__ uint32_t four_codes(const float (&y)[4], const uint32_t (&random)[4]) {
  uint32_t r;
  asm("{\n.reg .pred a, b, c, d;\n.reg .b32 s, t, u, v, h, k;\n"
      "setp.lt.f32 a, %1, 0f38800000;\nsetp.lt.f32 b, %2, 0f38800000;\n"
      "setp.lt.f32 c, %3, 0f38800000;\nsetp.lt.f32 d, %4, 0f38800000;\n"
      "mov.b32 s, %1;\nmov.b32 t, %2;\nmov.b32 u, %3;\nmov.b32 v, %4;\n"
      "@a add.f32 s, s, 0f38800000;\n@b add.f32 t, t, 0f38800000;\n"
      "@c add.f32 u, u, 0f38800000;\n@d add.f32 v, v, 0f38800000;\n"
      "mad.lo.u32 s, %5, %9, s;\nmad.lo.u32 t, %6, %9, t;\nmad.lo.u32 u, %7, %9, u;\nmad.lo.u32 v, %8, %9, v;\n"
      "cvt.rz.f16x2.f32 h, t, s;\ncvt.rz.f16x2.f32 k, v, u;\n"
      "shl.b32 h, h, %10;\nshl.b32 k, k, %10;\n"
      "prmt.b32 %0, h, k, 0x7531;\n"
      "@a add.u32 %0, %0, %11;\n@b add.u32 %0, %0, %12;\n@c add.u32 %0, %0, %13;\n@d add.u32 %0, %0, %14;\n}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "r"(random[0]), "r"(random[1]), "r"(random[2]), "r"(random[3]),
        "n"(1 << (kDrop - 16)), "n"(21 - kDrop), "n"(-(1 << (23 - kDrop))), "n"(-(1 << (31 - kDrop))),
        "n"(-(1 << (39 - kDrop))), "n"(-(1ll << (47 - kDrop))));
  return r;
}

template <bool kFlush>
__device__ __forceinline__ float2 updated8(float2 p, float2 m, float2 v, const Adam8& a) {
  if constexpr (kFlush) {
    float2 root, inv;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root.x) : "f"(v.x));
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root.y) : "f"(v.y));
    const float2 denom = fma2(root, both(a.inv_sqrt_bc2), both(a.eps));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv.x) : "f"(denom.x));   // denom >= eps: not subnormal
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv.y) : "f"(denom.y));
    return fma2(both(-a.step_size), mul2(m, inv, a.zero), mul2(p, both(a.decay), a.zero));
  }
  const float2 denom = fma2(make_float2(sqrt_approx(v.x), sqrt_approx(v.y)), both(a.inv_sqrt_bc2), both(a.eps));
  return fma2(both(-a.step_size), make_float2(__fdividef(m.x, denom.x), __fdividef(m.y, denom.y)), mul2(p, both(a.decay), a.zero));
}

// A lane's eight elements of a block: updates p, m and v, whose codes are four
// to a register, and returns the block's scale bytes.  `random` gives the
// first element's random numbers and `next` leads from one to the next.
// store_p takes the new p, early: it needs no register after that.
template <bool kFlush, typename S>
__device__ __forceinline__ uint32_t adamw8_core(const Adam8& a, float (&pv)[8], const float (&gv)[8], uint32_t (&mc)[2],
                                                uint32_t (&vc)[2], uint32_t sc, uint32_t random, uint32_t next,
                                                S store_p) {
  // beta * (code * scale) = code * (beta * scale), both products rounded
  // alike, unless subnormal numbers occur
  const uint32_t sm = sc & 0xffu, sv = sc >> 8;
  const float ms = __uint_as_float(sm << 23), vs = __uint_as_float(sv << 23);
  float bm = a.beta1, bv = a.beta2;
  float2 m[4], v[4];
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    e4m3x4_to_float2(mc[j / 2], m[j], m[j + 1]);
    e5m2x4_to_float2(vc[j / 2], v[j], v[j + 1]);
  }
  if (min(sm, sv) >= 64u) {
    bm *= ms;
    bv *= vs;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[j] = mul2(m[j], both(ms), a.zero);
      v[j] = mul2(v[j], both(vs), a.zero);
    }
  }
  float mtop = 0.f, vtop = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 g = make_float2(gv[2 * j], gv[2 * j + 1]);
    m[j] = add2(mul2(both(bm), m[j], a.zero), mul2(both(a.one_minus_beta1), g, a.zero));
    v[j] = add2(mul2(both(bv), v[j], a.zero), mul2(both(a.one_minus_beta2), mul2(g, g, a.zero), a.zero));
    const float2 q = updated8<kFlush>(make_float2(pv[2 * j], pv[2 * j + 1]), m[j], v[j], a);
    pv[2 * j] = q.x;
    pv[2 * j + 1] = q.y;
    mtop = max_abs3(mtop, m[j].x, m[j].y);
    vtop = max_abs3(vtop, v[j].x, v[j].y);
  }
  store_p(pv);
  uint32_t mmax = __reduce_max_sync(0xffffffffu, __float_as_uint(mtop));
  uint32_t vmax = __reduce_max_sync(0xffffffffu, __float_as_uint(vtop));
  const bool broken = max(mmax, vmax) >= kInfBits;   // the same for the whole warp
  if (broken) {
    // scales from the finite elements
    mmax = vmax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t mb = __float_as_uint(j & 1 ? m[j / 2].y : m[j / 2].x) & 0x7fffffffu;
      const uint32_t vb = __float_as_uint(j & 1 ? v[j / 2].y : v[j / 2].x) & 0x7fffffffu;
      if (mb < kInfBits) mmax = max(mmax, mb);
      if (vb < kInfBits) vmax = max(vmax, vb);
    }
    mmax = __reduce_max_sync(0xffffffffu, mmax);
    vmax = __reduce_max_sync(0xffffffffu, vmax);
  }
  const int cm = max((int)(mmax >> 23) - 7, 1), cv = max((int)(vmax >> 23) - 14, 1);
  // |m| / 2^8 in units of its scale: an e4m3 number is then an fp16 number
  // whose code is bits 7 to 13; and v in units of its scale: an e5m2 code is
  // the upper byte of an fp16 number
  if (cm > 240) {   // the same for the whole warp
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = mul2(m[j], both(0x1p-16f), a.zero);
  }
  const float mup = __uint_as_float((uint32_t)(cm > 240 ? 262 - cm : 246 - cm) << 23);
  const float vup = __uint_as_float((uint32_t)(254 - cv) << 23);

#pragma unroll
  for (int j = 0; j < 2; ++j) {   // four elements
    const float m4[4] = {m[2 * j].x, m[2 * j].y, m[2 * j + 1].x, m[2 * j + 1].y};
    const float v4[4] = {v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y};
    const float2 ya = mul2(v[2 * j], both(vup), a.zero), yb = mul2(v[2 * j + 1], both(vup), a.zero);
    float ym[4], yv[4] = {ya.x, ya.y, yb.x, yb.y};
    uint32_t rm[4], rv[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      mix32_halves(random + (4 * j + q) * next, rm[q], rv[q]);
      ym[q] = fabsf(m4[q]) * mup;
      // a v > 0 becomes at least the smallest code: one below it would be
      // rounded to it or to 0
      asm("{\n.reg .pred q;\nsetp.gt.f32 q, %1, 0f00000000;\n@q max.f32 %0, %0, 0f37800000;\n}" : "+f"(yv[q]) : "f"(v4[q]));
    }
    const uint32_t sign = __byte_perm(__byte_perm(__float_as_uint(m4[0]), __float_as_uint(m4[1]), 0x0073),
                                      __byte_perm(__float_as_uint(m4[2]), __float_as_uint(m4[3]), 0x0073), 0x5410);
    mc[j] = four_codes<20>(ym, rm) | (sign & 0x80808080u);
    vc[j] = four_codes<21>(yv, rv);
    if (broken) {   // NaN where a number is not finite
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t nan = 0x7fu << (8 * q), rest = ~(0xffu << (8 * q));
        if ((__float_as_uint(m4[q]) & 0x7fffffffu) >= kInfBits) mc[j] = (mc[j] & rest) | nan;
        if ((__float_as_uint(v4[q]) & 0x7fffffffu) >= kInfBits) vc[j] = (vc[j] & rest) | nan;
      }
    }
  }
  return (uint32_t)(cm | cv << 8);
}

// Whole blocks on vector boundaries.  Each warp has `count` consecutive blocks
// from block b on; lane l works on elements 8 l .. 8 l + 7 of each.  The next
// kStages - 1 blocks are copied to shared memory while one is worked on: the
// copies hold no registers, which decide how many warps there are to issue.
constexpr int kStages = 3;
template <typename P, typename G> constexpr int kBlockBytes = kStateBlock * (sizeof(P) + sizeof(G) + 2);
constexpr int kAdam8Smem = kStages * (kThreads / 32) * kBlockBytes<float, float>;
constexpr int kAdam8SmemBf16 = kStages * (kThreads / 32) * kBlockBytes<__nv_bfloat16, __nv_bfloat16>;

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

template <typename P, typename G, bool kFlush>
__device__ __forceinline__ void adamw8_blocks(const AdamHead& params, const AdamTensor& t, int64_t b, int count,
                                              uint8_t* shared) {
  const Adam8 a = adam8(params, t);
  const int lane = threadIdx.x & 31;
  constexpr int kB = kBlockBytes<P, G>, kAtG = kStateBlock * sizeof(P), kAtM = kAtG + kStateBlock * sizeof(G);
  uint8_t* ring = shared + (threadIdx.x >> 5) * (kStages * kB);
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring) + lane * 16;
  const int64_t e0 = b * kStateBlock;
  // this lane's pieces of 16 bytes
  const uint8_t* p_from = static_cast<const uint8_t*>(t.P) + e0 * sizeof(P) + lane * 16;
  const uint8_t* g_from = static_cast<const uint8_t*>(t.G) + e0 * sizeof(G) + lane * 16;
  const uint8_t* s_from = static_cast<const uint8_t*>(lane < 16 ? t.M : t.V) + e0 + (lane & 15) * 16;
  int to_fetch = count;
  uint32_t fetch_slot = 0;
  auto fetch = [&]() {   // the next block, if there is one
    if (to_fetch > 0) {
      const uint32_t to = ring_at + fetch_slot;
#pragma unroll
      for (int q = 0; q < (int)sizeof(P) / 2; ++q) copy16(to + q * 512, p_from + q * 512);
#pragma unroll
      for (int q = 0; q < (int)sizeof(G) / 2; ++q) copy16(to + kAtG + q * 512, g_from + q * 512);
      copy16(to + kAtM, s_from);
      p_from += kStateBlock * sizeof(P);
      g_from += kStateBlock * sizeof(G);
      s_from += kStateBlock;
      --to_fetch;
      fetch_slot = fetch_slot == (kStages - 1) * kB ? 0 : fetch_slot + kB;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch();

  P* p_to = static_cast<P*>(t.P) + e0 + lane * 8;
  uint8_t* m_to = static_cast<uint8_t*>(t.M) + e0 + lane * 8;
  uint8_t* v_to = static_cast<uint8_t*>(t.V) + e0 + lane * 8;
  uint16_t* scales = reinterpret_cast<uint16_t*>(t.scales) + b;
  uint32_t mine = lane < count ? scales[lane] : 0u;   // block `lane`'s scales, then its new ones
  const uint32_t key_hi = t.key_hi, first = lane * 8u * 0x9E3779B9u, block = (uint32_t)b + t.key_lo;
  const uint32_t mixed = mix32(block + lane) ^ key_hi;   // block `lane`'s part of the random numbers
  uint32_t slot = 0;
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();   // everybody's pieces have arrived, and everybody has read the block before
    fetch();
    const uint8_t* at = ring + slot;
    slot = slot == (kStages - 1) * kB ? 0 : slot + kB;
    float pv[8], gv[8];
    load8(reinterpret_cast<const P*>(at) + lane * 8, pv);
    load8(reinterpret_cast<const G*>(at + kAtG) + lane * 8, gv);
    const uint2 mr = *reinterpret_cast<const uint2*>(at + kAtM + lane * 8);
    const uint2 vr = *reinterpret_cast<const uint2*>(at + kAtM + kStateBlock + lane * 8);
    uint32_t mc[2] = {mr.x, mr.y}, vc[2] = {vr.x, vr.y};
    const uint32_t s = adamw8_core<kFlush>(a, pv, gv, mc, vc, __shfl_sync(0xffffffffu, mine, i),
                                         __shfl_sync(0xffffffffu, mixed, i) + first, 0x9E3779B9u,
                                         [&](const float (&x)[8]) { store8(p_to, x); });
    if (lane == i) mine = s;
    *reinterpret_cast<uint2*>(m_to) = make_uint2(mc[0], mc[1]);
    *reinterpret_cast<uint2*>(v_to) = make_uint2(vc[0], vc[1]);
    m_to += kStateBlock;
    v_to += kStateBlock;
    p_to += kStateBlock;
  }
  if (lane < count) scales[lane] = (uint16_t)mine;
}

// Any block: lane l has elements l, l + 32, ..., in single accesses that are
// coalesced all the same.
__device__ __forceinline__ void adamw8_any(const AdamHead& params, const AdamTensor& t, int64_t b) {
  const Adam8 a = adam8(params, t);
  const uint32_t lane = threadIdx.x & 31;
  uint8_t* m8 = static_cast<uint8_t*>(t.M);
  uint8_t* v8 = static_cast<uint8_t*>(t.V);
  const int64_t e0 = b * kStateBlock + lane;
  float pv[8], gv[8];
  uint32_t mc[2] = {0u, 0u}, vc[2] = {0u, 0u};
  const int left = (int)min((int64_t)kStateBlock, t.n - b * kStateBlock) - (int)lane;   // elements from this lane's first on
  auto each = [&](auto f) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (32 * j < left) f(j);
  };
#pragma unroll
  for (int j = 0; j < 8; ++j) pv[j] = gv[j] = 0.f;
  if (t.p_bf16) each([&](int j) { pv[j] = load1(static_cast<const __nv_bfloat16*>(t.P) + e0 + 32 * j); });
  else each([&](int j) { pv[j] = load1(static_cast<const float*>(t.P) + e0 + 32 * j); });
  if (t.g_bf16) each([&](int j) { gv[j] = load1(static_cast<const __nv_bfloat16*>(t.G) + e0 + 32 * j); });
  else each([&](int j) { gv[j] = load1(static_cast<const float*>(t.G) + e0 + 32 * j); });
  m8 += e0;
  v8 += e0;
  each([&](int j) {
    mc[j >> 2] |= (uint32_t)m8[32 * j] << (8 * (j & 3));
    vc[j >> 2] |= (uint32_t)v8[32 * j] << (8 * (j & 3));
  });
  uint16_t* scales = reinterpret_cast<uint16_t*>(t.scales + 2 * b);
  const uint32_t s = adamw8_core<false>(a, pv, gv, mc, vc, *scales,
                                        (mix32((uint32_t)b + t.key_lo) ^ t.key_hi) + lane * 0x9E3779B9u,
                                        32u * 0x9E3779B9u, [&](const float (&x)[8]) {
                                          if (t.p_bf16)
                                            each([&](int j) { store1(static_cast<__nv_bfloat16*>(t.P) + e0 + 32 * j, x[j]); });
                                          else
                                            each([&](int j) { store1(static_cast<float*>(t.P) + e0 + 32 * j, x[j]); });
                                        });
  each([&](int j) {
    m8[32 * j] = (uint8_t)(mc[j >> 2] >> (8 * (j & 3)));
    v8[32 * j] = (uint8_t)(vc[j >> 2] >> (8 * (j & 3)));
  });
  __syncwarp();   // every lane has read the scales
  if (lane == 0) *scales = (uint16_t)s;
}

template <bool kFlush>
__device__ __forceinline__ void adamw8_blocks(const AdamHead& p, const AdamTensor& t, int64_t b, int count,
                                              uint8_t* shared) {
  if (t.p_bf16) {
    if (t.g_bf16) adamw8_blocks<__nv_bfloat16, __nv_bfloat16, kFlush>(p, t, b, count, shared);
    else adamw8_blocks<__nv_bfloat16, float, kFlush>(p, t, b, count, shared);
  } else {
    if (t.g_bf16) adamw8_blocks<float, __nv_bfloat16, kFlush>(p, t, b, count, shared);
    else adamw8_blocks<float, float, kFlush>(p, t, b, count, shared);
  }
}

template <bool kFlush, int kTensors>
__global__ void __launch_bounds__(kThreads, 3) k_adamw8(const __grid_constant__ AdamBlock<kTensors> p) {
  extern __shared__ __align__(16) uint8_t shared[];
  grid_dependency_wait();
  allow_dependent_launch();
  const AdamTensor& t = find_tensor(p, blockIdx.x);
  const int per_warp = p.chunk / (kStateBlock * (kThreads / 32));   // at most 32
  const int64_t b = ((int64_t)(blockIdx.x - t.chunk_begin) * (kThreads / 32) + (threadIdx.x >> 5)) * per_warp;
  const int64_t end = min(b + per_warp, (t.n + kStateBlock - 1) / kStateBlock);
  // blocks that go whole
  int64_t rest = b;
  const int64_t fast_end = t.vec ? min(end, t.n / kStateBlock) : 0;
  if (b < fast_end) {
    adamw8_blocks<kFlush>(p, t, b, (int)(fast_end - b), shared);
    rest = fast_end;
  }
  for (; rest < end; ++rest) adamw8_any(p, t, rest);
}

// ---------------------------------------------------------------- gradient clipping
//
// Two passes: every CTA sums the squares of its chunks (fp32 within a chunk of
// a thread, 64 elements, fp64 across; in fp64 throughout where fp32 does not
// hold the squares), then every CTA adds up the CTAs' sums and scales its
// chunks.  HBM bounds both: 268 M bf16 gradients clipped into fp32
// take 335 us, 6.4 TB/s over the 2.15 GB of two reads and a write (the second
// read can only be saved for what L2 still holds, so the second pass starts
// where the first ended: 2 % less time for 17 to 67 M elements, none for
// 268 M).  A short call (49 vectors) takes 5 + 6 us.

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

// Calls f(row, first column, end, full) for this thread's groups of up to four
// columns of the chunk; `full` groups lie on a vector boundary.
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

// A whole chunk of one row, all of it full groups: the usual case, unrolled so
// that a thread has kAhead groups in flight.  Groups of four and not of eight:
// a warp's 16-byte stores of fp32 results are then consecutive.
constexpr int kAhead = 16;
__device__ __forceinline__ bool whole(const ClipTensor& t, const ClipChunk& k) {
  return t.vec && k.nr == 1 && k.nc == kClipChunk && k.c0 >= 0;
}

// This thread's part of a chunk, and the elements' bits, or'ed into `any`.
template <typename G>
__device__ __forceinline__ float sum_squares(const ClipTensor& t, const ClipChunk& k, uint32_t& any) {
  const G* g = static_cast<const G*>(t.G);
  float s = 0.f;
  auto add = [&](float x) {
    s = fmaf(x, x, s);
    any |= __float_as_uint(x);
  };
  if (whole(t, k)) {
    const G* at = g + k.r0 * t.ldg + k.c0 + threadIdx.x * 4;
#pragma unroll 1
    for (int i = 0; i < kClipChunk; i += kThreads * 4 * kAhead) {
      float x[kAhead][4];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) load4(at + i + u * (kThreads * 4), x[u]);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q) add(x[u][q]);
    }
    return s;
  }
  for_groups(t, k, [&](int64_t r, int64_t c, int64_t c1, bool full) {
    const G* at = g + r * t.ldg;
    if (full) {
      float x[4];
      load4(at + c, x);
#pragma unroll
      for (int q = 0; q < 4; ++q) add(x[q]);
    } else {
      for (int64_t e = c < 0 ? 0 : c; e < c1; ++e) add(load1(at + e));
    }
  });
  return s;
}

// The same elements, squared and summed in fp64.
template <typename G>
__device__ __noinline__ double sum_squares_wide(const ClipTensor& t, const ClipChunk& k) {
  const G* g = static_cast<const G*>(t.G);
  double s = 0.0;
  for_groups(t, k, [&](int64_t r, int64_t c, int64_t c1, bool) {
    for (int64_t e = c < 0 ? 0 : c; e < c1; ++e) {
      const double x = load1(g + r * t.ldg + e);
      s = fma(x, x, s);
    }
  });
  return s;
}

// The square of a number above 1.8e19 overflows in fp32, and one below its
// normal numbers loses up to 2^-150: 64 times that is 2^-34 of a sum of
// kLeastSum.  Sums outside this range are formed again in fp64, those of zeros
// alone (an embedding's unused rows) not.  268 M bf16 gradients: 85 us for the
// norm, and where every sum is formed twice 1003 us.
constexpr float kLeastSum = 0x1p-110f;
template <typename G>
__device__ __forceinline__ double chunk_squares(const ClipTensor& t, const ClipChunk& k) {
  uint32_t any = 0u;
  const float s = sum_squares<G>(t, k, any);
  if (s >= kLeastSum && s <= 3.4e38f) return s;
  return any << 1 ? sum_squares_wide<G>(t, k) : 0.0;
}

// The sum of v over the CTA, in a fixed order, for every thread.  One warp adds
// all of it: the fp64 unit has a fraction of the fp32 rate, and additions by
// every thread would take most of a small call's time.
__device__ __forceinline__ double block_sum(double v, double* red) {
  red[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += red[threadIdx.x + 32 * i];
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x == 0) red[kThreads] = s;
  }
  __syncthreads();
  return red[kThreads];
}

template <int kTensors>
__global__ void __launch_bounds__(kThreads) k_clip_sumsq(const __grid_constant__ ClipBlock<kTensors> p) {
  __shared__ double red[kThreads + 1];
  grid_dependency_wait();
  allow_dependent_launch();
  double s = 0.0;
  for (uint32_t chunk = blockIdx.x; chunk < p.chunks; chunk += gridDim.x) {
    const ClipTensor& t = find_tensor(p, chunk);
    const ClipChunk k = clip_chunk(t, chunk - t.chunk_begin);
    s += t.g_bf16 ? chunk_squares<__nv_bfloat16>(t, k) : chunk_squares<float>(t, k);
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) p.partial[p.partial_begin + blockIdx.x] = s;
}

// The factor is f * after.  after is 1, or the power of two that a factor too
// small for a normal fp32 number is split into.
struct ClipFactor {
  float f, after;
};
constexpr float kLeastFactor = 0x1p-100f;

__device__ __forceinline__ ClipFactor clip_factor(float max_norm, double norm) {
  // min(1, max_norm / (norm + 1e-6)), a NaN kept
  const float q = max_norm / ((float)norm + 1e-6f);
  // a huge norm (in fp32 perhaps infinite) or a tiny max_norm
  if (q < kLeastFactor && norm < (double)INFINITY) return {max_norm / (float)((norm + 1e-6) * 0x1p-64), 0x1p-64f};
  return {q >= 1.f ? 1.f : q, 1.f};
}

template <typename G, typename O>
__device__ __forceinline__ void scale_chunk(const ClipTensor& t, const ClipChunk& k, ClipFactor factor) {
  const G* g = static_cast<const G*>(t.G);
  O* out = static_cast<O*>(t.out);
  const float f = factor.f;
  if (whole(t, k) && factor.after == 1.f) {
    const G* at = g + k.r0 * t.ldg + k.c0 + threadIdx.x * 4;
    O* to = out + k.r0 * t.ldo + k.c0 + threadIdx.x * 4;
#pragma unroll 1
    for (int i = 0; i < kClipChunk; i += kThreads * 4 * kAhead) {
      float x[kAhead][4];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) load4(at + i + u * (kThreads * 4), x[u]);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
#pragma unroll
        for (int q = 0; q < 4; ++q) x[u][q] *= f;
        store4(to + i + u * (kThreads * 4), x[u], t.vec_out);
      }
    }
    return;
  }
  for_groups(t, k, [&](int64_t r, int64_t c, int64_t c1, bool full) {
    const G* at = g + r * t.ldg;
    O* to = out + r * t.ldo;
    if (full) {
      float x[4];
      load4(at + c, x);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[q] = x[q] * f * factor.after;
      store4(to + c, x, t.vec_out);
    } else {
      for (int64_t e = c < 0 ? 0 : c; e < c1; ++e) store1(to + e, load1(at + e) * f * factor.after);
    }
  });
}

// Every CTA sums the partials for itself, in the same order; one thread takes
// the root (in fp64, which all threads together would wait 1 us for).
template <int kTensors>
__global__ void __launch_bounds__(kThreads) k_clip_scale(const __grid_constant__ ClipBlock<kTensors> p) {
  __shared__ double red[kThreads + 1];
  __shared__ ClipFactor factor;
  grid_dependency_wait();
  allow_dependent_launch();
  double s = 0.0;
  for (int i = threadIdx.x; i < p.partials; i += kThreads) s += p.partial[i];
  s = block_sum(s, red);
  if (threadIdx.x == 0) {
    const double norm = sqrt(s);
    if (p.write_norm && blockIdx.x == 0) *p.norm = (float)norm;
    factor = clip_factor(p.max_norm, norm);
  }
  __syncthreads();
  const ClipFactor f = factor;
  // from the end: a part of what the sum read last is still in L2 (67 M bf16
  // elements: 88.1 us against 89.6 from the start)
  for (uint32_t i = blockIdx.x; i < p.chunks; i += gridDim.x) {
    const uint32_t chunk = p.chunks - 1 - i;
    const ClipTensor& t = find_tensor(p, chunk);
    if (f.f == 1.f && f.after == 1.f && t.out == t.G) continue;   // in place: unchanged
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

// Calls f with the launch's block, or with a small one where that holds it.
template <typename Few, typename Block, typename F>
int with_block(const Block& p, F f) {
  if (p.n > Few::kTensors) return f(p);
  Few few;
  static_cast<typename Few::Head&>(few) = p;
  for (int i = 0; i < p.n; ++i) few.t[i] = p.t[i];
  return f(few);
}
using FewAdam = AdamBlock<kFewTensors>;
using FewClip = ClipBlock<kFewTensors>;

}  // namespace

int launch_adamw32(const AdamParams& p, void* stream, bool pdl) {
  return with_block<FewAdam>(p, [&](const auto& b) {
    constexpr int kN = std::decay_t<decltype(b)>::kTensors;
    return launch_kernel(k_adamw32<kN>, dim3(p.chunks), dim3(kThreads), 0, stream, pdl, b);
  });
}

int launch_adamw8(const AdamParams& p, void* stream, bool pdl) {
  // room for the widest of the launch's tensors
  bool wide = false;
  for (int i = 0; i < p.n; ++i) wide = wide || !p.t[i].p_bf16 || !p.t[i].g_bf16;
  const int smem = wide ? kAdam8Smem : kAdam8SmemBf16;
  return with_block<FewAdam>(p, [&](const auto& b) {
    constexpr int kN = std::decay_t<decltype(b)>::kTensors;
    auto* kernel = p.eps >= kFlushEps ? k_adamw8<true, kN> : k_adamw8<false, kN>;
    if (smem > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return (int)e;
    }
    return launch_kernel(kernel, dim3(p.chunks), dim3(kThreads), (size_t)smem, stream, pdl, b);
  });
}

int launch_clip_sumsq(const ClipParams& p, int grid, void* stream, bool pdl) {
  return with_block<FewClip>(p, [&](const auto& b) {
    constexpr int kN = std::decay_t<decltype(b)>::kTensors;
    return launch_kernel(k_clip_sumsq<kN>, dim3((unsigned)grid), dim3(kThreads), 0, stream, pdl, b);
  });
}

int launch_clip_scale(const ClipParams& p, int grid, void* stream, bool pdl) {
  return with_block<FewClip>(p, [&](const auto& b) {
    constexpr int kN = std::decay_t<decltype(b)>::kTensors;
    return launch_kernel(k_clip_scale<kN>, dim3((unsigned)grid), dim3(kThreads), 0, stream, pdl, b);
  });
}

}  // namespace muon
