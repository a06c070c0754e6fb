// Gated feed-forward products for a few rows in bf16: the tokens that a served
// model decodes.
//
// The weights of the experts that have a token are read once, and everything is
// bound by that.  A CTA has 16 columns of the result (of gate and up both) and the
// rows of one expert, up to 8 or 16 of them (4 in the second product); its eight warps share the depth,
// 64 elements at a time in turn (or 32).  A lane reads 32 bytes of a weight row (or 16) straight into the
// registers of MMAs (mma.sync: with so few rows the tensor cores wait for memory in
// either form, and this one needs no stage in shared memory).  The unit h stands
// between the products as the sum of two bf16, itself rounded and what that left: two rows
// of the second product's MMAs.  Which depth an
// element of the operands stands for is the MMA's to choose as long as both sides
// agree: a lane's 16 bytes are eight depths in a row.
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "ffn_act.cuh"
#include "ffn_rows.cuh"
#include "launch_util.cuh"

namespace muon {

namespace {

constexpr int kWarps = 8, kCols = 16;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 or 32 bytes of a weight's row, read once: not kept in L1.
template <int kVec> struct Piece16 {
  uint4 v[kVec];
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (kVec == 2) {
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y), "=r"(v[1].z), "=r"(v[1].w)
                   : "l"(p)
                   : "memory");
    } else {
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w) : "l"(p) : "memory");
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
};

// The expert and rows of the part'th chunk of at most kRows rows; all threads.
template <int kRows>
__device__ __forceinline__ bool find_chunk(const FfnRows& r, int part, int& expert, int& first, int& n) {
  __shared__ int found[3];
  if (!r.offsets) {
    expert = 0;
    first = part * kRows;
    n = min(kRows, r.rows - first);
    return n > 0;
  }
  __shared__ int sums[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (r.experts + 32 * kWarps - 1) / (32 * kWarps), e0 = (int)threadIdx.x * per;
  int mine = 0;
  for (int e = e0; e < min(e0 + per, r.experts); ++e) mine += (ffn_expert(r, e).count + kRows - 1) / kRows;
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) sums[warp] = upto;
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  int at = upto - mine;
  for (int w = 0; w < warp; ++w) at += sums[w];
  if (part >= at && part < at + mine) {
    for (int e = e0; e < min(e0 + per, r.experts); ++e) {
      const FfnExpert x = ffn_expert(r, e);
      const int chunks = (x.count + kRows - 1) / kRows;
      if (part < at + chunks) {
        found[0] = e;
        found[1] = x.offset + (part - at) * kRows;
        found[2] = min(kRows, x.count - (part - at) * kRows);
        break;
      }
      at += chunks;
    }
  }
  __syncthreads();
  expert = found[0];
  first = found[1];
  n = found[2];
  return expert >= 0;
}

// Four CTAs per SM with 64 or 128 bytes of a lane in flight: a CTA lives for a few us,
// and others load while it finds its rows and joins its sums.  (2 rows of 2 experts,
// 2048 x 8192, both products: 39.6 us, 5.1 TB/s; with twice as much in flight and two
// CTAs 40.4, three CTAs 48.7, half as much and five CTAs 54; with 16 bytes at a time 46.)
// 9 to 16 rows have more sums and more of x in registers in the first product: two CTAs with
// twice as much in flight (16 rows of one layer 33.5 us, with the limits of fewer rows 44.6;
// since the second product is as below, 30).
// The second product, with h as one bf16 and up to 16 rows a CTA, took 39.8 us for 2 rows of 2
// experts (40.1 with the rest of the rounding), 200 for 16 rows of 16 experts (195), 81 for 12
// rows of 4 (74), but 21.5 for 8 rows of one layer (23.3) and 46.7 for 12 rows of 2 experts (48.2).
template <int kBlocks, bool kGated, int kVec>
__global__ void __launch_bounds__(32 * kWarps, kBlocks == 2 ? 2 : kGated && kVec == 1 ? 3 : 4) k_ffn_few(const __grid_constant__ FfnFewParams p) {
  // rows of an MMA, and the tokens that they stand for
  constexpr int kRows = 8 * kBlocks, kTokens = kGated ? kRows : kRows / 2, kMats = kGated ? 2 : 1, kLane = 8 * kVec, kDepth = 4 * kLane;
  constexpr int kAhead = (kGated ? 2 * kBlocks : 4) / kVec;   // steps whose weights are in flight
  __shared__ float red[kWarps][kMats][kCols][kRows + 1];
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / 4, t = lane % 4;
  if (!kGated && blockIdx.y == 0)
    ffn_clear_rows(p.r, static_cast<__nv_bfloat16*>(p.out), p.ldo, p.n, blockIdx.x * kWarps + warp, gridDim.x * kWarps);
  int expert, first, n;
  if (!find_chunk<kTokens>(p.r, blockIdx.y, expert, first, n)) return;
  const int64_t c0 = (int64_t)blockIdx.x * kCols;
  // this lane's rows of the weights, g and g + 8 of the 16 (the last one again behind the last)
  const __nv_bfloat16* w[kMats][2];
#pragma unroll
  for (int m = 0; m < kMats; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[m][h] = static_cast<const __nv_bfloat16*>(p.w[m].p) + expert * p.w[m].se + min(c0 + g + 8 * h, p.n - 1) * p.w[m].si + kLane * t;
  const __nv_bfloat16* x[kBlocks];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) {
    const int r = 8 * b + g;
    x[b] = static_cast<const __nv_bfloat16*>(p.x) + (int64_t)(first + min(r % kTokens, n - 1)) * p.ldx + (r < kTokens ? 0 : p.rest) + kLane * t;
  }
  float acc[kMats][kBlocks][4] = {};
  const int k_lane = (int)p.k - kLane * t;   // depths that this lane still has at step 0
  const int k_warp = warp * kDepth, steps = ((int)p.k + kDepth * kWarps - 1) / (kDepth * kWarps);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int s = 0; s < steps; s += kAhead) {
    Piece16<kVec> a[kAhead][kMats][2];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int k = (s + q) * kDepth * kWarps + k_warp;
#pragma unroll
      for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (k < k_lane) a[q][m][h].load(w[m][h] + k);
          else a[q][m][h].clear();
        }
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int k = (s + q) * kDepth * kWarps + k_warp;
      if (k >= p.k) break;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const uint4 v = k < k_lane ? *reinterpret_cast<const uint4*>(x[b] + k + 8 * i) : zero;
#pragma unroll
          for (int m = 0; m < kMats; ++m) {
            const uint4 &p0 = a[q][m][0].v[i], &p1 = a[q][m][1].v[i];
            mma16816(acc[m][b], p0.x, p1.x, p0.y, p1.y, v.x, v.y);
            mma16816(acc[m][b], p0.z, p1.z, p0.w, p1.w, v.z, v.w);
          }
        }
    }
  }
#pragma unroll
  for (int m = 0; m < kMats; ++m)
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][m][g + (i & 2 ? 8 : 0)][8 * b + 2 * t + (i & 1)] = acc[m][b][i];
  __syncthreads();
  for (int i = threadIdx.x; i < kCols * kTokens; i += 32 * kWarps) {
    const int c = i % kCols, row = i / kCols;
    if (row >= n || c0 + c >= p.padded) continue;
    float s[kMats];
#pragma unroll
    for (int m = 0; m < kMats; ++m) {
      s[m] = 0.f;
#pragma unroll
      for (int q = 0; q < kWarps; ++q) s[m] += kGated ? red[q][m][c][row] : red[q][m][c][row] + red[q][m][c][row + kRows - kTokens];
    }
    float v = kGated ? ffn_act<true>(s[0], p.activation).act * s[kMats - 1] : s[0];
    if (c0 + c >= p.n) v = 0.f;
    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + (int64_t)(first + row) * p.ldo + c0 + c;
    const __nv_bfloat16 rounded = __float2bfloat16_rn(v);
    *to = rounded;
    if constexpr (kGated) {   // nothing is left of an infinity
      const float is = __bfloat162float(rounded);
      to[p.rest] = __float2bfloat16_rn(fabsf(is) < __uint_as_float(0x7f800000u) ? v - is : 0.f);
    }
  }
}

template <bool kGated, int kVec>
int launch_vec(const FfnFewParams& p, void* stream, bool pdl) {
  const int rows = p.r.rows;
  auto launch = [&](auto* kernel, int full) {
    // chunks of rows: one for each expert with a row, and one more for each chunk that is full
    const dim3 grid((unsigned)((p.n + kCols - 1) / kCols), (unsigned)((rows < p.r.experts ? rows : p.r.experts) + rows / full));
    return launch_kernel(kernel, grid, dim3(32 * kWarps), 0, stream, pdl, p);
  };
  if constexpr (kGated) {
    return rows <= 8 ? launch(k_ffn_few<1, kGated, kVec>, 8) : launch(k_ffn_few<2, kGated, kVec>, 16);
  } else {
    return launch(k_ffn_few<1, kGated, kVec>, 4);
  }
}

// 32 bytes at a time where the weights' rows are made of them.
template <bool kGated>
int launch_few(const FfnFewParams& p, void* stream, bool pdl) {
  bool whole = p.k % 16 == 0;
  for (const FfnStack& w : p.w)
    whole = whole && (!w.p || (reinterpret_cast<uintptr_t>(w.p) % 32 == 0 && w.si % 16 == 0 && w.se % 16 == 0));
  return whole ? launch_vec<kGated, 2>(p, stream, pdl) : launch_vec<kGated, 1>(p, stream, pdl);
}

}  // namespace

int launch_ffn_few(bool gated, const FfnFewParams& p, void* stream, bool pdl) {
  return gated ? launch_few<true>(p, stream, pdl) : launch_few<false>(p, stream, pdl);
}

}  // namespace muon
