// Gated feed-forward products for a few rows in bf16: the tokens that a served
// model decodes.
//
// The weights of the experts that have a token are read once, and everything is
// bound by that.  A CTA has 16 columns of the result (of gate and up both) and the
// rows of one expert, up to 8 or 16 of them; its eight warps share the depth,
// 32 elements at a time in turn.  A lane reads 16 bytes of a weight row straight into the
// registers of an MMA (mma.sync: with so few rows the tensor cores wait for memory in
// either form, and this one needs no stage in shared memory).  Which depth an
// element of the operands stands for is the MMA's to choose as long as both sides
// agree: each lane's eight elements are the depths 8 (lane % 4) .. + 7.
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "ffn_act.cuh"
#include "ffn_rows.cuh"
#include "launch_util.cuh"

namespace muon {

namespace {

constexpr int kWarps = 8, kCols = 16, kDepth = 32;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 stream16(const void* p) {   // read once: not kept in L1
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

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

// Three or four CTAs per SM with two and four steps in flight: a CTA lives for a few
// us, and others load while it finds its rows and joins its sums (2 rows of 2
// experts, 2048 x 8192: 46 us for both products; four steps and two CTAs 47, eight
// steps and one CTA 62; 16 rows of 11 experts 184 us against 210 and 289).
template <int kBlocks, bool kGated>
__global__ void __launch_bounds__(32 * kWarps, kGated ? 3 : 4) k_ffn_few(const __grid_constant__ FfnFewParams p) {
  constexpr int kRows = 8 * kBlocks, kMats = kGated ? 2 : 1, kAhead = kGated ? 2 : 4;   // steps whose weights are in flight
  __shared__ float red[kWarps][kMats][kCols][kRows + 1];
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / 4, t = lane % 4;
  if (!kGated && blockIdx.y == 0)
    ffn_clear_rows(p.r, static_cast<__nv_bfloat16*>(p.out), p.ldo, p.n, blockIdx.x * kWarps + warp, gridDim.x * kWarps);
  int expert, first, n;
  if (!find_chunk<kRows>(p.r, blockIdx.y, expert, first, n)) return;
  const int64_t c0 = (int64_t)blockIdx.x * kCols;
  // this lane's rows of the weights, g and g + 8 of the 16 (the last one again behind the last)
  const __nv_bfloat16* w[kMats][2];
#pragma unroll
  for (int m = 0; m < kMats; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[m][h] = static_cast<const __nv_bfloat16*>(p.w[m].p) + expert * p.w[m].se + min(c0 + g + 8 * h, p.n - 1) * p.w[m].si + 8 * t;
  const __nv_bfloat16* x[kBlocks];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) x[b] = static_cast<const __nv_bfloat16*>(p.x) + (int64_t)(first + min(8 * b + g, n - 1)) * p.ldx + 8 * t;
  float acc[kMats][kBlocks][4] = {};
  const int k_lane = (int)p.k - 8 * t;   // depths that this lane still has at step 0
  const int k_warp = warp * kDepth, steps = ((int)p.k + kDepth * kWarps - 1) / (kDepth * kWarps);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int s = 0; s < steps; s += kAhead) {
    uint4 a[kAhead][kMats][2];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int k = (s + q) * kDepth * kWarps + k_warp;
#pragma unroll
      for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) a[q][m][h] = k < k_lane ? stream16(w[m][h] + k) : zero;
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int k = (s + q) * kDepth * kWarps + k_warp;
      if (k >= p.k) break;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        const uint4 v = k < k_lane ? *reinterpret_cast<const uint4*>(x[b] + k) : zero;
#pragma unroll
        for (int m = 0; m < kMats; ++m) {
          mma16816(acc[m][b], a[q][m][0].x, a[q][m][1].x, a[q][m][0].y, a[q][m][1].y, v.x, v.y);
          mma16816(acc[m][b], a[q][m][0].z, a[q][m][1].z, a[q][m][0].w, a[q][m][1].w, v.z, v.w);
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
  for (int i = threadIdx.x; i < kCols * kRows; i += 32 * kWarps) {
    const int c = i % kCols, row = i / kCols;
    if (row >= n || c0 + c >= p.n) continue;
    float s[kMats];
#pragma unroll
    for (int m = 0; m < kMats; ++m) {
      s[m] = 0.f;
#pragma unroll
      for (int q = 0; q < kWarps; ++q) s[m] += red[q][m][c][row];
    }
    const float v = kGated ? ffn_act<true>(s[0], p.activation).act * s[kMats - 1] : s[0];
    static_cast<__nv_bfloat16*>(p.out)[(int64_t)(first + row) * p.ldo + c0 + c] = __float2bfloat16_rn(v);
  }
}

template <bool kGated>
int launch_few(const FfnFewParams& p, void* stream, bool pdl) {
  // chunks of rows: one for each expert with a row, and one more for each chunk that is full
  const unsigned cols = (unsigned)((p.n + kCols - 1) / kCols);
  const int rows = p.r.rows, full = rows <= 8 ? 8 : 16;
  const dim3 grid(cols, (unsigned)((rows < p.r.experts ? rows : p.r.experts) + rows / full)), block(32 * kWarps);
  if (rows <= 8) return launch_kernel(k_ffn_few<1, kGated>, grid, block, 0, stream, pdl, p);
  return launch_kernel(k_ffn_few<2, kGated>, grid, block, 0, stream, pdl, p);

}

}  // namespace

int launch_ffn_few(bool gated, const FfnFewParams& p, void* stream, bool pdl) {
  return gated ? launch_few<true>(p, stream, pdl) : launch_few<false>(p, stream, pdl);
}

}  // namespace muon
