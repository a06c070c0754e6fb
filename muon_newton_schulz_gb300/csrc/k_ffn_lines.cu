// Rows of bf16 from and to matrices whose rows do not begin 16 bytes apart.
//
// The tensor cores' copies take rows on 16-byte boundaries.  Widths that are no
// multiple of 8 are therefore laid out in the workspace first, and results of such
// widths from there: one launch for all matrices of a pass, a warp for each row.
// Weights of experts without a token are left out.  Bound by HBM.
#include <cuda_runtime.h>

#include "ffn_rows.cuh"
#include "launch_util.cuh"
#include "train_internal.h"

namespace muon {

namespace {

constexpr int kAhead = 8;   // pairs of elements that a thread has in flight

__global__ void __launch_bounds__(kThreads256) k_ffn_lines(const __grid_constant__ FfnLinesParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads256 / 32);
  int i = 0;
  for (int64_t at = (int64_t)blockIdx.x * (kThreads256 / 32) + (threadIdx.x >> 5); at < p.lines; at += warps) {
    while (i + 1 < p.n && at >= p.job[i + 1].begin) ++i;
    const FfnLines& j = p.job[i];
    const int64_t line = at - j.begin, e = line / j.lines, l = line - e * j.lines;
    if (j.used_only && ffn_expert(p.r, (int)e).count == 0) continue;
    const uint16_t* from = static_cast<const uint16_t*>(j.from) + e * j.from_se + l * j.from_ld;
    uint16_t* to = static_cast<uint16_t*>(j.to) + e * j.to_se + l * j.to_ld;
    const bool pairs_in = reinterpret_cast<uintptr_t>(from) % 4 == 0, pairs_out = reinterpret_cast<uintptr_t>(to) % 4 == 0;
    for (int c0 = 2 * lane; c0 < j.padded; c0 += 64 * kAhead) {
      uint32_t v[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int c = c0 + 64 * q;
        v[q] = 0u;
        if (pairs_in && c + 1 < j.length) {
          v[q] = *reinterpret_cast<const uint32_t*>(from + c);
        } else {
          if (c < j.length) v[q] = from[c];
          if (c + 1 < j.length) v[q] |= (uint32_t)from[c + 1] << 16;
        }
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int c = c0 + 64 * q;
        if (pairs_out && c + 1 < j.padded) {
          *reinterpret_cast<uint32_t*>(to + c) = v[q];
        } else {
          if (c < j.padded) to[c] = (uint16_t)v[q];
          if (c + 1 < j.padded) to[c + 1] = (uint16_t)(v[q] >> 16);
        }
      }
    }
  }
}

}  // namespace

int launch_ffn_lines(const FfnLinesParams& p, void* stream, bool pdl) {
  const int64_t ctas = (p.lines + kThreads256 / 32 - 1) / (kThreads256 / 32);
  return launch_kernel(k_ffn_lines, dim3((unsigned)(ctas < 152 * 8 ? ctas : 152 * 8)), dim3(kThreads256), 0, stream, pdl, p);
}

}  // namespace muon
