// Rows of the sorted tokens: which belong to an expert, and which hold no token.
#pragma once

#include <cuda_runtime.h>

#include "ffn_internal.h"

namespace muon {

struct FfnExpert { int offset, count; };

// An expert's rows; those that a route names outside the buffer are left out.
__device__ __forceinline__ FfnExpert ffn_expert(const FfnRows& r, int e) {
  if (!r.offsets) return {0, r.rows};
  const int offset = min(max(r.offsets[e], 0), r.rows);
  return {offset, max(0, min(r.counts[e], r.rows - offset))};
}

// Sets the rows that hold no token to zero: after each expert's last token up to
// the next expert, and after the last expert.  `warps` warps share them, row by row;
// the caller is number `me`.
template <typename T>
__device__ __forceinline__ void ffn_clear_rows(const FfnRows& r, T* out, int64_t ld, int64_t cols, uint32_t me, uint32_t warps) {
  if (!r.offsets) return;   // every row holds one
  const int lane = threadIdx.x & 31;
  for (int e0 = 0; e0 <= r.experts; e0 += 32) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < r.experts) {
      lo = max(r.offsets[e], 0) + max(r.counts[e], 0);
      hi = r.offsets[e + 1];
    } else if (e == r.experts) {
      lo = r.offsets[e];
      hi = r.rows;
    }
    lo = max(lo, 0);
    hi = min(hi, r.rows);
    const uint32_t first = (uint32_t)lo + (me + warps - (uint32_t)lo % warps) % warps;   // this warp's first row of the expert
    unsigned some = __ballot_sync(0xffffffffu, lo < hi && first < (uint32_t)hi);
    while (some) {
      const int src = __ffs(some) - 1;
      some &= some - 1;
      const uint32_t a = __shfl_sync(0xffffffffu, first, src), b = __shfl_sync(0xffffffffu, (uint32_t)hi, src);
      for (uint32_t i = a; i < b; i += warps) {
        T* to = out + (int64_t)i * ld;
        const int64_t bytes = cols * (int64_t)sizeof(T);
        if ((reinterpret_cast<uintptr_t>(to) | (uintptr_t)bytes) % 16 == 0) {
          for (int64_t c = lane; c < bytes / 16; c += 32) reinterpret_cast<uint4*>(to)[c] = make_uint4(0u, 0u, 0u, 0u);
        } else {
          for (int64_t c = lane; c < cols; c += 32) to[c] = (T)0.f;
        }
      }
    }
  }
}

}  // namespace muon
