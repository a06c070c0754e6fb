// Gated feed-forward products in fp32, for every size and stride.
//
// The tokens of an expert are consecutive rows.  A CTA of 256 threads computes a
// tile of 64 x 64 or 128 x 128 elements of a product (128 x 64 where it has two
// results), each thread 4 or 8 rows by 4 or 8 columns; both operands pass through a
// ring of steps 16 deep in shared memory, copied ahead (cp.async, element by element
// where an operand runs along the depth or off its 16-byte boundaries).  The products over rows take
// their tiles from the counts on the device; a weight's gradient sums over the rows
// of its expert.  Where there are few tiles, the CTAs of a cluster share the sums of one,
// and the first joins their parts in order through distributed shared memory.
// 6376 rows of 21 experts, 309 x 800: 26 TFLOP/s; 539 rows of 5 experts, 201 x 333, a
// training step: 116 us in seven launches (168 without the ring and the clusters).
#include <cuda_runtime.h>

#include "code8.cuh"
#include "ffn_act.cuh"
#include "ffn_rows.cuh"
#include "launch_util.cuh"
#include "train_internal.h"

namespace muon {

namespace {

constexpr int kDeep = 16;
constexpr int kClearCtas = 64;   // that clear rows without a token

// The expert and the first of its rows that row tile t covers; false behind the last.
__device__ bool find_tile(const FfnRows& r, int64_t t, int rows_per_tile, int& expert, int& first, int& count, int& offset) {
  const int lane = threadIdx.x & 31;
  for (int e0 = 0; e0 < r.experts; e0 += 32) {
    const FfnExpert x = e0 + lane < r.experts ? ffn_expert(r, e0 + lane) : FfnExpert{0, 0};
    const int tiles = (x.count + rows_per_tile - 1) / rows_per_tile;
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const unsigned has = __ballot_sync(0xffffffffu, t < upto);
    if (has) {
      const int src = __ffs(has) - 1;
      expert = e0 + src;
      offset = __shfl_sync(0xffffffffu, x.offset, src);
      count = __shfl_sync(0xffffffffu, x.count, src);
      first = (int)(t - __shfl_sync(0xffffffffu, upto - tiles, src)) * rows_per_tile;
      return true;
    }
    t -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

__device__ __forceinline__ void copy_async4(float* to, const float* from, bool has) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from), "r"(has ? 4 : 0)
               : "memory");
}

// n of the four elements at `from`, zero for the others.
__device__ __forceinline__ void copy_async16(float* to, const float* from, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from), "r"(4 * n)
               : "memory");
}

// kRows x 16 elements of an operand on their way to shared memory, [k][row]; threads
// follow the direction in which it is contiguous.  Zero outside of the operand.
template <int kRows> struct Fetch {
  static constexpr int N = kRows * kDeep / kThreads256;      // elements of a thread
  static constexpr int kRowsApart = kThreads256 / kDeep, kDeepApart = kThreads256 / kRows;
  const float* at;       // this thread's first element at depth 0 of the sum
  const float* any;      // an address that may be read
  int64_t sj, apart;     // between depths, and between a thread's elements
  int left, i, k;        // rows from the first element on; where that goes in shared memory
  bool along_k, vec;
  __device__ __forceinline__ void begin(const FfnStack& s, int64_t e, int64_t base, int64_t first, int64_t rows) {
    any = static_cast<const float*>(s.p) + e * s.se + base;
    sj = s.sj;
    along_k = sj == 1;
    vec = s.si == 1 && !along_k && sj % 4 == 0 && reinterpret_cast<uintptr_t>(any) % 16 == 0;   // `first` is a multiple of 64
    const int t = threadIdx.x;
    i = along_k ? t / kDeep : vec ? t % (kRows / 4) * 4 : t % kRows;
    k = along_k ? t % kDeep : vec ? t / (kRows / 4) : t / kRows;
    at = any + (first + i) * s.si + k * sj;
    apart = along_k ? kRowsApart * s.si : (vec ? 4 * kDeepApart : kDeepApart) * sj;
    left = (int)min(max(rows - first - i, (int64_t)0), (int64_t)kRows);
  }
  __device__ __forceinline__ void copy(float (*to)[kRows + 4], int k0, int kn) const {
    const float* from = at + k0 * sj;
    const int deep = kn - k0 - k;
    if (vec) {
#pragma unroll
      for (int q = 0; q < (N + 3) / 4; ++q) {
        const int n = q * 4 * kDeepApart < deep ? min(left, 4) : 0;
        copy_async16(&to[k + q * 4 * kDeepApart][i], n ? from + q * apart : any, n);
      }
    } else if (along_k) {
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const bool has = q * kRowsApart < left && deep > 0;
        copy_async4(&to[k][i + q * kRowsApart], has ? from + q * apart : any, has);
      }
    } else {
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const bool has = left > 0 && q * kDeepApart < deep;
        copy_async4(&to[k + q * kDeepApart][i], has ? from + q * apart : any, has);
      }
    }
  }
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A float at the same place in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ float of_rank(const float* mine, uint32_t rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// Keeps four values of a row, columns c .. c + 3 of 32 that eight neighbouring lanes share.
__device__ __forceinline__ void keep(void* to, uint8_t* scales, const float (&v)[4], int64_t row, int64_t c, int64_t n,
                                     int64_t ldf, bool valid) {
  if (!scales) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (valid && c + q < n) static_cast<float*>(to)[row * ldf + c + q] = v[q];
    return;
  }
  uint32_t most = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) most = max(most, c + q < n ? finite_bits(v[q]) : 0u);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  const uint32_t s = scale_byte(most);
  if (!valid) return;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (c + q < n) static_cast<uint8_t*>(to)[row * ldf + c + q] = (uint8_t)encode2(v[q], 0.f, scale_up(s));
  if (c % 32 == 0 && c < n) scales[row * (ldf / 32) + c / 32] = (uint8_t)s;
}

__device__ __forceinline__ float kept(const void* from, const uint8_t* scales, int64_t row, int64_t c, int64_t ldf) {
  if (!scales) return static_cast<const float*>(from)[row * ldf + c];
  return decode2(static_cast<const uint8_t*>(from)[row * ldf + c]).x * scale_down(scales[row * (ldf / 32) + c / 32]);
}

template <FfnProduct kWhat, int kI, int kJ> struct Tiles {
  static constexpr int kMats = kWhat == FfnProduct::kGated ? 2 : 1, kM = 64 * kI, kN = 64 * kJ;
  static constexpr int kStages = kI == 1 ? 6 : 3;
  struct Stage {
    float a[kDeep][kM + 4], b[kMats][kDeep][kN + 4];
  };
  static constexpr int kAccs = kMats * kI * kJ * 16;   // sums of a thread
  static constexpr size_t kBytes = sizeof(Stage) * kStages > kAccs * kThreads256 * 4 ? sizeof(Stage) * kStages : kAccs * kThreads256 * 4;
};

// kI x kJ groups of 4 x 4 elements a thread, 64 rows or columns apart.  The CTAs of a
// cluster (along z) share the depth.
template <FfnProduct kWhat, int kI, int kJ>
__global__ void __launch_bounds__(kThreads256) k_ffn_simt(const __grid_constant__ FfnSimtParams p) {
  using S = Tiles<kWhat, kI, kJ>;
  constexpr bool kTwo = kWhat == FfnProduct::kGated, kSegments = kWhat == FfnProduct::kInput, kWeight = kWhat == FfnProduct::kWeight;
  constexpr int kMats = S::kMats, kTileM = S::kM, kTileN = S::kN;
  extern __shared__ float4 smem[];
  auto* stage = reinterpret_cast<typename S::Stage*>(smem);
  grid_dependency_wait();
  allow_dependent_launch();
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t n0 = (int64_t)blockIdx.y * kTileN;
  const int part = blockIdx.z % p.splits;
  int e = 0, first = 0, count = 0, offset = 0;
  int64_t m0, mn, k_all = p.k;
  bool tile = true;
  if constexpr (kWeight) {
    e = blockIdx.z / p.splits;
    m0 = (int64_t)blockIdx.x * kTileM;
    mn = p.m;
    const FfnExpert x = ffn_expert(p.r, e);
    offset = x.offset;
    k_all = count = x.count;
  } else {
    if constexpr (kWhat == FfnProduct::kDown || kSegments) {
      // the CTAs behind those that may have a tile clear the rows without a token
      if ((int)blockIdx.x >= p.row_tiles) {
        tile = false;
        if (blockIdx.y == 0 && part == 0)
          ffn_clear_rows(p.r, static_cast<float*>(p.out.p), p.out.si, p.n, (blockIdx.x - p.row_tiles) * (kThreads256 / 32) + (threadIdx.x >> 5),
                         (gridDim.x - p.row_tiles) * (kThreads256 / 32));
      }
    }
    tile = tile && find_tile(p.r, blockIdx.x, kTileM, e, first, count, offset);
    m0 = first;
    mn = count;
  }
  if (!tile) return;   // all CTAs of a cluster alike
  const int share = ((int)((k_all + kDeep - 1) / kDeep) + p.splits - 1) / p.splits * kDeep;
  const int k_begin = (int)min((int64_t)part * share, k_all), k_end = (int)min((int64_t)k_begin + share, k_all);
  float acc[kMats][kI][kJ][4][4] = {}, before[kSegments ? kI : 1][kSegments ? kJ : 1][4][4];
#pragma unroll 1
  for (int seg = 0; seg < (kSegments ? 2 : 1); ++seg) {
    const FfnStack &a = p.a[seg], &b = p.b[seg];
    // operands over the sorted rows begin at the expert's
    Fetch<kTileM> fa;
    Fetch<kTileN> fb[kMats];
    fa.begin(a, 0, offset * (kWeight ? a.sj : a.si), m0, mn);
    fb[0].begin(b, kWeight ? 0 : e, kWeight ? offset * b.sj : 0, n0, p.n);
    if constexpr (kTwo) fb[1].begin(p.b[1], e, 0, n0, p.n);
    if constexpr (kSegments) {
      // each product by itself, then their sum
#pragma unroll
      for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            before[i][j][q / 4][q % 4] = acc[0][i][j][q / 4][q % 4];
            acc[0][i][j][q / 4][q % 4] = 0.f;
          }
    }
    auto copy = [&](int at, int k0) {   // one group per step, also behind the last
      if (k0 < k_end) {
        fa.copy(stage[at].a, k0, k_end);
#pragma unroll
        for (int w = 0; w < kMats; ++w) fb[w].copy(stage[at].b[w], k0, k_end);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) copy(i, k_begin + i * kDeep);
    int at = 0, to = S::kStages - 1;
    for (int k0 = k_begin; k0 < k_end; k0 += kDeep) {
      asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 2) : "memory");
      __syncthreads();   // the step is there for all, and the one before it is read
      copy(to, k0 + (S::kStages - 1) * kDeep);
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        float4 x[kI], y[kMats][kJ];
#pragma unroll
        for (int i = 0; i < kI; ++i) x[i] = *reinterpret_cast<const float4*>(&stage[at].a[k][64 * i + ty * 4]);
#pragma unroll
        for (int w = 0; w < kMats; ++w)
#pragma unroll
          for (int j = 0; j < kJ; ++j) y[w][j] = *reinterpret_cast<const float4*>(&stage[at].b[w][k][64 * j + tx * 4]);
#pragma unroll
        for (int w = 0; w < kMats; ++w)
#pragma unroll
          for (int i = 0; i < kI; ++i)
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
              const float xv[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, yv[4] = {y[w][j].x, y[w][j].y, y[w][j].z, y[w][j].w};
#pragma unroll
              for (int q = 0; q < 16; ++q) acc[w][i][j][q / 4][q % 4] = fmaf(xv[q / 4], yv[q % 4], acc[w][i][j][q / 4][q % 4]);
            }
      }
      if (++at == S::kStages) at = 0;
      if (++to == S::kStages) to = 0;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();   // the ring is read
  }
  if constexpr (kSegments) {
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[0][i][j][q / 4][q % 4] += before[i][j][q / 4][q % 4];
  }
  if (p.splits > 1) {
    // the first CTA of the cluster adds the others' sums in order
    float* mine = reinterpret_cast<float*>(smem) + threadIdx.x;
    float* flat = &acc[0][0][0][0][0];
    if (part > 0) {
#pragma unroll
      for (int q = 0; q < S::kAccs; ++q) mine[q * kThreads256] = flat[q];
    }
    cluster_barrier();
    if (part == 0) {
      for (int r = 1; r < p.splits; ++r)
#pragma unroll
        for (int q = 0; q < S::kAccs; ++q) flat[q] += of_rank(mine + q * kThreads256, r);
    }
    cluster_barrier();   // no CTA leaves while its sums are read
    if (part > 0) return;
  }
#pragma unroll
  for (int i = 0; i < kI; ++i)
#pragma unroll
    for (int ii = 0; ii < 4; ++ii) {
      const int64_t m = m0 + 64 * i + ty * 4 + ii, row = offset + m;
      const bool valid = m < mn;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const int64_t c0 = n0 + 64 * j + tx * 4;
        if constexpr (kTwo) {
          if (p.saved.gate) {
            keep(p.saved.gate, p.saved.gate_scales, acc[0][i][j][ii], row, c0, p.n, p.ldf, valid);
            keep(p.saved.up, p.saved.up_scales, acc[1][i][j][ii], row, c0, p.n, p.ldf, valid);
          }
        }
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const int64_t c = c0 + jj;
          if (!valid || c >= p.n) continue;
          const float v = acc[0][i][j][ii][jj];
          if constexpr (kTwo) {
            static_cast<float*>(p.act)[row * p.ldf + c] = ffn_act<false>(v, p.activation).act * acc[1][i][j][ii][jj];
          } else if constexpr (kWhat == FfnProduct::kSlope) {
            const float g = kept(p.saved.gate, p.saved.gate_scales, row, c, p.ldf);
            const float u = kept(p.saved.up, p.saved.up_scales, row, c, p.ldf);
            const FfnSlope s = ffn_act<false>(g, p.activation);
            static_cast<float*>(p.dgate)[row * p.ldf + c] = v * u * s.slope;
            static_cast<float*>(p.dup)[row * p.ldf + c] = v * s.act;
            if (p.act) static_cast<float*>(p.act)[row * p.ldf + c] = s.act * u;
          } else if constexpr (kWeight) {
            static_cast<float*>(p.out.p)[e * p.out.se + m * p.out.si + c] = v;
          } else {
            static_cast<float*>(p.out.p)[row * p.out.si + c] = v;
          }
        }
      }
    }
}

template <FfnProduct kWhat, int kI, int kJ>
int launch_tiles(FfnSimtParams p, void* stream, bool pdl) {
  using S = Tiles<kWhat, kI, kJ>;
  constexpr bool kWeight = kWhat == FfnProduct::kWeight;
  auto tiles = [](int64_t n, int per) { return (unsigned)((n + per - 1) / per); };
  dim3 grid(1, tiles(p.n, S::kN));
  int64_t deep = p.k;
  if (kWeight) {
    grid.x = tiles(p.m, S::kM);
    grid.z = (unsigned)p.r.experts;
    deep = p.r.rows / p.r.experts;
  } else {
    // an expert's last tile may be short: at most one more for each that has a row
    p.row_tiles = p.r.rows / S::kM + (p.r.rows < p.r.experts ? p.r.rows : p.r.experts);
    const bool clears = (kWhat == FfnProduct::kDown || kWhat == FfnProduct::kInput) && p.r.offsets;
    grid.x = (unsigned)(p.row_tiles + (clears ? kClearCtas : 0));
  }
  // CTAs that share a tile: as long as there are fewer than two for every SM, and
  // each has 64 of the depth
  const int64_t most = kWeight ? (int64_t)grid.x * grid.y * grid.z : (int64_t)p.row_tiles * grid.y;
  // (not for pre-activations that become codes of 8 bits: one at the border of two
  // codes goes by the order of its sum, which should be the same for every shape)
  p.splits = 1;
  const bool one_order = kWhat == FfnProduct::kGated && p.saved.bits == 8;
  while (!one_order && p.splits < 8 && most * p.splits * 2 <= 304 && deep >= p.splits * 128) p.splits *= 2;
  grid.z *= (unsigned)p.splits;
  auto* kernel = k_ffn_simt<kWhat, kI, kJ>;
  if (S::kBytes > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kBytes);
    if (e != cudaSuccess) return (int)e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads256);
  cfg.dynamicSmemBytes = S::kBytes;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = (unsigned)p.splits;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return (int)cudaLaunchKernelEx(&cfg, kernel, p);
}

// Large tiles where they give every SM one.
template <FfnProduct kWhat>
int launch_size(const FfnSimtParams& p, void* stream, bool pdl) {
  constexpr int kJ = kWhat == FfnProduct::kGated ? 1 : 2;
  const int64_t m = kWhat == FfnProduct::kWeight ? p.m * p.r.experts : p.r.rows;
  if (m / 128 * (p.n / (64 * kJ)) >= 152) return launch_tiles<kWhat, 2, kJ>(p, stream, pdl);
  return launch_tiles<kWhat, 1, 1>(p, stream, pdl);
}

}  // namespace

int launch_ffn_simt(FfnProduct what, const FfnSimtParams& p, void* stream, bool pdl) {
  switch (what) {
    case FfnProduct::kGated: return launch_size<FfnProduct::kGated>(p, stream, pdl);
    case FfnProduct::kDown: return launch_size<FfnProduct::kDown>(p, stream, pdl);
    case FfnProduct::kSlope: return launch_size<FfnProduct::kSlope>(p, stream, pdl);
    case FfnProduct::kInput: return launch_size<FfnProduct::kInput>(p, stream, pdl);
    default: return launch_size<FfnProduct::kWeight>(p, stream, pdl);
  }
}

}  // namespace muon
