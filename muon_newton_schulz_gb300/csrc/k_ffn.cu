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
// The backward pass's gradients are one launch: the input's tiles, then all weights'.
// 6376 rows of 21 experts, 309 x 800: 26 TFLOP/s; 539 rows of 5 experts, 201 x 333, a
// training step: 80 us in four launches (116 with four launches for the gradients, one
// after another, and stores element by element; 168 without the ring and the clusters).
#include <cuda_runtime.h>

#include <algorithm>

#include "code8.cuh"
#include "ffn_act.cuh"
#include "ffn_rows.cuh"
#include "launch_util.cuh"
#include "train_internal.h"

namespace muon {

namespace {

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

// kRows x kDeep elements of an operand on their way to shared memory, [k][row], zero
// outside of the operand: 16 bytes at a time along aligned rows (`vec`), else element
// by element in the direction in which it is contiguous, along the depth 8 by 4 rows a
// warp, which fills 32 banks.
template <int kRows, int kDeep> struct Fetch {
  static constexpr int N = kRows * kDeep / kThreads256;      // elements of a thread
  static constexpr int kDeepApart = kThreads256 / kRows, kR = kRows / 32, kQ = kDeep / 8, kLine = kRows + 4;
  const float* at;       // this thread's first element at depth 0 of the sum
  const float* any;      // an address that may be read
  int64_t sj, apart[2];  // between depths, and between a thread's elements
  int left, i, k;        // rows from the first element on; where that goes in shared memory
  int rows, deep[2], to[2];
  bool vec;
  __device__ __forceinline__ void begin(const FfnStack& s, int64_t e, int64_t base, int64_t first, int64_t rows_all) {
    any = static_cast<const float*>(s.p) + e * s.se + base;
    sj = s.sj;
    const bool along_k = sj == 1;
    vec = s.si == 1 && !along_k && sj % 4 == 0 && reinterpret_cast<uintptr_t>(any) % 16 == 0;   // `first` is a multiple of 64
    const int t = threadIdx.x;
    i = along_k ? t / 8 : vec ? t % (kRows / 4) * 4 : t % kRows;
    k = along_k ? t % 8 : vec ? t / (kRows / 4) : t / kRows;
    at = any + (first + i) * s.si + k * sj;
    // element (r, q) of a thread: along the depth 32 r rows and 8 q deep, else kDeepApart (r kQ + q) deep
    rows = along_k ? 32 : 0;
    deep[0] = along_k ? 0 : kDeepApart * kQ;
    deep[1] = along_k ? 8 : kDeepApart;
    apart[0] = rows * s.si + deep[0] * sj;
    apart[1] = (vec ? 4 * kDeepApart : deep[1]) * sj;
    to[0] = rows + deep[0] * kLine;
    to[1] = deep[1] * kLine;
    left = (int)min(max(rows_all - first - i, (int64_t)0), (int64_t)kRows);
  }
  __device__ __forceinline__ void copy(float (*stage)[kLine], int k0, int kn) const {
    const float* from = at + k0 * sj;
    const int n = kn - k0 - k;
    if (vec) {
#pragma unroll
      for (int q = 0; q < N / 4; ++q) {
        const int some = q * 4 * kDeepApart < n ? min(left, 4) : 0;
        copy_async16(&stage[k + q * 4 * kDeepApart][i], some ? from + q * apart[1] : any, some);
      }
      return;
    }
    float* at_ = &stage[k][i];
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const bool has = r * rows < left && r * deep[0] + q * deep[1] < n;
        copy_async4(at_ + r * to[0] + q * to[1], has ? from + r * apart[0] + q * apart[1] : any, has);
      }
  }
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Four floats at the same place in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ float4 of_rank(const float4* mine, uint32_t rank) {
  uint32_t at;
  float4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}

// Four values of a row of ldf elements, a multiple of 128.  What lies behind the width is
// zero in what is kept for the backward pass, and never read elsewhere.
__device__ __forceinline__ void put4(void* to, const float (&v)[4], int64_t row, int64_t c, int64_t ldf) {
  *reinterpret_cast<float4*>(static_cast<float*>(to) + row * ldf + c) = make_float4(v[0], v[1], v[2], v[3]);
}

// Keeps four values of a row, columns c .. c + 3 of 32 that eight neighbouring lanes share.
__device__ __forceinline__ void keep(void* to, uint8_t* scales, const float (&v)[4], int64_t row, int64_t c, int64_t n,
                                     int64_t ldf, bool valid) {
  if (!scales) {
    const float z[4] = {c < n ? v[0] : 0.f, c + 1 < n ? v[1] : 0.f, c + 2 < n ? v[2] : 0.f, c + 3 < n ? v[3] : 0.f};
    if (valid) put4(to, z, row, c, ldf);
    return;
  }
  uint32_t most = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) most = max(most, c + q < n ? finite_bits(v[q]) : 0u);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  const uint32_t s = scale_byte(most);
  if (!valid || c >= n) return;
  *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(to) + row * ldf + c) = encode2(v[0], v[1], scale_up(s)) | encode2(v[2], v[3], scale_up(s)) << 16;
  if (c % 32 == 0) scales[row * (ldf / 32) + c / 32] = (uint8_t)s;
}

__device__ __forceinline__ void kept4(const void* from, const uint8_t* scales, int64_t row, int64_t c, int64_t ldf, float (&v)[4]) {
  const int64_t at = row * ldf + c;
  if (!scales) {
    const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(from) + at);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    return;
  }
  const uint32_t codes = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(from) + at);
  const float s = scale_down(scales[at / 32]);
  const float2 lo = decode2(codes), hi = decode2(codes >> 16);
  v[0] = lo.x * s, v[1] = lo.y * s, v[2] = hi.x * s, v[3] = hi.y * s;
}

template <FfnProduct kWhat, int kI, int kJ> struct Tiles {
  static constexpr int kMats = kWhat == FfnProduct::kGated ? 2 : 1, kM = 64 * kI, kN = 64 * kJ;
  static constexpr int kDeep = 16, kStages = kI == 1 ? 6 : 3;
  struct Stage {
    float a[kDeep][kM + 4], b[kMats][kDeep][kN + 4];
  };
  static constexpr int kAccs = kMats * kI * kJ * 16;   // sums of a thread
  static constexpr size_t kBytes = sizeof(Stage) * kStages > kAccs * kThreads256 * 4 ? sizeof(Stage) * kStages : kAccs * kThreads256 * 4;
};

// Where a CTA's tile lies: rows m0 .. (of mn) by columns n0 .. (of n) of an expert's
// product, whose sums are k_all long.
struct TileAt {
  int64_t m0, n0, mn, n, k_all;
  int e, offset, job;
};

// kI x kJ groups of 4 x 4 elements a thread, 64 rows or columns apart.  `splits` CTAs of a
// cluster, from rank `rank0` on, share the depth; this one has the part'th share.
template <FfnProduct kWhat, int kI, int kJ, int kAct>
__device__ __forceinline__ void run_tile(const FfnSimtParams& p, float4* smem, const TileAt& x, int splits, int part, int rank0) {
  using S = Tiles<kWhat, kI, kJ>;
  constexpr bool kTwo = kWhat == FfnProduct::kGated, kSegments = kWhat == FfnProduct::kInput, kWeight = kWhat == FfnProduct::kWeight;
  constexpr int kMats = S::kMats, kTileM = S::kM, kTileN = S::kN, kDeep = S::kDeep;
  auto* stage = reinterpret_cast<typename S::Stage*>(smem);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t m0 = x.m0, n0 = x.n0, mn = x.mn, n = x.n, k_all = x.k_all;
  const int e = x.e, offset = x.offset, job = x.job;
  const int64_t share = ((k_all + splits - 1) / splits + 7) / 8 * 8;
  const int k_begin = (int)min(part * share, k_all), k_end = (int)min(k_begin + share, k_all);
  const int per = (k_end - k_begin + kDeep - 1) / kDeep, steps = (kSegments ? 2 : 1) * per;
  Fetch<kTileM, kDeep> fa;
  Fetch<kTileN, kDeep> fb[kMats];
  // operands over the sorted rows begin at the expert's; two segments follow one another
  auto begin = [&](int seg) {
    const FfnStack& a = p.a[kWeight ? job : seg];
    fa.begin(a, 0, offset * (kWeight ? a.sj : a.si), m0, mn);
#pragma unroll
    for (int w = 0; w < kMats; ++w) {
      const FfnStack& b = p.b[kWeight ? job : kTwo ? w : seg];
      fb[w].begin(b, kWeight ? 0 : e, kWeight ? offset * b.sj : 0, n0, n);
    }
  };
  float acc[kMats][kI][kJ][4][4] = {};
  constexpr int kAhead = S::kStages - 1, kChunk = kI == 1 ? 8 : 16;   // deep at once
  int at = 0, to = 0;    // the step's place in the ring, and its copies'
  // the steps before 0 only begin copies: one piece of code for the instruction cache
#pragma unroll 1
  for (int t = -kAhead; t < steps; ++t) {
    if (t >= 0) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
      __syncthreads();   // the step is there for all, and the one before it is read
    }
    if (t + kAhead < steps) {
      if (t == -kAhead) begin(0);
      if (kSegments && t + kAhead == per) begin(1);
      const int k0 = k_begin + (t + kAhead < per ? t + kAhead : t + kAhead - per) * kDeep;
      fa.copy(stage[to].a, k0, k_end);
#pragma unroll
      for (int w = 0; w < kMats; ++w) fb[w].copy(stage[to].b[w], k0, k_end);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");   // one group per step, also behind the last
    if (++to == S::kStages) to = 0;
    if (t >= 0) {
      const int deep = k_end - k_begin - (t < per ? t : t - per) * kDeep;
#pragma unroll 1
      for (int k8 = 0; k8 < kDeep && k8 < deep; k8 += kChunk) {
#pragma unroll
        for (int k = k8; k < k8 + kChunk; ++k) {
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
      }
      if (++at == S::kStages) at = 0;
    }
  }
  if (splits > 1) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();   // the ring is read
    // the first CTA of the cluster adds the others' sums in order
    float4* mine = smem + threadIdx.x;
    float* flat = &acc[0][0][0][0][0];
    if (part > 0) {
#pragma unroll
      for (int q = 0; q < S::kAccs / 4; ++q) mine[q * kThreads256] = make_float4(flat[4 * q], flat[4 * q + 1], flat[4 * q + 2], flat[4 * q + 3]);
    }
    cluster_barrier();
    if (part == 0) {
      for (int r = 1; r < splits; ++r) {
#pragma unroll
        for (int q = 0; q < S::kAccs / 4; ++q) {
          const float4 v = of_rank(mine + q * kThreads256, rank0 + r);
          flat[4 * q] += v.x, flat[4 * q + 1] += v.y, flat[4 * q + 2] += v.z, flat[4 * q + 3] += v.w;
        }
      }
    }
    cluster_barrier();   // no CTA leaves while its sums are read
  }
  if (part == 0) {
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      constexpr int kOnce = kI == 1 ? 4 : 1;   // rows whose kept values are loaded before the first store
      float g[kOnce][kJ][4], u[kOnce][kJ][4];
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        const int64_t m = m0 + 64 * i + ty * 4 + ii, row = offset + m;
        const bool valid = m < mn;
        if constexpr (kWhat == FfnProduct::kSlope) {
          if (ii % kOnce == 0) {
#pragma unroll
            for (int q = 0; q < kOnce * kJ; ++q) {
              const int64_t c = n0 + 64 * (q % kJ) + tx * 4;
              if (m + q / kJ >= mn || c >= n) continue;
              kept4(p.saved.gate, p.saved.gate_scales, row + q / kJ, c, p.ldf, g[q / kJ][q % kJ]);
              kept4(p.saved.up, p.saved.up_scales, row + q / kJ, c, p.ldf, u[q / kJ][q % kJ]);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const int64_t c0 = n0 + 64 * j + tx * 4;
          const float(&v)[4] = acc[0][i][j][ii];
          if constexpr (kTwo) {
            const float(&up)[4] = acc[kMats - 1][i][j][ii];
            if (p.saved.gate) {
              keep(p.saved.gate, p.saved.gate_scales, v, row, c0, n, p.ldf, valid);
              keep(p.saved.up, p.saved.up_scales, up, row, c0, n, p.ldf, valid);
            }
            if (!valid) continue;
            float h[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) h[q] = c0 + q < n ? ffn_act<false, kAct>(v[q]).act * up[q] : 0.f;
            put4(p.act, h, row, c0, p.ldf);
            if (p.saved.bits == 32 && n0 + kTileN >= n && n0 + kTileN < p.ldf) {   // rows end behind the last tile
              const float zero[4] = {};
              put4(p.saved.gate, zero, row, c0 + kTileN, p.ldf);
              put4(p.saved.up, zero, row, c0 + kTileN, p.ldf);
              put4(p.act, zero, row, c0 + kTileN, p.ldf);
            }
          } else if constexpr (kWhat == FfnProduct::kSlope) {
            if (!valid || c0 >= n) continue;
            float dg[4], du[4], h[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const bool in = c0 + q < n;   // behind the width nothing was kept
              const FfnSlope s = ffn_act<false, kAct>(in ? g[ii % kOnce][j][q] : 0.f);
              const float uq = in ? u[ii % kOnce][j][q] : 0.f;
              dg[q] = v[q] * uq * s.slope;
              du[q] = v[q] * s.act;
              h[q] = s.act * uq;
            }
            put4(p.dgate, dg, row, c0, p.ldf);
            put4(p.dup, du, row, c0, p.ldf);
            if (p.act) put4(p.act, h, row, c0, p.ldf);
          } else {
            const FfnStack& out = p.out[job];
            float* to_row = static_cast<float*>(out.p) + (kWeight ? e * out.se + m * out.si : row * out.si);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (valid && c0 + q < n) to_row[c0 + q] = v[q];
          }
        }
      }
    }
  }
}

// The tile of a weight's gradient: the t'th of all jobs, of expert e.
template <int kTileM, int kTileN>
__device__ __forceinline__ TileAt weight_tile(const FfnSimtParams& p, int t, int e) {
  TileAt x;
  x.job = 0;
  while (x.job + 1 < p.jobs && t >= p.begin[x.job + 1]) ++x.job;
  t -= p.begin[x.job];
  x.n = p.wn[x.job];
  const int nt = (int)((x.n + kTileN - 1) / kTileN);
  x.n0 = (int64_t)(t % nt) * kTileN;
  x.m0 = (int64_t)(t / nt) * kTileM;
  x.mn = p.wm[x.job];
  x.e = e;
  const FfnExpert of = ffn_expert(p.r, e);
  x.offset = of.offset;
  x.k_all = of.count;
  return x;
}

// The CTAs of a cluster (along z) share the depth.
template <FfnProduct kWhat, int kI, int kJ, int kAct>
__global__ void __launch_bounds__(kThreads256, kI == 1 && kWhat != FfnProduct::kGated ? 3 : 2) k_ffn_simt(const __grid_constant__ FfnSimtParams p) {
  using S = Tiles<kWhat, kI, kJ>;
  constexpr bool kWeight = kWhat == FfnProduct::kWeight;
  extern __shared__ float4 smem[];
  // `beside`: launched in stream order, when the grids before it are complete
  if (!kWeight || !p.beside) grid_dependency_wait();
  allow_dependent_launch();
  const int part = blockIdx.z % p.splits;
  TileAt x{0, (int64_t)blockIdx.y * S::kN, 0, p.n, p.k, 0, 0, 0};
  bool tile = true;
  if constexpr (kWeight) {
    x = weight_tile<S::kM, S::kN>(p, blockIdx.x, blockIdx.z / p.splits);
  } else {
    if constexpr (kWhat == FfnProduct::kDown || kWhat == FfnProduct::kInput) {
      // the CTAs behind those that may have a tile clear the rows without a token
      if ((int)blockIdx.x >= p.row_tiles) {
        tile = false;
        if (blockIdx.y == 0 && part == 0)
          ffn_clear_rows(p.r, static_cast<float*>(p.out[0].p), p.out[0].si, p.n, (blockIdx.x - p.row_tiles) * (kThreads256 / 32) + (threadIdx.x >> 5),
                         (gridDim.x - p.row_tiles) * (kThreads256 / 32));
      }
    }
    int first = 0, count = 0;
    tile = tile && find_tile(p.r, blockIdx.x, S::kM, x.e, first, count, x.offset);
    x.m0 = first;
    x.mn = count;
  }
  if (!tile) return;   // all CTAs of a cluster alike
  run_tile<kWhat, kI, kJ, kAct>(p, smem, x, p.splits, part, 0);
  // nothing is pending then: this one returns at once
  if (kWeight && p.beside) grid_dependency_wait();
}

// The input's gradient and the weights' in one grid: none needs the other's results, and
// each alone has too few tiles for the machine.  The first CTAs are the input's: for each
// column of tiles `row_ctas` (times the splits), one for each row tile and then kClearCtas that
// clear the rows without a token.  Clusters lie along x and are as large as the larger of both splits; a
// tile's CTAs are consecutive ranks of one.  (Two launches of which the second waits for the
// first: 92 us for the training step of 539 rows, 201 x 333; one: 80.)
template <int kI>
__global__ void __launch_bounds__(kThreads256, kI == 1 ? 3 : 2) k_ffn_grads(const __grid_constant__ FfnGradsParams p) {
  using S = Tiles<FfnProduct::kInput, kI, kI>;
  extern __shared__ float4 smem[];
  grid_dependency_wait();
  allow_dependent_launch();
  const bool input = blockIdx.x < p.first_weight;
  const FfnSimtParams& q = input ? p.input : p.weights;
  const int cta = input ? blockIdx.x : blockIdx.x - p.first_weight;
  const int splits = q.splits, part = cta % splits, unit = cta / splits;
  const int rank0 = (int)blockIdx.x % p.cluster / splits * splits;
  TileAt x{0, 0, 0, q.n, q.k, 0, 0, 0};
  bool tile = true;
  if (input) {
    const int row_tile = unit % p.row_ctas, column = unit / p.row_ctas;
    tile = column < p.columns;
    x.n0 = (int64_t)column * S::kN;
    if (row_tile >= q.row_tiles) {
      if (column == 0 && part == 0)
        ffn_clear_rows(q.r, static_cast<float*>(q.out[0].p), q.out[0].si, q.n, (row_tile - q.row_tiles) * (kThreads256 / 32) + (threadIdx.x >> 5),
                       (p.row_ctas - q.row_tiles) * (kThreads256 / 32));
      tile = false;
    }
    int first = 0, count = 0;
    tile = tile && find_tile(q.r, row_tile, S::kM, x.e, first, count, x.offset);
    x.m0 = first;
    x.mn = count;
  } else {
    tile = unit / p.weight_ctas < q.r.experts;
    if (tile) x = weight_tile<S::kM, S::kN>(q, unit % p.weight_ctas, unit / p.weight_ctas);
  }
  if (!tile) {
    if (splits > 1) {   // the cluster's other tiles count on everyone
      cluster_barrier();
      cluster_barrier();
    }
    return;
  }
  if (input) run_tile<FfnProduct::kInput, kI, kI, kFfnSilu>(p.input, smem, x, splits, part, rank0);
  else run_tile<FfnProduct::kWeight, kI, kI, kFfnSilu>(p.weights, smem, x, splits, part, rank0);
}

// Fills in how a product is cut up into tiles and shares, and returns the CTAs of one split.
template <FfnProduct kWhat, int kI, int kJ>
dim3 plan_tiles(FfnSimtParams& p) {
  using S = Tiles<kWhat, kI, kJ>;
  constexpr bool kWeight = kWhat == FfnProduct::kWeight;
  auto tiles = [](int64_t n, int per) { return (unsigned)((n + per - 1) / per); };
  dim3 grid(1, kWeight ? 1 : tiles(p.n, S::kN));
  int64_t deep = p.k;
  if (kWeight) {
    p.begin[0] = 0;
    for (int i = 0; i < p.jobs; ++i) {
      grid.x = (unsigned)p.begin[i] + tiles(p.wm[i], S::kM) * tiles(p.wn[i], S::kN);
      if (i + 1 < p.jobs) p.begin[i + 1] = (int32_t)grid.x;
    }
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
  // codes goes by the order of its sum, which should be the same for every shape; a
  // training step of 64 rows, 512 x 2048, takes 155 us for it in place of 147, one of 300 rows
  // of 4 experts, 1024 x 1024, 687 either way)
  p.splits = 1;
  const bool one_order = kWhat == FfnProduct::kGated && p.saved.bits == 8;
  while (!one_order && p.splits < 8 && most * p.splits * 2 <= 304 && deep >= p.splits * 128) p.splits *= 2;
  return grid;
}

template <typename Params>
int launch_clusters(void (*kernel)(Params), dim3 grid, dim3 cluster, size_t smem, void* stream, bool pdl, const Params& p) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return (int)e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster.x;
  attr[0].val.clusterDim.y = cluster.y;
  attr[0].val.clusterDim.z = cluster.z;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return (int)cudaLaunchKernelEx(&cfg, kernel, p);
}

template <FfnProduct kWhat, int kI, int kJ>
int launch_tiles(FfnSimtParams p, void* stream, bool pdl) {
  dim3 grid = plan_tiles<kWhat, kI, kJ>(p);
  grid.z *= (unsigned)p.splits;
  constexpr bool kActs = kWhat == FfnProduct::kGated || kWhat == FfnProduct::kSlope;
  auto* kernel = kActs && p.activation == kFfnGelu ? k_ffn_simt<kWhat, kI, kJ, kActs ? kFfnGelu : kFfnSilu> : k_ffn_simt<kWhat, kI, kJ, kFfnSilu>;
  // what does not wait is started when the grids before it are complete
  if (kWhat == FfnProduct::kWeight && p.beside) pdl = false;
  return launch_clusters(kernel, grid, dim3(1, 1, (unsigned)p.splits), Tiles<kWhat, kI, kJ>::kBytes, stream, pdl, p);
}

// Large tiles where they give every SM one.
template <FfnProduct kWhat>
bool large_tiles(const FfnSimtParams& p) {
  constexpr int kJ = kWhat == FfnProduct::kGated ? 1 : 2;
  int64_t tiles = p.r.rows / 128 * (p.n / (64 * kJ));
  if (kWhat == FfnProduct::kWeight) {
    tiles = 0;
    for (int i = 0; i < p.jobs; ++i) tiles += p.wm[i] * p.r.experts / 128 * (p.wn[i] / 128);
  }
  return tiles >= 152;
}

template <FfnProduct kWhat>
int launch_size(const FfnSimtParams& p, void* stream, bool pdl) {
  if (large_tiles<kWhat>(p)) return launch_tiles<kWhat, 2, kWhat == FfnProduct::kGated ? 1 : 2>(p, stream, pdl);
  return launch_tiles<kWhat, 1, 1>(p, stream, pdl);
}

template <int kI>
int launch_both(const FfnSimtParams& input, const FfnSimtParams& weights, void* stream, bool pdl) {
  FfnGradsParams p{input, weights};
  const dim3 gi = plan_tiles<FfnProduct::kInput, kI, kI>(p.input), gw = plan_tiles<FfnProduct::kWeight, kI, kI>(p.weights);
  p.cluster = std::max(p.input.splits, p.weights.splits);
  auto whole = [&](int64_t ctas) { return (ctas + p.cluster - 1) / p.cluster * p.cluster; };
  const int64_t in = whole((int64_t)gi.x * gi.y * p.input.splits), all = in + whole((int64_t)gw.x * gw.z * p.weights.splits);
  p.row_ctas = (int32_t)gi.x;
  p.columns = (int32_t)gi.y;
  p.weight_ctas = (int32_t)gw.x;
  p.first_weight = (uint32_t)in;
  constexpr size_t a = Tiles<FfnProduct::kInput, kI, kI>::kBytes, b = Tiles<FfnProduct::kWeight, kI, kI>::kBytes;
  return launch_clusters(k_ffn_grads<kI>, dim3((unsigned)all), dim3((unsigned)p.cluster), a > b ? a : b, stream, pdl, p);
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

bool ffn_grads_in_one(const FfnSimtParams& input, const FfnSimtParams& weights) {
  return large_tiles<FfnProduct::kInput>(input) == large_tiles<FfnProduct::kWeight>(weights);
}

int launch_ffn_grads(const FfnSimtParams& input, const FfnSimtParams& weights, void* stream, bool pdl) {
  return large_tiles<FfnProduct::kInput>(input) ? launch_both<2>(input, weights, stream, pdl) : launch_both<1>(input, weights, stream, pdl);
}

}  // namespace muon
