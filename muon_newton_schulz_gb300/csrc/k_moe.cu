// Tokens sorted by expert, and back.
//
// The sort is a stable counting sort of the slots (token, choice): a slot's
// row is its expert's first row plus the number of earlier slots of the same
// expert.  The row kernels go through the tokens, not through the sorted rows:
// a token's row is then read once however many experts it goes to, and a sum
// over its choices stays in one thread.  All of them are bound by HBM on
// batches and by launch latency on a few tokens.  16384 tokens, 8 choices among
// 128 experts, rows of 2048 bf16 (share of a plain copy's 6.8 TB/s, counting each
// row once):
//   sort 7 us;  dispatch 90 us (99 %);  combine 95 us (94 %);
//   backward of combine 178 us (95 %).
// One token of 2 choices: sort 3.2 us, dispatch 2.9 us; combine of 5 tokens of 8
// choices, 6144 wide, 5 us.
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

// Counts each CTA's slots by expert, for hist[expert][CTA].
__global__ void __launch_bounds__(kSortThreads) k_moe_count(const __grid_constant__ SortParams p) {
  extern __shared__ int32_t sm[];
  for (int e = threadIdx.x; e < p.experts; e += kSortThreads) sm[e] = 0;
  __syncthreads();
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t i0 = (int64_t)blockIdx.x * p.per_cta;
  const int64_t i1 = min(i0 + p.per_cta, (int64_t)p.slots);
  constexpr int kAhead = 4;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kAhead * kSortThreads) {
    int e[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) e[u] = i + u * kSortThreads < i1 ? expert_of(p, i + u * kSortThreads) : -1;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (e[u] >= 0) atomicAdd(&sm[e[u]], 1);   // integer sums: the order does not matter
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += kSortThreads) p.hist[(int64_t)e * p.ctas + blockIdx.x] = sm[e];
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

__device__ __forceinline__ int warp_scan(int v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

// Places each CTA's slots.  (Up to 2048 slots one CTA does it all; more are
// counted by all CTAs first: a single CTA took 15 us for 8192 slots, both
// launches together take 6.)  Each warp has a run of consecutive slots, 32 at a
// time: a slot's rank among its warp's is the number of the warp's earlier
// slots of that expert, kept in shared memory, plus the lower lanes with the
// same expert.  The warps' totals, summed in their order after those of the
// CTAs before, then give the rank at which each warp starts.
// A run of at most kTile rounds keeps its experts and ranks in registers; with
// kTile = 0 the slots are read a second time.
static_assert(kSortThreads == 1024, "thread e has expert e, and lane w of a warp has warp w's count");

template <int kTile>
__global__ void __launch_bounds__(kSortThreads) k_moe_place(const __grid_constant__ SortParams p) {
  extern __shared__ int32_t sm[];
  constexpr int kWarps = kSortThreads / 32;
  const int E = p.experts, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ld = E | 1;             // odd: a warp then reads one expert's column without bank conflicts
  int32_t* start = sm;              // [kWarps][ld] each warp's slots of an expert, then the rank it starts at
  int32_t* total = sm + kWarps * ld;   // [E] slots of each expert in all CTAs, then its first row
  __shared__ int32_t wsum[kWarps];
  for (int i = threadIdx.x; i < kWarps * ld; i += kSortThreads) start[i] = 0;
  const int64_t i0 = (int64_t)blockIdx.x * p.per_cta;
  const int64_t i1 = min(i0 + p.per_cta, (int64_t)p.slots);
  const int rounds = (int)((i1 - i0 + kSortThreads - 1) / kSortThreads);
  const int64_t w0 = min(i0 + (int64_t)warp * rounds * 32, i1), w1 = min(w0 + (int64_t)rounds * 32, i1);
  int32_t* mine = start + warp * ld;
  // for the counts and for the ids: k_moe_count has waited for those itself, but
  // what it has seen is visible here only behind this grid's own wait
  grid_dependency_wait();
  allow_dependent_launch();

  // the rank of lane's slot (expert x) among the warp's; counts it
  auto count = [&](int x) {
    const unsigned same = __match_any_sync(0xffffffffu, x);
    const int rank = x >= 0 ? mine[x] + __popc(same & ((1u << lane) - 1)) : 0;
    __syncwarp();
    if (x >= 0 && (same >> lane) == 1u) mine[x] = rank + 1;   // the highest of its lanes
    __syncwarp();
    return rank;
  };
  int own[kTile + 1], rank[kTile + 1];
  if constexpr (kTile > 0) {
#pragma unroll
    for (int r = 0; r < kTile; ++r) own[r] = w0 + r * 32 + lane < w1 ? expert_of(p, w0 + r * 32 + lane) : -1;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kTile; ++r)
      if (r < rounds) rank[r] = count(own[r]);
  } else {
    __syncthreads();
    for (int64_t i = w0 + lane; i < w1; i += 32) {
      const int e = expert_of(p, i);
      if (e >= 0) atomicAdd(&mine[e], 1);
    }
  }
  __syncthreads();
  // a warp for each expert: lane w has warp w's slots, and lane c, c + 32, ...
  // those of CTAs c, c + 32, ...; several experts at a time, so that their
  // loads are in flight together
  constexpr int kAhead = 4, kLoads = (kSortGrid + 31) / 32;
  for (int e0 = warp; e0 < E; e0 += kAhead * kWarps) {
    int before[kAhead], all[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) before[q] = all[q] = 0;
    if (p.hist) {
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int e = e0 + q * kWarps;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int c = lane + 32 * i;
          const int n = e < E && c < p.ctas ? p.hist[(int64_t)e * p.ctas + c] : 0;
          all[q] += n;
          before[q] += c < (int)blockIdx.x ? n : 0;
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int e = e0 + q * kWarps;
      if (e >= E) break;
      const int n = start[lane * ld + e];
      const int incl = warp_scan(n, lane);
      start[lane * ld + e] = warp_sum(before[q]) + incl - n;
      const int sum = p.hist ? warp_sum(all[q]) : incl;
      if (lane == 31) total[e] = sum;
    }
  }
  __syncthreads();
  // first rows: a sum over the experts before, each rounded up; thread e has expert e
  const int e = threadIdx.x;
  const int all = e < E ? total[e] : 0;
  const int room = e >= E ? 0 : p.capacity > 0 ? p.capacity : p.align == 1 ? all : (all + p.align - 1) / p.align * p.align;
  const int incl = warp_scan(room, lane);
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int base = warp_sum(lane < warp ? wsum[lane] : 0);
  if (e < E) {
    total[e] = base + incl - room;
    if (blockIdx.x == 0) {
      p.offsets[e] = base + incl - room;
      p.counts[e] = p.capacity > 0 ? min(all, p.capacity) : all;
      if (e == E - 1) p.offsets[E] = base + incl;
    }
  }
  __syncthreads();
  auto row_of = [&](int x, int r) { return x >= 0 && (p.capacity == 0 || r < p.capacity) ? total[x] + r : -1; };
  if constexpr (kTile > 0) {
#pragma unroll
    for (int r = 0; r < kTile; ++r) {
      const int64_t i = w0 + r * 32 + lane;
      if (i < w1) p.row[i] = row_of(own[r], own[r] >= 0 ? mine[own[r]] + rank[r] : 0);
    }
  } else {
    for (int64_t i = w0; i < w1; i += 32) {
      const int x = i + lane < w1 ? expert_of(p, i + lane) : -1;
      const int r = count(x);
      if (i + lane < w1) p.row[i + lane] = row_of(x, r);
    }
  }
}

// A few slots (up to 256), a thread for each: its rank is counted directly (8 slots:
// 3.2 us by itself, the general kernel needs about 2 us more).
__global__ void __launch_bounds__(kSortThreads) k_moe_place_few(const __grid_constant__ SortParams p) {
  extern __shared__ int32_t sm[];
  int32_t* ids = sm;                  // [slots]
  int32_t* total = sm + kSortFew;     // [E] slots of each expert, then its first row
  __shared__ int32_t wsum[kSortThreads / 32];
  grid_dependency_wait();
  allow_dependent_launch();
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  const int x = i < p.slots ? expert_of(p, i) : -1;
  if (i < p.slots) ids[i] = x;
  if (i < p.experts) total[i] = 0;
  __syncthreads();
  if (x >= 0) atomicAdd(&total[x], 1);
  int rank = 0;
  if (warp * 32 < p.slots) {
    const int upto = min(warp * 32 + 32, p.slots);
    for (int j = 0; j < upto; ++j) rank += j < i && ids[j] == x;
  }
  __syncthreads();
  const int all = i < p.experts ? total[i] : 0;
  const int room = i >= p.experts ? 0 : p.capacity > 0 ? p.capacity : p.align == 1 ? all : (all + p.align - 1) / p.align * p.align;
  const int incl = warp_scan(room, lane);
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  const int base = warp_sum(lane < warp ? wsum[lane] : 0);
  if (i < p.experts) {
    total[i] = base + incl - room;
    p.offsets[i] = base + incl - room;
    p.counts[i] = p.capacity > 0 ? min(all, p.capacity) : all;
    if (i == p.experts - 1) p.offsets[p.experts] = base + incl;
  }
  __syncthreads();
  if (i < p.slots) p.row[i] = x >= 0 && (p.capacity == 0 || rank < p.capacity) ? total[x] + rank : -1;
}

// ---------------------------------------------------------------- rows

// What a thread moves at once: 16 bytes where the row length and all addresses
// are multiples of 16 bytes; else kMost units, a row of threads apart, of 4
// bytes or of one element of an odd row of bf16.  Four in flight are faster than
// one or eight for dispatch and combine (16384 x 4 rows of 2047 bf16: combine
// 108 us against 130 and 126; 2048 wide 60), one for the backward pass, which
// has more rows in flight anyway (169 us against 184 and 223; 2048 wide 97).
// A thread starts at first() and goes on kStep * tx elements later.
template <typename T, int kBytes, int kMost = kRowUnits> struct Piece {
  static constexpr int kUnit = kBytes / sizeof(T), kUnits = kBytes == 16 ? 1 : kMost;
  static constexpr int N = kUnit * kUnits, kStep = N;
  static constexpr int kWords = kBytes == 16 ? 4 : 1;   // registers of a unit
  uint32_t raw[kUnits][kWords];
  static __device__ __forceinline__ int64_t first(int thread) { return (int64_t)thread * kUnit; }
  __device__ __forceinline__ void load(const T* row, int64_t c, int64_t end, int tx) {
    if constexpr (kBytes == 16) {
      const uint4 t = *reinterpret_cast<const uint4*>(row + c);
      raw[0][0] = t.x; raw[0][1] = t.y; raw[0][2] = t.z; raw[0][3] = t.w;
    } else {
#pragma unroll
      for (int q = 0; q < kUnits; ++q) {
        const int64_t e = c + q * (tx * kUnit);
        raw[q][0] = 0u;
        if (kUnits == 1 || e < end) {   // the caller has looked at the first
          if constexpr (kBytes == 4) raw[q][0] = *reinterpret_cast<const uint32_t*>(row + e);
          else raw[q][0] = *reinterpret_cast<const uint16_t*>(row + e);
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* row, int64_t c, int64_t end, int tx) const {
    if constexpr (kBytes == 16) {
      *reinterpret_cast<uint4*>(row + c) = make_uint4(raw[0][0], raw[0][1], raw[0][2], raw[0][3]);
    } else {
#pragma unroll
      for (int q = 0; q < kUnits; ++q) {
        const int64_t e = c + q * (tx * kUnit);
        if (kUnits == 1 || e < end) {   // the caller has looked at the first
          if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(row + e) = raw[q][0];
          else *reinterpret_cast<uint16_t*>(row + e) = (uint16_t)raw[q][0];
        }
      }
    }
  }
  __device__ __forceinline__ void get(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < kUnits * kWords; ++i) {
      const uint32_t w = raw[i / kWords][i % kWords];
      if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w);
      else if constexpr (kBytes == 2) v[i] = __uint_as_float(w << 16);
      else {
        v[2 * i] = __uint_as_float(w << 16);
        v[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void set(const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < kUnits * kWords; ++i) {
      uint32_t& w = raw[i / kWords][i % kWords];
      if constexpr (sizeof(T) == 4) w = __float_as_uint(v[i]);
      else if constexpr (kBytes == 2) w = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
      else {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w = *reinterpret_cast<const uint32_t*>(&t);
      }
    }
  }
};

__device__ __forceinline__ float weight(const RowsParams& p, int64_t slot) {
  return p.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.w)[slot]) : static_cast<const float*>(p.w)[slot];
}

// Sets the rows of the sorted buffer that hold no token to zero: after each
// expert's last token up to the next expert, and after the last expert.  The
// warps of the launch's last CTAs share them, row by row.
template <typename T, int kBytes>
__device__ __forceinline__ void clear_rows(const RowsParams& p) {
  using P = Piece<T, kBytes>;
  const P zero = {};
  const int lane = threadIdx.x & 31;
  const uint32_t nw = (gridDim.x - p.token_ctas) * (kThreads256 / 32);
  const uint32_t me = (blockIdx.x - p.token_ctas) * (kThreads256 / 32) + (threadIdx.x >> 5);
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
    // this warp's first row of the expert: rows go to the warps in turn.  Each
    // lane looks at one expert, and only those with a row for this warp are
    // gone through (all of them in turn took 35 us for 232 experts)
    const uint32_t first = (uint32_t)lo + (me + nw - (uint32_t)lo % nw) % nw;
    unsigned some = __ballot_sync(0xffffffffu, lo < hi && first < (uint32_t)hi);
    while (some) {
      const int src = __ffs(some) - 1;
      some &= some - 1;
      const uint32_t a = __shfl_sync(0xffffffffu, first, src), b = __shfl_sync(0xffffffffu, (uint32_t)hi, src);
      for (uint32_t r = a; r < b; r += nw) {
        T* to = out + (int64_t)r * p.ldo;
        for (int64_t c = P::first(lane); c < p.hidden; c += 32 * P::kStep) zero.store(to, c, p.hidden, 32);
      }
    }
  }
}

// The rows and weights of a CTA's tokens, in shared memory: the row kernels
// then wait for memory once per row and not twice.  A row outside the buffer
// becomes -1.
struct Staged {
  int32_t* row;
  float* w;
};

__device__ __forceinline__ Staged stage(const RowsParams& p, int64_t t0, int nt) {
  extern __shared__ int32_t sm[];
  Staged s = {sm, reinterpret_cast<float*>(sm + p.tokens_per_cta * p.topk)};
  const int64_t slot = t0 * p.topk;
  for (int i = threadIdx.x; i < nt * p.topk; i += kThreads256) {
    const int r = p.row[slot + i];
    const bool has = (uint32_t)r < (uint32_t)p.rows;
    s.row[i] = has ? r : -1;
    s.w[i] = has && p.w ? weight(p, slot + i) : 1.f;
  }
  __syncthreads();
  return s;
}

template <typename T, int kBytes>
__global__ void __launch_bounds__(kThreads256) k_moe_dispatch(const __grid_constant__ RowsParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  using P = Piece<T, kBytes>;
  if ((int)blockIdx.x >= p.token_ctas) {
    clear_rows<T, kBytes>(p);
    return;
  }
  const int64_t t = (int64_t)blockIdx.x * p.tokens_per_cta + threadIdx.x / p.tx;
  if (t >= p.tokens) return;
  const T* x = static_cast<const T*>(p.x) + t * p.ldx;
  T* out = static_cast<T*>(p.out);
  const int32_t* row = p.row + t * p.topk;
  for (int64_t c = P::first(threadIdx.x % p.tx); c < p.hidden; c += p.tx * P::kStep) {
    P v;
    v.load(x, c, p.hidden, p.tx);
    for (int k = 0; k < p.topk; ++k) {
      const int r = row[k];
      if ((uint32_t)r < (uint32_t)p.rows) v.store(out + r * p.ldo, c, p.hidden, p.tx);
    }
  }
}

// Choices are taken kK at a time so that their rows are loaded together, and
// kU tokens, so that a thread has several rows in flight when a token has few.
// Five CTAs per SM where the registers allow (2 and 4 choices, 4096 and 6144
// wide: 105 and 96 us against 109 and 97 with four), else four (8 choices: 98 us;
// five would spill, 152 us, and three take 102 us).
template <typename T, int kBytes, int kK>
__global__ void __launch_bounds__(kThreads256, kK == 2 || kK == 4 ? 5 : 4) k_moe_combine(const __grid_constant__ RowsParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  using P = Piece<T, kBytes>;
  constexpr int N = P::N, kU = kK >= 4 ? 1 : 4 / kK;
  const int split = blockIdx.x % p.splits;   // of the row's columns
  const int64_t t0 = (int64_t)(blockIdx.x / p.splits) * p.tokens_per_cta;
  const int nt = (int)min((int64_t)p.tokens_per_cta, p.tokens - t0);
  const Staged st = stage(p, t0, nt);
  const int ty = kThreads256 / p.tx;
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out) + t0 * p.ldo;
  for (int j = (threadIdx.x / p.tx) * kU; j < nt; j += ty * kU) {
    const int64_t c0 = (int64_t)split * p.tx * P::kStep + P::first(threadIdx.x % p.tx);
    for (int64_t c = c0; c < p.hidden; c += (int64_t)p.splits * p.tx * P::kStep) {
      float acc[kU][N];
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int q = 0; q < N; ++q) acc[u][q] = 0.f;
      for (int k0 = 0; k0 < p.topk; k0 += kK) {   // once, unless topk > 8
        P v[kU][kK];
        int r[kU][kK];
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            r[u][k] = j + u < nt && k0 + k < p.topk ? st.row[(j + u) * p.topk + k0 + k] : -1;
            if (r[u][k] >= 0) v[u][k].load(x + r[u][k] * p.ldx, c, p.hidden, p.tx);
          }
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            if (r[u][k] < 0) continue;
            const float w = st.w[(j + u) * p.topk + k0 + k];
            float f[N];
            v[u][k].get(f);
#pragma unroll
            for (int q = 0; q < N; ++q) acc[u][q] = fmaf(w, f[q], acc[u][q]);
          }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (j + u >= nt) break;
        P o;
        o.set(acc[u]);
        o.store(out + (j + u) * p.ldo, c, p.hidden, p.tx);
      }
    }
  }
}

// Sums kN values over a warp, halving the number of values at each exchange
// while there are several: kN - 1 exchanges and log2(32 / kN) more instead of
// 5 kN.  Returns the sum of value `at`, which depends on the lane.
template <int kN>
__device__ __forceinline__ float warp_sums(float (&v)[kN], int lane, int& at) {
  at = 0;
  int o = 16;
#pragma unroll
  for (int n = kN; n > 1; n >>= 1, o >>= 1) {
    const bool up = lane & o;
    at = 2 * at + up;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      // the lower lane keeps the even value, the upper one the odd value
      const float give = up ? v[2 * i] : v[2 * i + 1], keep = up ? v[2 * i + 1] : v[2 * i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  for (; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

template <typename T, int kBytes, int kK>
__global__ void __launch_bounds__(kThreads256) k_moe_backward(const __grid_constant__ RowsParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  using P = Piece<T, kBytes, 1>;
  constexpr int N = P::N, kU = kK == 1 ? 4 : kK == 2 ? 2 : 1, kN = kU * kK;
  if ((int)blockIdx.x >= p.token_ctas) {
    clear_rows<T, kBytes>(p);
    return;
  }
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_cta;
  const int nt = (int)min((int64_t)p.tokens_per_cta, p.tokens - t0);
  const Staged st = stage(p, t0, nt);
  // tx is at least 32: a warp works on one row of tokens.  Its sums for the
  // dot products go to red[slot][warp of the row].
  float* red = st.w + p.tokens_per_cta * p.topk;
  const int ty = kThreads256 / p.tx, y0 = threadIdx.x / p.tx;
  const int lane = threadIdx.x & 31, warps = p.tx >> 5, warp = (threadIdx.x >> 5) % warps;
  const T* dout = static_cast<const T*>(p.x) + t0 * p.ldx;
  const T* y = static_cast<const T*>(p.y);
  T* out = static_cast<T*>(p.out);
  for (int j = y0 * kU; j < nt; j += ty * kU) {
    for (int k0 = 0; k0 < p.topk; k0 += kK) {
      float dot[kN];
      int r[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int u = i / kK, k = k0 + i % kK;
        dot[i] = 0.f;
        r[i] = j + u < nt && k < p.topk ? st.row[(j + u) * p.topk + k] : -1;
      }
      for (int64_t c = P::first(threadIdx.x % p.tx); c < p.hidden; c += p.tx * P::kStep) {
        P draw[kU], v[kN];
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (j + u < nt) draw[u].load(dout + (j + u) * p.ldx, c, p.hidden, p.tx);
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (r[i] >= 0) v[i].load(y + r[i] * p.ldy, c, p.hidden, p.tx);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          float d[N];
          draw[u].get(d);
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            const int i = u * kK + k;
            if (r[i] < 0) continue;
            const float w = st.w[(j + u) * p.topk + k0 + k];
            float f[N], o[N];
            v[i].get(f);
#pragma unroll
            for (int q = 0; q < N; ++q) {
              dot[i] = fmaf(d[q], f[q], dot[i]);
              o[q] = w * d[q];
            }
            P ro;
            ro.set(o);
            ro.store(out + r[i] * p.ldo, c, p.hidden, p.tx);
          }
        }
      }
      int at;
      const float s = warp_sums<kN>(dot, lane, at);
      // value `at`, its bits in the order in which the exchanges chose them
      int i = 0;
#pragma unroll
      for (int n = 1, q = kN >> 1; n < kN; n <<= 1, q >>= 1) i |= (at & q) ? n : 0;
      const int u = i / kK, k = k0 + i % kK;
      if (lane % (32 / kN) == 0 && j + u < nt && k < p.topk) red[((j + u) * p.topk + k) * warps + warp] = s;
    }
  }
  __syncthreads();
  const int64_t slot = t0 * p.topk;
  for (int i = threadIdx.x; i < nt * p.topk; i += kThreads256) {
    float s = 0.f;
    for (int q = 0; q < warps; ++q) s += red[i * warps + q];
    if (p.w_bf16) static_cast<__nv_bfloat16*>(p.dw)[slot + i] = __float2bfloat16_rn(s);
    else static_cast<float*>(p.dw)[slot + i] = s;
  }
}

// Shared memory of k_moe_place for a number of experts.
constexpr size_t place_bytes(int experts) { return ((size_t)(experts | 1) * (kSortThreads / 32) + experts) * 4; }

// More than 48 KB of shared memory has to be asked for.  Always the most that
// any number of experts needs: the limit belongs to the function, and a thread
// that set its own smaller need would take from another's launch.
template <typename F>
int opt_in_smem(F* kernel, size_t bytes) {
  if (bytes <= 48 * 1024) return 0;
  return (int)cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)place_bytes(kMoeMaxExperts));
}

// Shared memory of a row kernel: rows and weights of the CTA's slots, and the
// warps' parts of the dot products.
size_t staged_bytes(const RowsParams& p, bool backward) {
  return (size_t)p.tokens_per_cta * p.topk * (8 + (backward ? p.tx / 32 * 4 : 0));
}

template <typename T, int kBytes>
int launch_combine_k(const RowsParams& p, int grid, void* stream, bool pdl) {
  const size_t smem = staged_bytes(p, false);
  const dim3 g((unsigned)grid), b(kThreads256);
  if (p.topk == 1) return launch_kernel(k_moe_combine<T, kBytes, 1>, g, b, smem, stream, pdl, p);
  if (p.topk == 2) return launch_kernel(k_moe_combine<T, kBytes, 2>, g, b, smem, stream, pdl, p);
  if (p.topk <= 4) return launch_kernel(k_moe_combine<T, kBytes, 4>, g, b, smem, stream, pdl, p);
  return launch_kernel(k_moe_combine<T, kBytes, 8>, g, b, smem, stream, pdl, p);
}

template <typename T, int kBytes>
int launch_backward_k(const RowsParams& p, int grid, void* stream, bool pdl) {
  const size_t smem = staged_bytes(p, true);
  const dim3 g((unsigned)grid), b(kThreads256);
  if (p.topk == 1) return launch_kernel(k_moe_backward<T, kBytes, 1>, g, b, smem, stream, pdl, p);
  if (p.topk == 2) return launch_kernel(k_moe_backward<T, kBytes, 2>, g, b, smem, stream, pdl, p);
  if (p.topk <= 4) return launch_kernel(k_moe_backward<T, kBytes, 4>, g, b, smem, stream, pdl, p);
  return launch_kernel(k_moe_backward<T, kBytes, 8>, g, b, smem, stream, pdl, p);
}

}  // namespace

int launch_moe_sort_count(const SortParams& p, void* stream, bool pdl) {
  return launch_kernel(k_moe_count, dim3((unsigned)p.ctas), dim3(kSortThreads), (size_t)p.experts * 4, stream, pdl, p);
}

int launch_moe_sort_place(const SortParams& p, void* stream, bool pdl) {
  if (p.slots <= kSortFew) {
    const int threads = ((p.slots > p.experts ? p.slots : p.experts) + 31) / 32 * 32;
    return launch_kernel(k_moe_place_few, dim3(1), dim3((unsigned)threads), (size_t)(kSortFew + p.experts) * 4, stream, pdl, p);
  }
  const size_t smem = place_bytes(p.experts);
  const dim3 g((unsigned)p.ctas), b(kSortThreads);
  auto launch = [&](auto* kernel) {
    const int e = opt_in_smem(kernel, smem);
    return e ? e : launch_kernel(kernel, g, b, smem, stream, pdl, p);
  };
  // fewer registers for short runs: 2 us less at 16384 to 32768 slots
  if (p.per_cta <= 4 * kSortThreads) return launch(k_moe_place<4>);
  if (p.per_cta <= 16 * kSortThreads) return launch(k_moe_place<16>);
  return launch(k_moe_place<0>);
}

// Calls f with the element type and the bytes that a thread moves at once.
template <typename T, int kBytes> struct Kind {
  using Type = T;
  static constexpr int bytes = kBytes;
};
template <typename F>
int with_kind(bool bf16, int bytes, F f) {
  if (!bf16) return bytes == 16 ? f(Kind<float, 16>()) : f(Kind<float, 4>());
  if (bytes == 16) return f(Kind<__nv_bfloat16, 16>());
  return bytes == 4 ? f(Kind<__nv_bfloat16, 4>()) : f(Kind<__nv_bfloat16, 2>());
}

int launch_moe_dispatch(const RowsParams& p, bool bf16, int bytes, int grid, void* stream, bool pdl) {
  return with_kind(bf16, bytes, [&](auto k) {
    return launch_kernel(k_moe_dispatch<typename decltype(k)::Type, decltype(k)::bytes>, dim3((unsigned)grid),
                         dim3(kThreads256), 0, stream, pdl, p);
  });
}

int launch_moe_combine(const RowsParams& p, bool bf16, int bytes, int grid, void* stream, bool pdl) {
  return with_kind(bf16, bytes, [&](auto k) {
    return launch_combine_k<typename decltype(k)::Type, decltype(k)::bytes>(p, grid, stream, pdl);
  });
}

int launch_moe_backward(const RowsParams& p, bool bf16, int bytes, int grid, void* stream, bool pdl) {
  return with_kind(bf16, bytes, [&](auto k) {
    return launch_backward_k<typename decltype(k)::Type, decltype(k)::bytes>(p, grid, stream, pdl);
  });
}

}  // namespace muon
