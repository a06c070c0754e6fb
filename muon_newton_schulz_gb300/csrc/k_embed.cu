// Embedding rows with scaling, and their gradient by sorted tokens.
//
// out[t] = scale * table[id[t]];  dtable[v] = scale * sum of dout[t] over the
// tokens with id[t] = v, in the order of t.  The gradient sorts the tokens by id
// (stable, whole numbers only), sums runs of equal ids in registers and writes
// every row of dtable once: no atomic sums, the same bits on every call.  Tokens
// are summed in chunks of a fixed length; an id whose run crosses from one chunk
// to the next leaves fp32 sums of its parts, which a last kernel joins in order.
// All of it is bound by HBM on batches and by launches on a few tokens.
#include <cuda_runtime.h>

#include "launch_util.cuh"
#include "layer_internal.h"
#include "row_piece.cuh"

namespace muon {

namespace {

// The row of the table for token i, -1 for an id outside of it.
__device__ __forceinline__ int64_t row_of(const void* ids, bool ids64, int64_t vocab, int64_t i) {
  const int64_t v = ids64 ? static_cast<const int64_t*>(ids)[i] : (int64_t)static_cast<const int32_t*>(ids)[i];
  return v >= 0 && v < vocab ? v : -1;
}

// ---------------------------------------------------------------- rows

// kU tokens at a time, so that a thread has several rows in flight.
template <typename T, int kBytes, int kU>
__global__ void __launch_bounds__(kThreads256) k_embed(const __grid_constant__ EmbedParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  using P = Piece<T, kBytes>;
  constexpr int N = P::N;
  const int split = blockIdx.x % p.splits;   // of the row's columns
  const int64_t t0 = (int64_t)(blockIdx.x / p.splits) * p.tokens_per_cta;
  const int nt = (int)min((int64_t)p.tokens_per_cta, p.tokens - t0);
  const int ty = kThreads256 / p.tx;
  const T* table = static_cast<const T*>(p.table);
  T* out = static_cast<T*>(p.out) + t0 * p.ldo;
  for (int j = (threadIdx.x / p.tx) * kU; j < nt; j += ty * kU) {
    int64_t r[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) r[u] = j + u < nt ? row_of(p.ids, p.ids64, p.vocab, t0 + j + u) : -1;
    const int64_t c0 = (int64_t)split * p.tx * P::kStep + P::first(threadIdx.x % p.tx);
    for (int64_t c = c0; c < p.hidden; c += (int64_t)p.splits * p.tx * P::kStep) {
      P v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (r[u] >= 0) v[u].load(table + r[u] * p.ldt, c, p.hidden, p.tx);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (j + u >= nt) break;
        float f[N];
        if (r[u] >= 0) {
          v[u].get(f);
#pragma unroll
          for (int q = 0; q < N; ++q) f[q] *= p.scale;
        } else {
#pragma unroll
          for (int q = 0; q < N; ++q) f[q] = 0.f;
        }
        P o;
        o.set(f);
        o.store(out + (j + u) * p.ldo, c, p.hidden, p.tx);
      }
    }
  }
}

// ---------------------------------------------------------------- tokens sorted by id

__device__ __forceinline__ int warp_total(int v) { return __reduce_add_sync(0xffffffffu, v); }

__device__ __forceinline__ int warp_upto(int v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

__device__ __forceinline__ int32_t key_of(const IdSortParams& p, int64_t i) {
  if (p.key_in) return p.key_in[i];
  const int64_t r = row_of(p.ids, p.ids64, p.vocab, i);
  return r < 0 ? p.vocab : (int32_t)r;
}

// A few ids, a thread for each: its place is the number of smaller ids, and of
// equal ones before it.
__global__ void __launch_bounds__(kIdFew) k_id_sort_few(const __grid_constant__ IdSortParams p) {
  __shared__ int32_t key[kIdFew];
  grid_dependency_wait();
  allow_dependent_launch();
  const int i = threadIdx.x;
  const int32_t x = i < p.n ? key_of(p, i) : 0;
  key[i] = x;
  __syncthreads();
  if (i >= p.n) return;
  int place = 0;
  for (int j = 0; j < p.n; ++j) place += key[j] < x || (key[j] == x && j < i);
  p.key_out[place] = x;
  p.at_out[place] = i;
}

// One pass of a sort by digits, lowest first, each stable: counts of each digit
// in every CTA, then places.
__global__ void __launch_bounds__(kSortThreads) k_id_count(const __grid_constant__ IdSortParams p) {
  extern __shared__ int32_t sm[];
  for (int b = threadIdx.x; b < p.bins; b += kSortThreads) sm[b] = 0;
  __syncthreads();
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t i0 = (int64_t)blockIdx.x * p.per_cta;
  const int64_t i1 = min(i0 + p.per_cta, (int64_t)p.n);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads)
    atomicAdd(&sm[(key_of(p, i) >> p.shift) & (p.bins - 1)], 1);   // whole numbers: the order does not matter
  __syncthreads();
  for (int b = threadIdx.x; b < p.bins; b += kSortThreads) p.hist[(int64_t)b * p.ctas + blockIdx.x] = sm[b];
}

// Each warp has a run of consecutive tokens, 32 at a time: a token's rank among
// its warp's is the number of the warp's earlier tokens with that digit plus the
// lower lanes with it.  A run of at most kTile rounds stays in registers; with
// kTile = 0 the keys are read a second time.
static_assert(kSortThreads == 1024 && (1 << kIdDigitBits) <= kSortThreads, "thread b has digit b, lane w warp w's count");

template <int kTile>
__global__ void __launch_bounds__(kSortThreads) k_id_place(const __grid_constant__ IdSortParams p) {
  extern __shared__ int32_t sm[];
  constexpr int kWarps = kSortThreads / 32;
  const int bins = p.bins, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ld = bins | 1;             // odd: a warp then reads one digit's column without bank conflicts
  int32_t* start = sm;                 // [kWarps][ld] each warp's tokens of a digit, then the rank it starts at
  int32_t* total = sm + kWarps * ld;   // [bins] tokens of each digit in all CTAs, then its first place
  __shared__ int32_t wsum[kWarps];
  for (int i = threadIdx.x; i < kWarps * ld; i += kSortThreads) start[i] = 0;
  const int64_t i0 = (int64_t)blockIdx.x * p.per_cta;
  const int64_t i1 = min(i0 + p.per_cta, (int64_t)p.n);
  const int rounds = (int)((i1 - i0 + kSortThreads - 1) / kSortThreads);
  const int64_t w0 = min(i0 + (int64_t)warp * rounds * 32, i1), w1 = min(w0 + (int64_t)rounds * 32, i1);
  int32_t* mine = start + warp * ld;
  grid_dependency_wait();
  allow_dependent_launch();

  // the rank of lane's token (digit d, -1 for none) among the warp's; counts it
  auto count = [&](int d) {
    const unsigned same = __match_any_sync(0xffffffffu, d);
    const int rank = d >= 0 ? mine[d] + __popc(same & ((1u << lane) - 1)) : 0;
    __syncwarp();
    if (d >= 0 && (same >> lane) == 1u) mine[d] = rank + 1;   // the highest of its lanes
    __syncwarp();
    return rank;
  };
  auto digit = [&](int32_t k) { return (k >> p.shift) & (bins - 1); };
  int32_t key[kTile + 1];
  int rank[kTile + 1];
  if constexpr (kTile > 0) {
#pragma unroll
    for (int r = 0; r < kTile; ++r) key[r] = w0 + r * 32 + lane < w1 ? key_of(p, w0 + r * 32 + lane) : -1;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kTile; ++r)
      if (r < rounds) rank[r] = count(key[r] >= 0 ? digit(key[r]) : -1);
  } else {
    __syncthreads();
    for (int64_t i = w0 + lane; i < w1; i += 32) atomicAdd(&mine[digit(key_of(p, i))], 1);
  }
  __syncthreads();
  // a warp for each digit: lane w has warp w's tokens, and lane c, c + 32, ...
  // those of CTAs c, c + 32, ...
  constexpr int kAhead = 4, kLoads = (kIdGrid + 31) / 32;
  for (int d0 = warp; d0 < bins; d0 += kAhead * kWarps) {
    int before[kAhead], all[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) before[q] = all[q] = 0;
    if (p.hist) {
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int d = d0 + q * kWarps;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int c = lane + 32 * i;
          const int n = d < bins && c < p.ctas ? p.hist[(int64_t)d * p.ctas + c] : 0;
          all[q] += n;
          before[q] += c < (int)blockIdx.x ? n : 0;
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int d = d0 + q * kWarps;
      if (d >= bins) break;
      const int n = start[lane * ld + d];
      const int incl = warp_upto(n, lane);
      start[lane * ld + d] = warp_total(before[q]) + incl - n;
      const int sum = p.hist ? warp_total(all[q]) : incl;
      if (lane == 31) total[d] = sum;
    }
  }
  __syncthreads();
  const int d = threadIdx.x;   // first places: a sum over the smaller digits
  const int all = d < bins ? total[d] : 0;
  const int incl = warp_upto(all, lane);
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  const int base = warp_total(lane < warp ? wsum[lane] : 0);
  if (d < bins) total[d] = base + incl - all;
  __syncthreads();
  auto put = [&](int32_t k, int r, int64_t i) {
    const int place = total[digit(k)] + r;
    p.key_out[place] = k;
    p.at_out[place] = p.at_in ? p.at_in[i] : (int32_t)i;
  };
  if constexpr (kTile > 0) {
#pragma unroll
    for (int r = 0; r < kTile; ++r) {
      const int64_t i = w0 + r * 32 + lane;
      if (i < w1) put(key[r], mine[digit(key[r])] + rank[r], i);
    }
  } else {
    for (int64_t i = w0; i < w1; i += 32) {
      const int32_t k = i + lane < w1 ? key_of(p, i + lane) : -1;
      const int r = count(k >= 0 ? digit(k) : -1);
      if (k >= 0) put(k, r, i + lane);
    }
  }
}

// ---------------------------------------------------------------- sums

// The first of the n sorted keys that is at least v.
__device__ __forceinline__ int first_at_least(const int32_t* key, int n, int64_t v) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int m = lo + (hi - lo) / 2;
    if (key[m] < v) lo = m + 1;
    else hi = m;
  }
  return lo;
}

// Sets the rows of dtable without a token to zero: a warp looks at 32 rows, each
// lane for one.
template <typename T, int kBytes>
__device__ __forceinline__ void clear_unused(const EmbedGradParams& p) {
  using P = Piece<T, kBytes>;
  const P zero = {};
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)(gridDim.x - p.sum_ctas) * (kThreads256 / 32);
  const int64_t me = (int64_t)(blockIdx.x - p.sum_ctas) * (kThreads256 / 32) + (threadIdx.x >> 5);
  for (int64_t v0 = me * 32; v0 < p.vocab; v0 += warps * 32) {
    const int64_t v = v0 + lane;
    bool unused = v < p.vocab;
    if (unused) {
      const int i = first_at_least(p.key, p.n, v);
      unused = i == p.n || p.key[i] != v;
    }
    unsigned todo = __ballot_sync(0xffffffffu, unused);
    while (todo) {
      const int64_t row = v0 + __ffs(todo) - 1;
      todo &= todo - 1;
      T* to = static_cast<T*>(p.dtable) + row * p.lddt;
      for (int64_t c = P::first(lane); c < p.hidden; c += 32 * P::kStep) zero.store(to, c, p.hidden, 32);
    }
  }
}

// A group of tx threads sums a chunk of sorted tokens, kAhead rows in flight.
template <typename T, int kBytes>
__global__ void __launch_bounds__(kThreads256) k_embed_grad(const __grid_constant__ EmbedGradParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  if ((int)blockIdx.x >= p.sum_ctas) {
    clear_unused<T, kBytes>(p);
    return;
  }
  using P = Piece<T, kBytes, 1>;
  constexpr int N = P::N, kAhead = 8, kGroups = kThreads256 / 32;
  __shared__ int32_t keys[kGroups][kEmbedChunk + 2];   // of the chunk, and one on each side (-1: none)
  __shared__ int32_t tokens[kGroups][kEmbedChunk];
  const int split = blockIdx.x % p.splits, ty = kThreads256 / p.tx;
  const int group = threadIdx.x / p.tx, me = threadIdx.x % p.tx;
  const int64_t chunk = (int64_t)(blockIdx.x / p.splits) * ty + group;
  const int64_t i0 = chunk * p.chunk;
  const int n = (int)max((int64_t)0, min((int64_t)p.chunk, p.n - i0));
  for (int i = me; i < p.chunk + 2; i += p.tx) {
    const int64_t at = i0 + i - 1;
    keys[group][i] = at >= 0 && at < p.n ? p.key[at] : -1;
    if (i >= 1 && i <= n) tokens[group][i - 1] = p.at[at];
  }
  __syncthreads();
  const int32_t* key = keys[group] + 1;
  const int32_t* token = tokens[group];
  const T* dout = static_cast<const T*>(p.dout);
  for (int64_t c = (int64_t)split * p.tx * N + P::first(me); c < p.hidden; c += (int64_t)p.splits * p.tx * N) {
    float acc[N];
#pragma unroll
    for (int q = 0; q < N; ++q) acc[q] = 0.f;
    bool whole = key[-1] != key[0];   // the run of equal ids begins in this chunk
    for (int b = 0; b < n; b += kAhead) {
      P v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (b + u < n && key[b + u] < p.vocab) v[u].load(dout + token[b + u] * p.lddo, c, p.hidden, p.tx);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = b + u;
        if (i >= n || key[i] >= p.vocab) break;   // ids outside the table come last
        float f[N];
        v[u].get(f);
#pragma unroll
        for (int q = 0; q < N; ++q) acc[q] += f[q];
        if (key[i + 1] == key[i] && i + 1 < n) continue;
        const bool goes_on = key[i + 1] == key[i];
        if (whole && !goes_on) {
          P o;
#pragma unroll
          for (int q = 0; q < N; ++q) acc[q] *= p.scale;
          o.set(acc);
          o.store(static_cast<T*>(p.dtable) + (int64_t)key[i] * p.lddt, c, p.hidden, p.tx);
        } else {
          // slot 0: what an earlier chunk began; slot 1: what begins here and goes on
          float* to = p.part + (2 * chunk + (whole ? 1 : 0)) * p.ldp + c;
          if constexpr (N % 4 == 0) {
#pragma unroll
            for (int q = 0; q < N; q += 4) *reinterpret_cast<float4*>(to + q) = make_float4(acc[q], acc[q + 1], acc[q + 2], acc[q + 3]);
          } else {
#pragma unroll
            for (int q = 0; q < N; ++q) to[q] = acc[q];
          }
        }
#pragma unroll
        for (int q = 0; q < N; ++q) acc[q] = 0.f;
        whole = true;
      }
    }
  }
}

// Joins the parts of the ids whose runs begin in kEmbedJoin chunks and go on
// behind them, for 128 columns: a warp for each id with a few parts, the whole
// CTA for one with many.
template <typename T>
__global__ void __launch_bounds__(kThreads256) k_embed_join(const __grid_constant__ EmbedGradParams p) {
  constexpr int kWarps = kThreads256 / 32, kFew = 16;
  __shared__ int32_t ids[kEmbedJoin], more[kEmbedJoin];
  __shared__ float4 sums[kWarps][32];
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = (int64_t)blockIdx.y * kEmbedJoin;
  if (threadIdx.x < kEmbedJoin) {
    // chunks that the run goes on for behind the one it begins in, 0 for none
    const int64_t ch = first + threadIdx.x;
    int m = 0;
    int32_t k = 0;
    if (ch + 1 < p.chunks) {
      const int64_t a = ch * p.chunk, b = a + p.chunk;
      k = p.key[b - 1];
      const bool begins = p.key[a] != k || a == 0 || p.key[a - 1] != k;
      if (k < p.vocab && p.key[b] == k && begins) m = (first_at_least(p.key, p.n, (int64_t)k + 1) - 1) / p.chunk - (int)ch;
    }
    ids[threadIdx.x] = k;
    more[threadIdx.x] = m;
  }
  __syncthreads();
  const int64_t c = (int64_t)blockIdx.x * 128 + lane * 4;   // the parts' rows are padded to whole groups
  // part i of a run that begins in chunk ch
  auto part = [&](int64_t ch, int i) {
    return *reinterpret_cast<const float4*>(p.part + (i == 0 ? 2 * ch + 1 : 2 * (ch + i)) * p.ldp + c);
  };
  auto add = [](float4& a, const float4& b) { a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w; };
  auto sum = [&](int64_t ch, int from, int step, int upto) {   // parts from, from + step, ... up to upto
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    int i = from;
    for (; i + 3 * step <= upto; i += 4 * step) {
      const float4 a = part(ch, i), b = part(ch, i + step), d = part(ch, i + 2 * step), e = part(ch, i + 3 * step);
      add(acc, a); add(acc, b); add(acc, d); add(acc, e);
    }
    for (; i <= upto; i += step) add(acc, part(ch, i));
    return acc;
  };
  auto put = [&](int32_t id, const float4& s) {
    T* to = static_cast<T*>(p.dtable) + (int64_t)id * p.lddt + c;
    const float f[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + q < p.hidden) to[q] = (T)(f[q] * p.scale);
  };
  for (int i = warp; i < kEmbedJoin; i += kWarps)
    if (more[i] > 0 && more[i] < kFew) put(ids[i], sum(first + i, 0, 1, more[i]));
  for (int i = 0; i < kEmbedJoin; ++i) {
    if (more[i] < kFew) continue;
    sums[warp][lane] = sum(first + i, warp, kWarps, more[i]);
    __syncthreads();
    if (warp == 0) {
      float4 acc = sums[0][lane];
      for (int w = 1; w < kWarps; ++w) add(acc, sums[w][lane]);
      put(ids[i], acc);
    }
    __syncthreads();
  }
}

constexpr size_t place_bytes(int bins) { return ((size_t)(bins | 1) * (kSortThreads / 32) + bins) * 4; }

template <typename T, int kBytes>
int launch_embed_u(const EmbedParams& p, int grid, void* stream, bool pdl) {
  const dim3 g((unsigned)grid), b(kThreads256);
  if (p.tokens_per_cta >= 4 * (kThreads256 / p.tx)) return launch_kernel(k_embed<T, kBytes, 4>, g, b, 0, stream, pdl, p);
  return launch_kernel(k_embed<T, kBytes, 1>, g, b, 0, stream, pdl, p);
}

}  // namespace

int launch_embed(const EmbedParams& p, bool bf16, int bytes, int grid, void* stream, bool pdl) {
  return with_kind(bf16, bytes, [&](auto k) {
    return launch_embed_u<typename decltype(k)::Type, decltype(k)::bytes>(p, grid, stream, pdl);
  });
}

int launch_id_sort_few(const IdSortParams& p, void* stream, bool pdl) {
  const int threads = (p.n + 31) / 32 * 32;
  return launch_kernel(k_id_sort_few, dim3(1), dim3((unsigned)threads), 0, stream, pdl, p);
}

int launch_id_sort_count(const IdSortParams& p, void* stream, bool pdl) {
  return launch_kernel(k_id_count, dim3((unsigned)p.ctas), dim3(kSortThreads), (size_t)p.bins * 4, stream, pdl, p);
}

int launch_id_sort_place(const IdSortParams& p, void* stream, bool pdl) {
  const size_t smem = place_bytes(p.bins);
  auto launch = [&](auto* kernel) {
    if (smem > 48 * 1024) {   // the most that any digit needs: the limit belongs to the function, not to the launch
      const int e = (int)cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)place_bytes(1 << kIdDigitBits));
      if (e) return e;
    }
    return launch_kernel(kernel, dim3((unsigned)p.ctas), dim3(kSortThreads), smem, stream, pdl, p);
  };
  if (p.per_cta <= 2 * kSortThreads) return launch(k_id_place<2>);
  if (p.per_cta <= 16 * kSortThreads) return launch(k_id_place<16>);
  return launch(k_id_place<0>);
}

int launch_embed_grad(const EmbedGradParams& p, bool bf16, int bytes, int grid, void* stream, bool pdl) {
  return with_kind(bf16, bytes, [&](auto k) {
    return launch_kernel(k_embed_grad<typename decltype(k)::Type, decltype(k)::bytes>, dim3((unsigned)grid),
                         dim3(kThreads256), 0, stream, pdl, p);
  });
}

int launch_embed_join(const EmbedGradParams& p, bool bf16, void* stream, bool pdl) {
  const dim3 grid((unsigned)((p.hidden + 127) / 128), (unsigned)((p.chunks + kEmbedJoin - 1) / kEmbedJoin));
  if (bf16) return launch_kernel(k_embed_join<__nv_bfloat16>, grid, dim3(kThreads256), 0, stream, pdl, p);
  return launch_kernel(k_embed_join<float>, grid, dim3(kThreads256), 0, stream, pdl, p);
}

}  // namespace muon
