// Embedding rows with scaling, and their gradient by sorted tokens.
//
// out[t] = scale * table[id[t]];  dtable[v] = scale * sum of dout[t] over the
// tokens with id[t] = v, in the order of t.  The gradient sorts the tokens by id
// (stable, whole numbers only), while other CTAs clear dtable, and sums runs of equal
// ids in registers: no atomic sums, the same bits on every call.  Tokens
// are summed in chunks of a fixed length; an id whose run crosses from one chunk
// to the next leaves fp32 sums of its parts, which a last kernel joins in order.
// All of it is bound by HBM on batches and by launches on a few tokens: 65536 tokens of
// 2048 bf16, uneven as words are: rows 71 us (7.6 TB/s, frequent rows from L2),
// gradient with 65536 rows 117 us (4.6 TB/s counting what it has to move once): sort and
// clearing 46, sums 57, joining 11.  One token 3.8 us, 1003 tokens' gradient 15.
#include <cuda_runtime.h>

#include <type_traits>

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

__device__ __forceinline__ int warp_upto(int v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

// The launch's other CTAs clear rows of dtable meanwhile: the sort leaves most of the
// machine free.  (65536 tokens and rows, 2048 bf16 wide: 122 us; clearing only the rows
// without a token, beside the sums and found by search, took 128.  1003 tokens of 1001
// ids: 15 and 26.)
__device__ __forceinline__ bool clears_rows(const ZeroRows& z) {
  if ((int)blockIdx.x < z.first_cta) return false;
  const int64_t me = (int64_t)(blockIdx.x - z.first_cta) * blockDim.x + threadIdx.x;
  const int64_t step = (int64_t)(gridDim.x - z.first_cta) * blockDim.x;
  uint8_t* p = static_cast<uint8_t*>(z.p) + z.begin * z.pitch;
  const int64_t rows = z.end - z.begin;
  if ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)z.row_bytes | (uintptr_t)z.pitch) % 16 == 0) {
    const int64_t n = z.row_bytes / 16;
    if (z.row_bytes == z.pitch) {
      for (int64_t i = me; i < rows * n; i += step) reinterpret_cast<uint4*>(p)[i] = make_uint4(0u, 0u, 0u, 0u);
    } else {
      for (int64_t i = me; i < rows * n; i += step) reinterpret_cast<uint4*>(p + i / n * z.pitch)[i % n] = make_uint4(0u, 0u, 0u, 0u);
    }
  } else {   // elements of at least two bytes
    const int64_t n = z.row_bytes / 2;
    if (z.row_bytes == z.pitch && reinterpret_cast<uintptr_t>(p) % 2 == 0) {
      // up to the first and from the last 16-byte boundary by element
      const int64_t all = rows * n, head = min(all, (int64_t)((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16 / 2)), body = (all - head) / 8;
      uint16_t* q = reinterpret_cast<uint16_t*>(p);
      for (int64_t i = me; i < body; i += step) reinterpret_cast<uint4*>(q + head)[i] = make_uint4(0u, 0u, 0u, 0u);
      for (int64_t i = me; i < all - body * 8; i += step) q[i < head ? i : i + body * 8] = 0;
    } else {
      for (int64_t i = me; i < rows * n; i += step) reinterpret_cast<uint16_t*>(p + i / n * z.pitch)[i % n] = 0;
    }
  }
  return true;
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
  if (clears_rows(p.zero)) return;
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

// A sort by digits, lowest first, each pass stable.  hist[CTA][digit] counts the
// digits of each CTA's tokens: this kernel forms the first pass's and clears those
// of the others, which the pass before them counts while it places the tokens.
__global__ void __launch_bounds__(kThreads256) k_id_count(const __grid_constant__ IdSortParams p) {
  extern __shared__ int32_t sm[];
  for (int b = threadIdx.x; b < p.bins; b += kThreads256) sm[b] = 0;
  __syncthreads();
  grid_dependency_wait();
  allow_dependent_launch();
  if (clears_rows(p.zero)) return;
  for (int64_t i = (int64_t)blockIdx.x * kThreads256 + threadIdx.x; i < p.clear; i += (int64_t)p.ctas * kThreads256) p.hist_next[i] = 0;
  const int64_t i0 = (int64_t)blockIdx.x * p.per_cta;
  const int64_t i1 = min(i0 + p.per_cta, (int64_t)p.n);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads256)
    atomicAdd(&sm[key_of(p, i) & (p.bins - 1)], 1);   // whole numbers: the order does not matter
  __syncthreads();
  for (int b = threadIdx.x; b < p.bins; b += kThreads256) p.hist[blockIdx.x * p.bins + b] = sm[b];
}

// Adds up kPer digits' counts of all CTAs, and of those before this one, many loads in
// flight.
template <int kPer>
__device__ __forceinline__ void sum_counts(const IdSortParams& p, int d0, int (&before)[4], int (&all)[4]) {
  constexpr int kAhead = 32;
  for (int c0 = 0; c0 < p.ctas; c0 += kAhead) {
    int n[kAhead][kPer];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int32_t* h = p.hist + (int64_t)(c0 + u) * p.bins + d0;
      const bool has = c0 + u < p.ctas;
      if constexpr (kPer == 4) {
        const int4 v = has ? *reinterpret_cast<const int4*>(h) : make_int4(0, 0, 0, 0);
        n[u][0] = v.x; n[u][1] = v.y; n[u][2] = v.z; n[u][3] = v.w;
      } else if constexpr (kPer == 2) {
        const int2 v = has ? *reinterpret_cast<const int2*>(h) : make_int2(0, 0);
        n[u][0] = v.x; n[u][1] = v.y;
      } else {
        n[u][0] = has ? *h : 0;
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        all[q] += n[u][q];
        before[q] += c0 + u < (int)blockIdx.x ? n[u][q] : 0;
      }
  }
}

// Each warp has a run of consecutive tokens, 32 at a time: a token's rank among
// its warp's is the number of the warp's earlier tokens with that digit plus the
// lower lanes with it.  A run of at most kTile rounds stays in registers; with
// kTile = 0 the keys are read a second time.  A thread then has a digit, or a few:
// it sums those of the warps and of the CTAs before, which neighbours read side by side.
// (65536 ids, 512 digits, a pass: 10 us; a warp for each digit, with scans over 32
// warps, took 13.)
template <int kTile>
__global__ void __launch_bounds__(kThreads256) k_id_place(const __grid_constant__ IdSortParams p) {
  extern __shared__ int32_t sm[];
  constexpr int kWarps = kThreads256 / 32, kDigits = (1 << kIdDigitBits) / kThreads256;
  const int bins = p.bins, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t* start = sm;                   // [kWarps][bins] each warp's tokens of a digit, then the place it starts at
  __shared__ int32_t wsum[kWarps];
  for (int i = threadIdx.x; i < kWarps * bins; i += kThreads256) start[i] = 0;
  const int64_t i0 = (int64_t)blockIdx.x * p.per_cta;
  const int64_t i1 = min(i0 + p.per_cta, (int64_t)p.n);
  const int rounds = (int)((i1 - i0 + kThreads256 - 1) / kThreads256);
  const int64_t w0 = min(i0 + (int64_t)warp * rounds * 32, i1), w1 = min(w0 + (int64_t)rounds * 32, i1);
  int32_t* mine = start + warp * bins;
  grid_dependency_wait();
  allow_dependent_launch();
  if (clears_rows(p.zero)) return;

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
  // digits threadIdx.x * per .. + per - 1: tokens in this CTA, in those before, in all
  const int per = bins > kThreads256 ? bins / kThreads256 : 1, d0 = threadIdx.x * per;
  int before[kDigits], all[kDigits], sum = 0;
#pragma unroll
  for (int q = 0; q < kDigits; ++q) before[q] = all[q] = 0;
  if (d0 < bins) {
    if (p.hist) {
      if (per == 1) sum_counts<1>(p, d0, before, all);
      else if (per == 2) sum_counts<2>(p, d0, before, all);
      else sum_counts<4>(p, d0, before, all);
    } else {
#pragma unroll
      for (int q = 0; q < kDigits; ++q)
        for (int w = 0; q < per && w < kWarps; ++w) all[q] += start[w * bins + d0 + q];
    }
#pragma unroll
    for (int q = 0; q < kDigits; ++q) sum += all[q];
  }
  const int incl = warp_upto(sum, lane);
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int at = incl - sum;   // tokens with a smaller digit
  for (int w = 0; w < warp; ++w) at += wsum[w];
  if (d0 < bins) {
#pragma unroll
    for (int q = 0; q < kDigits; ++q) {
      if (q >= per) break;
      int place = at + before[q];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int n = start[w * bins + d0 + q];
        start[w * bins + d0 + q] = place;
        place += n;
      }
      at += all[q];
    }
  }
  __syncthreads();
  auto put = [&](int32_t k, int place, int64_t i) {
    p.key_out[place] = k;
    p.at_out[place] = p.at_in ? p.at_in[i] : (int32_t)i;
    if (p.hist_next) atomicAdd(&p.hist_next[place / p.per_cta * bins + ((k >> p.shift_next) & (bins - 1))], 1);
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
      const int place = count(k >= 0 ? digit(k) : -1);   // `mine` counts on from the place that the warp starts at
      if (k >= 0) put(k, place, i + lane);
    }
  }
}

// ---------------------------------------------------------------- sums

// A group of tx threads sums a chunk of sorted tokens, kAhead rows in flight.
template <typename T, int kBytes>
__global__ void __launch_bounds__(kThreads256) k_embed_grad(const __grid_constant__ EmbedGradParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
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
// behind them, for 256 columns: a warp for each id with a few parts, the whole
// CTA for one with many.
struct Columns8 {
  float v[8];   // columns 4 lane .. + 3, and the same 128 further on
  __device__ __forceinline__ void add(const Columns8& o) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += o.v[q];
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads256) k_embed_join(const __grid_constant__ EmbedGradParams p) {
  constexpr int kWarps = kThreads256 / 32, kFew = 16, kAhead = 4;
  __shared__ int32_t ids[kEmbedJoin], more[kEmbedJoin];
  __shared__ Columns8 sums[kWarps][32];
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int columns = (int)((p.hidden + 255) / 256);
  const int64_t first = (int64_t)(blockIdx.x / columns) * kEmbedJoin;
  if (threadIdx.x < kEmbedJoin) {
    // chunks that the run goes on for behind the one it begins in, 0 for none
    const int64_t ch = first + threadIdx.x;
    int m = 0;
    int32_t k = 0;
    if (ch + 1 < p.chunks) {
      const int64_t a = ch * p.chunk, b = a + p.chunk;
      k = p.key[b - 1];
      const int32_t next = p.key[b], own = p.key[a], last = a > 0 ? p.key[a - 1] : -1;
      if (k < p.vocab && next == k && (own != k || last != k)) {
        // chunks that begin with k: most runs end soon
        auto has = [&](int64_t j) { return ch + j < p.chunks && p.key[(ch + j) * p.chunk] == k; };
        int step = 1;
        m = 1;
        while (has(m + step)) {
          m += step;
          step *= 2;
        }
        for (step /= 2; step > 0; step /= 2)
          if (has(m + step)) m += step;
      }
    }
    ids[threadIdx.x] = k;
    more[threadIdx.x] = m;
  }
  __syncthreads();
  const int64_t c = (int64_t)(blockIdx.x % columns) * 256 + lane * 4;   // the parts' rows are padded to whole groups
  // part i of a run that begins in chunk ch
  auto part = [&](int64_t ch, int i) {
    const float* from = p.part + (i == 0 ? 2 * ch + 1 : 2 * (ch + i)) * p.ldp + c;
    Columns8 r;
    *reinterpret_cast<float4*>(r.v) = *reinterpret_cast<const float4*>(from);
    *reinterpret_cast<float4*>(r.v + 4) = *reinterpret_cast<const float4*>(from + 128);
    return r;
  };
  auto sum = [&](int64_t ch, int from, int step, int upto) {   // parts from, from + step, ... up to upto
    Columns8 acc = {};
    int i = from;
    for (; i + (kAhead - 1) * step <= upto; i += kAhead * step) {
      Columns8 v[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) v[q] = part(ch, i + q * step);
#pragma unroll
      for (int q = 0; q < kAhead; ++q) acc.add(v[q]);
    }
    for (; i <= upto; i += step) acc.add(part(ch, i));
    return acc;
  };
  auto put = [&](int32_t id, const Columns8& s) {
    T* row = static_cast<T*>(p.dtable) + (int64_t)id * p.lddt;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      T* to = row + c + 128 * h;
      alignas(16) T v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = (T)(s.v[4 * h + q] * p.scale);
      using Vec = std::conditional_t<sizeof(T) == 4, uint4, uint2>;
      if (c + 128 * h + 4 <= p.hidden && reinterpret_cast<uintptr_t>(to) % sizeof(Vec) == 0) {
        *reinterpret_cast<Vec*>(to) = *reinterpret_cast<const Vec*>(v);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c + 128 * h + q < p.hidden) to[q] = v[q];
      }
    }
  };
  for (int i = warp; i < kEmbedJoin; i += kWarps)
    if (more[i] > 0 && more[i] < kFew) put(ids[i], sum(first + i, 0, 1, more[i]));
  for (int i = 0; i < kEmbedJoin; ++i) {
    if (more[i] < kFew) continue;
    sums[warp][lane] = sum(first + i, warp, kWarps, more[i]);
    __syncthreads();
    if (warp == 0) {
      Columns8 acc = sums[0][lane];
      for (int w = 1; w < kWarps; ++w) acc.add(sums[w][lane]);
      put(ids[i], acc);
    }
    __syncthreads();
  }
}

static_assert((kThreads256 / 32) * (4 << kIdDigitBits) <= 48 * 1024, "shared memory that need not be asked for");

// CTAs that clear rows: as many as a few per SM have stores for.
int zero_ctas(const ZeroRows& z) {
  const int64_t ctas = ((z.end - z.begin) * z.row_bytes + 16 * kThreads256 * 4 - 1) / (16 * kThreads256 * 4);
  return (int)(ctas < 152 * 6 ? ctas : 152 * 6);
}

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
  const int threads = p.n <= kThreads256 ? kThreads256 : kIdFew;
  return launch_kernel(k_id_sort_few, dim3((unsigned)(p.zero.first_cta + zero_ctas(p.zero))), dim3((unsigned)threads), 0, stream, pdl, p);
}

int launch_id_sort_count(const IdSortParams& p, void* stream, bool pdl) {
  return launch_kernel(k_id_count, dim3((unsigned)(p.ctas + zero_ctas(p.zero))), dim3(kThreads256), (size_t)p.bins * 4, stream, pdl, p);
}

int launch_id_sort_place(const IdSortParams& p, void* stream, bool pdl) {
  const size_t smem = (size_t)p.bins * (kThreads256 / 32) * 4;
  const dim3 g((unsigned)(p.ctas + zero_ctas(p.zero))), b(kThreads256);
  if (p.per_cta <= 4 * kThreads256) return launch_kernel(k_id_place<4>, g, b, smem, stream, pdl, p);
  if (p.per_cta <= 16 * kThreads256) return launch_kernel(k_id_place<16>, g, b, smem, stream, pdl, p);
  return launch_kernel(k_id_place<0>, g, b, smem, stream, pdl, p);
}

int launch_embed_grad(const EmbedGradParams& p, bool bf16, int bytes, int grid, void* stream, bool pdl) {
  return with_kind(bf16, bytes, [&](auto k) {
    return launch_kernel(k_embed_grad<typename decltype(k)::Type, decltype(k)::bytes>, dim3((unsigned)grid),
                         dim3(kThreads256), 0, stream, pdl, p);
  });
}

int launch_embed_join(const EmbedGradParams& p, bool bf16, void* stream, bool pdl) {
  // one dimension: 2^31 tokens are more groups of chunks than fit another
  const dim3 grid((unsigned)((p.hidden + 255) / 256 * ((p.chunks + kEmbedJoin - 1) / kEmbedJoin)));
  if (bf16) return launch_kernel(k_embed_join<__nv_bfloat16>, grid, dim3(kThreads256), 0, stream, pdl, p);
  return launch_kernel(k_embed_join<float>, grid, dim3(kThreads256), 0, stream, pdl, p);
}

}  // namespace muon
