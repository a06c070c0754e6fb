// Gated feed-forward products in bf16 on the tensor cores: tcgen05 MMAs of CTA
// pairs with accumulators in TMEM, operands through TMA.
//
// One persistent, warp-specialised kernel.  A pair of CTAs on two SMs computes
// tiles of 256 x 256: each loads 128 rows of the left operand and 128 columns of
// the right one per step of 64, the even CTA issues the MMAs for both, and the
// accumulators (256 columns of TMEM, twice) let the epilogue of a tile run while
// the next one is summed.
//   rows x weights (forward, dh, dx): 256 rows of an expert's tokens; the tile list
//     is formed from the counts on the device.  Rows behind the expert's last are
//     loaded as far as a box of 64 reaches (they are the next expert's) and not stored;
//     a tile with at most 128 rows takes MMAs of 128.  For h the 256 columns are 128 of the gate and the
//     same 128 of the up projection, 64 of each from either CTA, so that a thread
//     has both of an element; the unit and its gradient are formed in the epilogue.
//     Where y or dx have few tiles, pairs share a tile's depth: each leaves its
//     sums in fp32, and a second kernel adds them up.
//   weights' gradients: sums over an expert's rows, both operands MN-major as they
//     lie.  Here the rows behind an expert's last must count as zero: every
//     expert has tensor maps of its own rows (k_ffn_maps), which end there.
//
// Bound by the tensor cores: 16 experts of 1024 rows each, 2048 x 8192, forward 866 us, 1.905
// PFLOP/s.  A stage of 64 takes 512 clocks of MMAs and brings 32 KB into each SM; one
// thread issues its copies and one its MMAs, each in about that time, so their loops form
// no addresses (h 700 -> 673 us).  A tile of 128 rows takes 0.6-0.8 of a full one's time.
// 16384 rows that a router spread over the 16 experts, each launch by itself: h 673 us
// (1.63 PFLOP/s), y 330 (1.67), dh 488 (1.13: its epilogue loads two values an element
// and stores two), dx 659 (1.67), the weights 964 (1.71), the rows counted that hold a
// token; one row in nine of the MMAs holds none.
//
// Every wait is bounded (one second): on a time-out the kernel records the role in
// the status word, lets its copies and MMAs in flight finish, frees its TMEM and
// returns.
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include <atomic>

#include "code8.cuh"
#include "ffn_act.cuh"
#include "ffn_rows.cuh"
#include "launch_util.cuh"
#include "muon_internal.h"
#include "ptx_rows.cuh"

namespace muon {

namespace {

// Words of the waits that ran out, and what a handle has read of one last (its own place:
// a word that several handles share may be read by two of them at once).
__device__ uint32_t g_ffn_status[kFfnStatusWords], g_ffn_taken[kFfnStatusWords];

constexpr int TM = 256, TN = 256;           // output tile of a pair
constexpr int TK = 64, UK = 16;             // depth of a stage, of an MMA
constexpr int kHalf = 128;                  // rows and columns that a CTA of the pair loads
constexpr int kOperand = kHalf * TK * 2;    // 16 KiB
constexpr int kStageBytes = 2 * kOperand;
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kTmemCols = 2 * TN;
constexpr int kMaxExperts = 1024;
constexpr int kGroup = 8;                   // row tiles that share a walk over the columns
constexpr uint64_t kWaitLimitNs = 1000000000ull;

struct Table {                              // of the experts, in shared memory
  int32_t begin[kMaxExperts + 1];           // first row tile
  int32_t offset[kMaxExperts];
  int32_t count[kMaxExperts];
  int32_t part[kThreads / 32];
};
constexpr int kSmemBytes = 1024 + kStages * kStageBytes + (int)sizeof(Table) + 256;
static_assert(kSmemBytes <= 232448, "shared memory over the per-CTA limit");

struct Bars {
  uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], drain;
  uint32_t tmem;
  int32_t abort;
};
static_assert(sizeof(Bars) <= 256, "barriers");

__device__ __forceinline__ uint32_t* status_of(const FfnTcParams& p) { return &g_ffn_status[p.status]; }

__device__ __forceinline__ bool wait_drain(uint64_t* bar, uint32_t parity) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity))
    if (ptx::globaltimer() - t0 > kWaitLimitNs) return false;
  return true;
}

// ---------------------------------------------------------------- tiles

struct Tile {
  int expert, row, col;     // first row (of the expert's) and column
  int count, offset;        // the expert's rows
  int k0, nk;               // first step of the depth, and how many
  int job, split;
  bool half;                // at most 128 rows are left: an MMA of 128
};

template <FfnProduct kWhat>
struct Walk {
  static constexpr bool kWeight = kWhat == FfnProduct::kWeight;
  static constexpr bool kSplits = kWhat == FfnProduct::kDown || kWhat == FfnProduct::kInput;
  const FfnTcParams& p;
  const Table& table;
  int t, step, total;
  int e = 0;
  __device__ Walk(const FfnTcParams& p_, const Table& table_) : p(p_), table(table_), t(blockIdx.x >> 1), step(gridDim.x >> 1) {
    total = kWeight ? p.r.experts * p.tiles_per_expert : table.begin[p.r.experts] * p.nt * (kSplits ? p.splits : 1);
  }
  __device__ __forceinline__ bool more() const { return t < total; }
  __device__ __forceinline__ void next() { t += step; }
  __device__ __forceinline__ Tile tile() {
    Tile x;
    int local, mt, nt;
    x.split = kSplits ? t % p.splits : 0;
    const int t0 = kSplits ? t / p.splits : t;   // the tile
    if (kWeight) {
      x.expert = t / p.tiles_per_expert;
      local = t - x.expert * p.tiles_per_expert;
      x.job = 0;
      while (x.job + 1 < p.jobs && local >= p.job[x.job + 1].begin) ++x.job;
      local -= p.job[x.job].begin;
      mt = p.job[x.job].mt;
      nt = p.job[x.job].nt;
    } else {
      while (t0 >= table.begin[e + 1] * p.nt) ++e;
      x.expert = e;
      x.job = 0;
      local = t0 - table.begin[e] * p.nt;
      mt = table.begin[e + 1] - table.begin[e];
      nt = p.nt;
    }
    // kGroup row tiles at a time, their rows fastest: pairs that run at once share
    // rows of both operands
    const int group = local / (kGroup * nt), rest = local - group * (kGroup * nt);
    const int rows = min(kGroup, mt - group * kGroup);
    x.col = rest / rows;
    x.row = (group * kGroup + rest - x.col * rows) * TM;
    x.col *= kWhat == FfnProduct::kGated ? TN / 2 : TN;
    x.count = table.count[x.expert];
    x.offset = table.offset[x.expert];
    x.half = !kWeight && x.count - x.row <= TM / 2;
    x.k0 = 0;
    x.nk = kWeight ? (x.count + TK - 1) / TK : kWhat == FfnProduct::kInput ? 2 * p.nk : p.nk;
    if (kSplits && p.splits > 1) {
      const int share = (x.nk + p.splits - 1) / p.splits;
      x.k0 = x.split * share;
      x.nk = min(share, x.nk - x.k0);
    }
    return x;
  }
};

// Rows of each expert, and where its row tiles begin.  All threads.
__device__ __forceinline__ void fill_table(const FfnRows& r, Table& table) {
  const int per = (r.experts + kThreads - 1) / kThreads, e0 = (int)threadIdx.x * per;
  int sum = 0;
  for (int e = e0; e < min(e0 + per, r.experts); ++e) {
    const FfnExpert x = ffn_expert(r, e);
    table.offset[e] = x.offset;
    table.count[e] = x.count;
    sum += (x.count + TM - 1) / TM;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) table.part[warp] = upto;
  __syncthreads();
  int at = upto - sum;
  for (int w = 0; w < warp; ++w) at += table.part[w];
  for (int e = e0; e < min(e0 + per, r.experts); ++e) {
    table.begin[e] = at;
    at += (table.count[e] + TM - 1) / TM;
    if (e == r.experts - 1) table.begin[r.experts] = at;
  }
  __syncthreads();
}

// ---------------------------------------------------------------- loads

// One thread issues the copies of a stage while the one before it is multiplied, and
// its instructions one after another take about as long as that: addresses are formed
// once, and what depends on the CTA's place in the pair is a parameter.
template <FfnProduct kWhat, bool kBMn, int kRank>
__device__ __forceinline__ void run_producer(const FfnTcParams& p, const Table& table, uint8_t* stages, Bars& bars) {
  constexpr bool kWeight = kWhat == FfnProduct::kWeight, kGated = kWhat == FfnProduct::kGated;
  constexpr int kBox = 64 * TK * 2;   // 64 rows or columns x 64 deep
  volatile int* abort = &bars.abort;
  const uint32_t smem = ptx::smem_u32(stages), full = ptx::smem_u32(&bars.full[0]), even = ptx::mapa(full, 0);
  int stage = 0;
  uint32_t phase = 0, outstanding = 0, parity = 0;
  bool ok = true;
  int known = -1;
  for (Walk<kWhat> w(p, table); ok && w.more(); w.next()) {
    const Tile x = w.tile();
    const CUtensorMap *ma = &p.a[0], *mb = &p.b[0];
    if (kWeight) {
      ma = p.maps + p.job[x.job].p * p.r.experts + x.expert;
      mb = p.maps + p.job[x.job].q * p.r.experts + x.expert;
      const int which = x.expert * 4 + x.job;
      if (which != known && x.nk > 0) {   // maps of a kernel before this one
        ptx::fence_tensormap_acquire(ma);
        ptx::fence_tensormap_acquire(mb);
        known = which;
      }
    }
    const int per_cta = x.half ? kHalf / 2 : kHalf;   // rows that a CTA has of the tile
    const int arow = (kWeight ? 0 : x.offset) + x.row + per_cta * kRank;
    // boxes of 64 rows that hold one of the expert's; the others are not needed
    auto boxes_of = [&](int r) { return min(max((x.count - x.row - per_cta * r + 63) / 64, 0), per_cta / 64); };
    const int boxes = kWeight ? 2 : boxes_of(kRank);
    // one copy of 128 rows, or of 64
    if (!kWeight && boxes < 2) ma = &p.a_few[0];
    const uint32_t bytes = (kWeight ? 4 : boxes_of(0) + boxes_of(1)) * kBox + 2u * kOperand;
    const int bcol = kGated ? x.col + 64 * kRank : x.col + kHalf * kRank;
    int k0 = x.k0 * TK;
    int left = kWhat == FfnProduct::kInput ? p.nk - x.k0 : x.nk;   // steps of the first pair of operands
    for (int kb = 0; kb < x.nk; ++kb, k0 += TK, --left) {
      if (kWhat == FfnProduct::kInput && (left == 0 || (kb == 0 && left < 0))) {   // the second pair
        ma = boxes < 2 ? &p.a_few[1] : &p.a[1];
        mb = &p.b[1];
        k0 -= p.nk * TK;
      }
      if (!ptx::mbar_wait_bounded(&bars.empty[stage], phase ^ 1u, abort, status_of(p), kStatusTimeoutProducer, kWaitLimitNs)) {
        ok = false;
        break;
      }
      outstanding &= ~(1u << stage);
      const uint32_t sa = smem + stage * kStageBytes, sb = sa + kOperand, at = (kRank == 0 ? full : even) + 8 * stage;
      if (!p.withhold_loads) {
        // the even CTA's barrier counts the bytes of both
        if (kRank == 0) ptx::mbar_arrive_expect_tx(&bars.full[stage], bytes);
        auto load = [&](uint32_t to, const CUtensorMap* m, int c0, int c1, int c2) { ptx::tma_load_4d_rank<kRank>(to, m, c0, c1, c2, at); };
        if (kWeight) {
          load(sa, ma, arow, k0, 0);
          load(sa + kBox, ma, arow + 64, k0, 0);
          load(sb, mb, bcol, k0, 0);
          load(sb + kBox, mb, bcol + 64, k0, 0);
        } else {
          if (kRank == 0 || boxes > 0) load(sa, ma, k0, arow, 0);
          if (kGated) {   // 64 columns of gate and the same of up
            load(sb, &p.b[0], kBMn ? bcol : k0, kBMn ? k0 : bcol, x.expert);
            load(sb + kBox, &p.b[1], kBMn ? bcol : k0, kBMn ? k0 : bcol, x.expert);
          } else if (kBMn) {
            load(sb, mb, bcol, k0, x.expert);
            load(sb + kBox, mb, bcol + 64, k0, x.expert);
          } else {
            load(sb, mb, k0, bcol, x.expert);
          }
        }
        outstanding |= 1u << stage;
      }
      parity = (parity & ~(1u << stage)) | (phase << stage);
      if (++stage == kStages) { stage = 0; phase ^= 1u; }
    }
  }
  if (!ok && kRank == 0) {
    // let every copy issued (the odd CTA's complete on these barriers too) land
    // before the CTAs exit
    for (int s = 0; s < kStages; ++s)
      if ((outstanding >> s) & 1u)
        if (!wait_drain(&bars.full[s], (parity >> s) & 1u)) atomicOr(status_of(p), kStatusTimeoutDrain);
  }
}

// ---------------------------------------------------------------- MMAs

template <FfnProduct kWhat, bool kBMn>
__device__ __forceinline__ void run_mma(const FfnTcParams& p, const Table& table, uint8_t* stages, Bars& bars) {
  constexpr bool kAMn = kWhat == FfnProduct::kWeight;
  constexpr uint32_t whole = ptx::idesc_bf16(TM, TN, kAMn, kBMn), half = ptx::idesc_bf16(TM / 2, TN, kAMn, kBMn);
  volatile int* abort = &bars.abort;
  // K-major, 128B swizzle: 8-row groups 1024 B apart, the depth is an offset in the
  // swizzled row.  MN-major: blocks of 64 columns 8 KiB apart, groups of 8 deep 1024 B
  // apart.  A stage, and a step of 16 in it, add to the address alone (in 16 bytes).
  constexpr uint32_t kAStep = (kAMn ? UK * 128 : UK * 2) / 16, kBStep = (kBMn ? UK * 128 : UK * 2) / 16;
  const uint32_t smem = ptx::smem_u32(stages);
  const uint64_t a0 = ptx::smem_desc(smem, kAMn ? 64 * TK * 2 : 16, 1024);
  const uint64_t b0 = ptx::smem_desc(smem + kOperand, kBMn ? 64 * TK * 2 : 16, 1024);
  int stage = 0, acc = 0;
  uint32_t phase = 0, acc_phase = 0;
  bool ok = true, issued = false;
  for (Walk<kWhat> w(p, table); ok && w.more(); w.next()) {
    const Tile x = w.tile();
    if (x.nk == 0) continue;
    if (!ptx::mbar_wait_bounded_cluster(&bars.tempty[acc], acc_phase ^ 1u, abort, status_of(p), kStatusTimeoutMma, kWaitLimitNs)) {
      ok = false;
      break;
    }
    ptx::tc_fence_after();
    const uint32_t d = bars.tmem + (uint32_t)(acc * TN), idesc = x.half ? half : whole;
    for (int kb = 0; kb < x.nk; ++kb) {
      if (!ptx::mbar_wait_bounded(&bars.full[stage], phase, abort, status_of(p), kStatusTimeoutMma, kWaitLimitNs)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      const uint64_t ad = a0 + (uint32_t)stage * (kStageBytes / 16), bd = b0 + (uint32_t)stage * (kStageBytes / 16);
#pragma unroll
      for (int kk = 0; kk < TK / UK; ++kk)
        ptx::umma_f16_pair(d, ad + kk * kAStep, bd + kk * kBStep, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
      ptx::umma_commit_pair_mc(&bars.empty[stage], 0x3);   // frees the stage in both CTAs
      issued = true;
      if (++stage == kStages) { stage = 0; phase ^= 1u; }
    }
    if (!ok) break;
    ptx::umma_commit_pair_mc(&bars.tfull[acc], 0x3);
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
  if (!ok && issued) {
    ptx::umma_commit_pair_mc(&bars.drain, 0x1);
    if (!wait_drain(&bars.drain, 0)) atomicOr(status_of(p), kStatusTimeoutDrain);
  }
}

// ---------------------------------------------------------------- epilogues

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 32 values of a row on a 64-byte boundary: each thread writes whole sectors.
__device__ __forceinline__ void put32(void* row, int64_t c, const float (&f)[32]) {
  __nv_bfloat16* to = static_cast<__nv_bfloat16*>(row) + c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack2(f[16 * h + 2 * i], f[16 * h + 2 * i + 1]);
    ptx::st_global_32(to + 16 * h, w);
  }
}

// Up to 32 values of a row of n columns, with stores of `vec` bytes where they fit.
__device__ __forceinline__ void put_some(__nv_bfloat16* row, int64_t c, int64_t n, int vec, const float (&f)[32]) {
  if (vec == 32 && c + 32 <= n) {
    put32(row, c, f);
  } else if (vec >= 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c + 8 * i + 8 <= n) {
        *reinterpret_cast<uint4*>(row + c + 8 * i) =
            make_uint4(pack2(f[8 * i], f[8 * i + 1]), pack2(f[8 * i + 2], f[8 * i + 3]), pack2(f[8 * i + 4], f[8 * i + 5]),
                       pack2(f[8 * i + 6], f[8 * i + 7]));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + 8 * i + j < n) row[c + 8 * i + j] = __float2bfloat16_rn(f[8 * i + j]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (c + j < n) row[c + j] = __float2bfloat16_rn(f[j]);
  }
}

// Keeps 32 values of a row in 8 or 16 bits: one block of their format.
// Returns the scale byte.
template <bool k8>
__device__ __forceinline__ uint32_t keep32(void* codes, int64_t row, int64_t c, int64_t ldf, const float (&f)[32]) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) most = max(most, finite_bits(f[i]));
  const uint32_t s = k8 ? scale_byte(most) : scale_byte16(most);
  const float up = scale_up(s);
  const int64_t at = row * ldf + c;
#pragma unroll
  for (int h = 0; h < (k8 ? 1 : 2); ++h) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (k8) w[i] = encode2(f[4 * i], f[4 * i + 1], up) | encode2(f[4 * i + 2], f[4 * i + 3], up) << 16;
      else w[i] = encode16(f[16 * h + 2 * i], f[16 * h + 2 * i + 1], up);
    }
    ptx::st_global_32(static_cast<uint8_t*>(codes) + (k8 ? at : 2 * at + 32 * h), w);
  }
  return s;
}

// 32 kept values of a row, as they lie in memory.
template <bool k8> struct Kept32 {
  uint32_t w[k8 ? 8 : 16];
  __device__ __forceinline__ void load(const void* from, int64_t at) {
    const uint8_t* codes = static_cast<const uint8_t*>(from) + (k8 ? at : 2 * at);
    ptx::ld_global_32(codes, reinterpret_cast<uint32_t(&)[8]>(w[0]));
    if constexpr (!k8) ptx::ld_global_32(codes + 32, reinterpret_cast<uint32_t(&)[8]>(w[8]));
  }
  __device__ __forceinline__ float2 get(int j, float scale) const {   // values 2 j and 2 j + 1; j is known to the compiler
    const float2 f = k8 ? decode2(w[j / 2] >> (j & 1 ? 16 : 0)) : decode16(w[j]);
    return make_float2(f.x * scale, f.y * scale);
  }
};

__device__ __forceinline__ void load_acc(uint32_t taddr, float (&f)[32]) {
  uint32_t v[32];
  ptx::tmem_ld_32x32b_x32(taddr, v);
  ptx::tmem_ld_wait_regs(v);
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
}

// What a warp has of a tile: rows `row` .. + 31 of its expert's and `chunks` times 32
// columns from `col` on (of the tile), which stand at column `acc` of the
// accumulators.  An MMA of 128 rows leaves 64 of them to each CTA, the first half of
// the columns in lanes 0 .. 63 of TMEM and the second in the others.
struct Part { int row, col, acc, chunks; };

template <FfnProduct kWhat>
__device__ __forceinline__ Part part_of(const Tile& x, int rank, int quarter, int slice) {
  constexpr bool kGated = kWhat == FfnProduct::kGated;
  if (x.half) {
    const int row = x.row + kHalf / 2 * rank + 32 * (quarter & 1), side = quarter >> 1;
    return kGated ? Part{row, 64 * side + 32 * slice, 32 * slice, 1} : Part{row, 128 * side + 64 * slice, 64 * slice, 2};
  }
  const int row = x.row + kHalf * rank + 32 * quarter;
  return kGated ? Part{row, 64 * slice, 128 * slice, 2} : Part{row, 128 * slice, 128 * slice, 4};
}

// A tile of dh: dg, du (and h, where the forward pass did not keep it).
template <bool k8, int kAct>
__device__ __forceinline__ void slope_tile(const FfnTcParams& p, const Part& part, uint32_t tbase, int64_t row, bool valid, int64_t c0,
                                           uint64_t* tfull, uint32_t parity, volatile int* abort, bool& ok) {
  Kept32<k8> g[2], u[2];
  const int64_t at0 = row * p.ldf + c0;
  auto fetch = [&](int i, int b) {
    if (!valid || i >= part.chunks || c0 + 32 * i >= p.ldf) return;
    g[b].load(p.saved.gate, at0 + 32 * i);
    u[b].load(p.saved.up, at0 + 32 * i);
  };
  // while the sums of the tile go on: the first chunk, and the scale bytes of all (a row
  // has a multiple of four of them; 16384 rows 2048 x 8192: 515 us, byte by byte 554)
  fetch(0, 0);
  uint32_t gs = 0, us = 0;
  if (valid && c0 < p.ldf) {
    const int64_t word = at0 / 128, shift = at0 / 32 % 4 * 8;
    gs = reinterpret_cast<const uint32_t*>(p.saved.gate_scales)[word] >> shift;
    us = reinterpret_cast<const uint32_t*>(p.saved.up_scales)[word] >> shift;
  }
  ok = ptx::mbar_wait_bounded(tfull, parity, abort, status_of(p), kStatusTimeoutEpilogue, kWaitLimitNs);
  if (!ok) return;
  ptx::tc_fence_after();
  // two chunks a round: less code for the instruction cache (8 bits: 418 us against 430)
#pragma unroll 1
  for (int i0 = 0; i0 < part.chunks; i0 += 2) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int i = i0 + b;
      if (c0 + 32 * i >= p.ldf) break;
      fetch(i + 1, b ^ 1);
      float dh[32];
      load_acc(tbase + (uint32_t)(part.acc + 32 * i), dh);
      if (!valid) continue;
      const float gscale = scale_down(gs >> (8 * i) & 255u), uscale = scale_down(us >> (8 * i) & 255u);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t wg[8], wu[8], wh[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int k = 8 * h + j;
          const float2 gv = g[b].get(k, gscale), uv = u[b].get(k, uscale);
          const FfnSlope s0 = ffn_act<true, kAct>(gv.x), s1 = ffn_act<true, kAct>(gv.y);
          wg[j] = pack2(dh[2 * k] * uv.x * s0.slope, dh[2 * k + 1] * uv.y * s1.slope);
          wu[j] = pack2(dh[2 * k] * s0.act, dh[2 * k + 1] * s1.act);
          if (k8) wh[j] = pack2(s0.act * uv.x, s1.act * uv.y);
        }
        const int64_t at = at0 + 32 * i + 16 * h;
        ptx::st_global_32(static_cast<__nv_bfloat16*>(p.dgate) + at, wg);
        ptx::st_global_32(static_cast<__nv_bfloat16*>(p.dup) + at, wu);
        if (k8) ptx::st_global_32(static_cast<__nv_bfloat16*>(p.act) + at, wh);
      }
    }
  }
}

template <FfnProduct kWhat, int kAct>
__device__ __forceinline__ void run_epilogue(const FfnTcParams& p, const Table& table, int rank, Bars& bars) {
  constexpr bool kWeight = kWhat == FfnProduct::kWeight;
  volatile int* abort = &bars.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;            // TMEM lanes 32 * quarter ..
  const int slice = (warp - 2) / 4;        // which half of the columns
  // rows without a token, while the first tile is summed
  if constexpr (kWhat == FfnProduct::kDown || kWhat == FfnProduct::kInput)
    ffn_clear_rows(p.r, static_cast<__nv_bfloat16*>(p.out), p.ldo, p.n, blockIdx.x * kEpiWarps + warp - 2, gridDim.x * kEpiWarps);
  int acc = 0;
  uint32_t acc_phase = 0;
  for (Walk<kWhat> w(p, table); w.more(); w.next()) {
    const Tile x = w.tile();
    const Part part = part_of<kWhat>(x, rank, quarter, slice);
    const int m = part.row + lane;         // row that this thread has
    if (kWeight && x.nk == 0) {            // an expert without a token
      const FfnJob& j = p.job[x.job];
      const float zero[32] = {};
      if (m < j.m)
        for (int c = x.col + slice * (TN / 2); c < min(x.col + (slice + 1) * (TN / 2), j.n); c += 32)
          put_some(static_cast<__nv_bfloat16*>(j.out) + x.expert * j.se + m * j.ld, c, j.n, j.vec, zero);
      continue;
    }
    const uint32_t tbase = bars.tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * TN);
    const bool valid = kWeight ? m < p.job[x.job].m : m < x.count;
    const bool some = __any_sync(0xffffffffu, valid);
    const int64_t row = (int64_t)x.offset + m;
    bool ok = true;
    if constexpr (kWhat == FfnProduct::kSlope) {
      if (p.saved.bits == 8) slope_tile<true, kAct>(p, part, tbase, row, valid, x.col + part.col, &bars.tfull[acc], acc_phase, abort, ok);
      else slope_tile<false, kAct>(p, part, tbase, row, valid, x.col + part.col, &bars.tfull[acc], acc_phase, abort, ok);
    } else {
      ok = ptx::mbar_wait_bounded(&bars.tfull[acc], acc_phase, abort, status_of(p), kStatusTimeoutEpilogue, kWaitLimitNs);
      if (ok) ptx::tc_fence_after();
      if (ok && some) {
        if constexpr (kWhat == FfnProduct::kGated) {
          uint32_t gs = 0, us = 0;   // scale bytes
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int64_t at = x.col + part.col + 32 * i;
            if (i >= part.chunks || at >= p.ldf) break;
            float g[32], u[32], h[32];
            load_acc(tbase + (uint32_t)(part.acc + 32 * i), g);
            load_acc(tbase + (uint32_t)(part.acc + 64 + 32 * i), u);
            if (!valid) continue;
#pragma unroll
            for (int j = 0; j < 32; ++j) h[j] = ffn_act<true, kAct>(g[j]).act * u[j];
            put32(static_cast<__nv_bfloat16*>(p.act) + row * p.ldf, at, h);
            if (p.saved.bits == 8) {
              gs |= keep32<true>(p.saved.gate, row, at, p.ldf, g) << 8 * i;
              us |= keep32<true>(p.saved.up, row, at, p.ldf, u) << 8 * i;
            } else if (p.saved.bits == 16) {
              gs |= keep32<false>(p.saved.gate, row, at, p.ldf, g) << 8 * i;
              us |= keep32<false>(p.saved.up, row, at, p.ldf, u) << 8 * i;
            }
          }
          if (valid && p.saved.bits && x.col + part.col < p.ldf) {
            const int64_t at = (row * p.ldf + x.col + part.col) / 32;
            if (part.chunks == 2) {   // a row has a multiple of four
              *reinterpret_cast<uint16_t*>(p.saved.gate_scales + at) = (uint16_t)gs;
              *reinterpret_cast<uint16_t*>(p.saved.up_scales + at) = (uint16_t)us;
            } else {
              p.saved.gate_scales[at] = (uint8_t)gs;
              p.saved.up_scales[at] = (uint8_t)us;
            }
          }
        } else {
          const int64_t n = kWeight ? p.job[x.job].n : p.n;
          const int vec = kWeight ? p.job[x.job].vec : p.vec;
          __nv_bfloat16* to = kWeight ? static_cast<__nv_bfloat16*>(p.job[x.job].out) + x.expert * p.job[x.job].se + m * p.job[x.job].ld
                                      : static_cast<__nv_bfloat16*>(p.out) + row * p.ldo;
#pragma unroll
          for (int i = 0; i < TN / 2 / 32; ++i) {
            const int64_t at = x.col + part.col + 32 * i;
            if (i >= part.chunks || at >= n) break;
            float f[32];
            load_acc(tbase + (uint32_t)(part.acc + 32 * i), f);
            if (!valid) continue;
            if (!kWeight && p.splits > 1) {
              float* sums = p.part + ((int64_t)x.split * p.r.rows + row) * p.ldp + at;
#pragma unroll
              for (int q = 0; q < 4; ++q) ptx::st_global_32(sums + 8 * q, reinterpret_cast<const uint32_t(&)[8]>(f[8 * q]));
            } else {
              put_some(to, at, n, vec, f);
            }
          }
        }
      }
    }
    if (!ok) break;
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa(ptx::smem_u32(&bars.tempty[acc]), 0));   // one per warp, at the even CTA
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
}

template <FfnProduct kWhat, bool kBMn, int kAct>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) k_ffn_tc(const __grid_constant__ FfnTcParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* stages = smem_raw + pad;
  Bars& bars = *reinterpret_cast<Bars*>(stages + kStages * kStageBytes);
  Table& table = *reinterpret_cast<Table*>(stages + kStages * kStageBytes + 256);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)ptx::cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&bars.full[s], 1);
      ptx::mbar_init(&bars.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&bars.tfull[a], 1);
      ptx::mbar_init(&bars.tempty[a], 2 * kEpiWarps);
    }
    ptx::mbar_init(&bars.drain, 1);
    bars.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(&bars.tmem, kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();   // both CTAs' barriers exist before any remote arrival
  ptx::tc_fence_after();
  grid_dependency_wait();
  if (threadIdx.x == 0) allow_dependent_launch();
  fill_table(p.r, table);

  if (warp == 0) {
    if (lane == 0) {
      if (rank == 0) run_producer<kWhat, kBMn, 0>(p, table, stages, bars);
      else run_producer<kWhat, kBMn, 1>(p, table, stages, bars);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) run_mma<kWhat, kBMn>(p, table, stages, bars);
    __syncwarp();
  } else {
    run_epilogue<kWhat, kAct>(p, table, rank, bars);
  }

  ptx::tc_fence_before();
  ptx::cluster_sync();   // no CTA leaves while its pair may still touch its memory
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(bars.tmem, kTmemCols);
  }
}

// Adds up the parts of rows whose depth several pairs have shared, in their order.  A warp for
// 128 columns of a row (64 x 2048, 9 parts: 4 us; a warp for a whole row took 47).
__global__ void __launch_bounds__(256) k_ffn_join(const __grid_constant__ FfnTcParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const int64_t blocks = (p.n + 127) / 128;
  for (int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); unit < p.r.rows * blocks; unit += (int64_t)gridDim.x * 8) {
    const int64_t row = unit / blocks, c = (unit - row * blocks) * 128 + 4 * lane;
    bool some = !p.r.offsets;   // the row holds a token
    for (int e0 = 0; e0 < p.r.experts && !some; e0 += 32) {
      const FfnExpert x = e0 + lane < p.r.experts ? ffn_expert(p.r, e0 + lane) : FfnExpert{0, 0};
      some = __any_sync(0xffffffffu, row >= x.offset && row < x.offset + x.count);
    }
    if (!some || c >= p.n) continue;   // ldp is a multiple of four
    const float* from = p.part + row * p.ldp + c;
    const int64_t apart = (int64_t)p.r.rows * p.ldp;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAhead = 8;
    for (int s0 = 0; s0 < p.splits; s0 += kAhead) {
      float4 v[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
        v[q] = s0 + q < p.splits ? *reinterpret_cast<const float4*>(from + (s0 + q) * apart) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        sum.x += v[q].x; sum.y += v[q].y; sum.z += v[q].z; sum.w += v[q].w;
      }
    }
    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + row * p.ldo + c;
    const float f[4] = {sum.x, sum.y, sum.z, sum.w};
    if (p.vec >= 16 && c + 4 <= p.n) {
      *reinterpret_cast<uint2*>(to) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (c + q < p.n) to[q] = __float2bfloat16_rn(f[q]);
    }
  }
}

// A tensor map of each expert's rows alone, for each matrix over the sorted rows.
// A warp for each.
__global__ void __launch_bounds__(128) k_ffn_maps(const __grid_constant__ FfnMapParams p) {
  __shared__ __align__(128) CUtensorMap map[4];
  grid_dependency_wait();
  allow_dependent_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = blockIdx.x * 4 + warp, i = blockIdx.y;
  if (e >= p.r.experts || !p.used[i]) return;
  const FfnExpert x = ffn_expert(p.r, e);
  if (x.count == 0) return;   // no tile of it loads anything
  reinterpret_cast<uint32_t*>(&map[warp])[lane] = reinterpret_cast<const uint32_t*>(&p.whole[i])[lane];
  __syncwarp();
  if (lane == 0) ptx::tensormap_replace(&map[warp], static_cast<const __nv_bfloat16*>(p.base[i]) + x.offset * p.ld[i], (uint32_t)x.count);
  __syncwarp();
  ptx::tensormap_publish(p.maps + i * p.r.experts + e, &map[warp]);
}

__global__ void k_ffn_take_status(int word, int reader) {
  grid_dependency_wait();
  g_ffn_taken[reader] = atomicExch(&g_ffn_status[word], 0u);   // a bit that is set meanwhile stays for the next
}

constexpr int kMaxDevices = 64;

// Pairs: as many as the device holds at once.
template <FfnProduct kWhat, bool kBMn, int kAct = kFfnSilu>
int launch_pair(const FfnTcParams& p, int sm_count, void* stream, bool pdl) {
  static std::atomic<int> fit[kMaxDevices];   // pairs that fit at once, per device; 0: not set up
  auto* kernel = &k_ffn_tc<kWhat, kBMn, kAct>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return (int)e;
  int pairs = dev < kMaxDevices ? fit[dev].load(std::memory_order_acquire) : 0;
  if (pairs == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return (int)e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sm_count);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    e = cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg);
    if (e != cudaSuccess) return (int)e;
    if (pairs > sm_count / 2) pairs = sm_count / 2;
    if (pairs <= 0) return (int)cudaErrorLaunchOutOfResources;
    if (dev < kMaxDevices) fit[dev].store(pairs, std::memory_order_release);
  }
  // no more than there can be tiles
  const int64_t tiles = kWhat == FfnProduct::kWeight
                            ? (int64_t)p.r.experts * p.tiles_per_expert
                            : ((int64_t)p.r.rows / TM + (p.r.rows < p.r.experts ? p.r.rows : p.r.experts)) * p.nt * p.splits;
  if (tiles == 0) return 0;
  if (tiles < pairs) pairs = (int)tiles;
  return launch_kernel(kernel, dim3((unsigned)(2 * pairs)), dim3(kThreads), kSmemBytes, stream, pdl, p);
}

template <FfnProduct kWhat>
int launch_major(bool b_mn, const FfnTcParams& p, int sm_count, void* stream, bool pdl) {
  return b_mn ? launch_pair<kWhat, true>(p, sm_count, stream, pdl) : launch_pair<kWhat, false>(p, sm_count, stream, pdl);
}

// The same for the products with the activation in their epilogue.
template <FfnProduct kWhat>
int launch_act(bool b_mn, const FfnTcParams& p, int sm_count, void* stream, bool pdl) {
  if (p.activation == kFfnSilu) return launch_major<kWhat>(b_mn, p, sm_count, stream, pdl);
  return b_mn ? launch_pair<kWhat, true, kFfnGelu>(p, sm_count, stream, pdl) : launch_pair<kWhat, false, kFfnGelu>(p, sm_count, stream, pdl);
}

}  // namespace

int launch_ffn_tc(FfnProduct what, bool b_mn, const FfnTcParams& p, int sm_count, void* stream, bool pdl) {
  switch (what) {
    case FfnProduct::kGated: return launch_act<FfnProduct::kGated>(b_mn, p, sm_count, stream, pdl);
    case FfnProduct::kDown: return launch_major<FfnProduct::kDown>(b_mn, p, sm_count, stream, pdl);
    case FfnProduct::kSlope: return launch_act<FfnProduct::kSlope>(b_mn, p, sm_count, stream, pdl);
    case FfnProduct::kInput: return launch_major<FfnProduct::kInput>(b_mn, p, sm_count, stream, pdl);
    default: return launch_pair<FfnProduct::kWeight, true>(p, sm_count, stream, pdl);
  }
}

int launch_ffn_join(const FfnTcParams& p, void* stream, bool pdl) {
  const int64_t ctas = ((int64_t)p.r.rows * ((p.n + 127) / 128) + 7) / 8;
  return launch_kernel(k_ffn_join, dim3((unsigned)(ctas < 152 * 8 ? ctas : 152 * 8)), dim3(256), 0, stream, pdl, p);
}

int launch_ffn_maps(const FfnMapParams& p, void* stream, bool pdl) {
  return launch_kernel(k_ffn_maps, dim3((unsigned)((p.r.experts + 3) / 4), kFfnMaps), dim3(128), 0, stream, pdl, p);
}

int read_ffn_status(int word, int reader, uint32_t* bits, void* stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = (cudaError_t)launch_kernel(k_ffn_take_status, dim3(1), dim3(1), 0, stream, false, word, reader);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(bits, g_ffn_taken, sizeof(*bits), sizeof(*bits) * (size_t)reader, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return (int)e;
}

}  // namespace muon
