// Parameter blocks of the training-step kernels around the Muon step (AdamW,
// gradient clipping, tokens by expert).  As for the step itself, everything a
// launch needs travels in its __grid_constant__ parameter block.
#pragma once

#include <cstdint>

namespace muon {

constexpr int kThreads256 = 256;
constexpr int kFewTensors = 64;     // tensors of a launch with a small parameter block

// ---- AdamW
constexpr int kAdamTensors = 400;   // tensors per launch: the block stays below the 32764-byte limit
constexpr int kAdamChunk = 4096;    // elements per CTA, 32-bit states
constexpr int kStateBlock = 256;    // elements that share the scales of an 8-bit state

constexpr uint8_t kVecP = 1, kVecG = 2, kVecV = 4;

struct AdamTensor {
  void* P;
  const void* G;
  void* M;
  void* V;
  uint8_t* scales;
  int64_t n;
  uint32_t chunk_begin;   // first chunk of this tensor in the launch
  uint8_t p_bf16, g_bf16;
  uint8_t vec;            // 32-bit states: kVec* of the buffers aligned like M; 8-bit states: all allow vectors
  uint8_t shift;          // 32-bit states: elements between M's preceding vector boundary and its element 0
  float decay;            // 1 - lr * weight_decay
  float step_size;        // lr / (1 - beta1^t)
  float inv_sqrt_bc2;     // 1 / sqrt(1 - beta2^t)
  uint32_t key_lo, key_hi;
};

struct AdamHead {
  int32_t n;
  uint32_t chunks;
  int32_t chunk;          // elements per CTA
  float beta1, one_minus_beta1, beta2, one_minus_beta2, eps;
  float minus_zero;       // -0
};
// A launch of at most kFewTensors tensors gets a small block: filling and
// copying the large one takes a few us of the host's time and most of its
// first-level cache (clipping 49 vectors: 24 us a call with the large one).
template <int N> struct AdamBlock : AdamHead {
  using Head = AdamHead;
  static constexpr int kTensors = N;
  AdamTensor t[N];
};
using AdamParams = AdamBlock<kAdamTensors>;
static_assert(sizeof(AdamParams) <= 32764, "kernel parameter limit");

int launch_adamw32(const AdamParams& p, void* stream, bool pdl);
int launch_adamw8(const AdamParams& p, void* stream, bool pdl);

// ---- gradient clipping
constexpr int kClipTensors = 400;
constexpr int kClipChunk = 16384;     // elements per chunk
constexpr int kClipPartials = 2048;   // partial sums the workspace holds

struct ClipTensor {
  const void* G;
  void* out;
  int64_t ldg, ldo;
  int64_t cols;           // a flat tensor is one row
  int32_t rows_per_chunk; // rows of a chunk (1 when cols >= kClipChunk)
  int32_t seg;            // columns of a chunk
  int64_t rows;
  int64_t segs_per_row;
  uint32_t chunk_begin;
  uint8_t g_bf16, o_bf16;
  uint8_t vec, vec_out;   // groups of four of G, and of out at the same places, lie on vector boundaries
  uint8_t shift;          // flat tensors: elements between G's preceding vector boundary and its element 0
};

struct ClipHead {
  int32_t n;
  uint32_t chunks;
  int32_t partial_begin;  // first partial sum of this launch
  int32_t partials;       // partial sums of the whole call
  int32_t write_norm;     // this launch's first CTA writes *norm
  float max_norm;
  double* partial;
  float* norm;
};
template <int N> struct ClipBlock : ClipHead {
  using Head = ClipHead;
  static constexpr int kTensors = N;
  ClipTensor t[N];
};
using ClipParams = ClipBlock<kClipTensors>;
static_assert(sizeof(ClipParams) <= 32764, "kernel parameter limit");

int launch_clip_sumsq(const ClipParams& p, int grid, void* stream, bool pdl);
int launch_clip_scale(const ClipParams& p, int grid, void* stream, bool pdl);

// ---- tokens by expert
constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopk = 64;
constexpr int kSortThreads = 1024;
constexpr int kSortFew = 256;        // slots that are sorted a thread for each
constexpr int kSortSingle = 2048;    // slots that one CTA sorts by itself
constexpr int kSortGrid = 152;        // most CTAs of a larger sort

struct SortParams {
  const void* ids;
  int32_t ids64;
  int32_t slots;          // tokens * topk
  int32_t per_cta;        // slots of a CTA
  int32_t experts, capacity, align;
  int32_t ctas;
  int32_t* row;
  int32_t* offsets;
  int32_t* counts;
  int32_t* hist;          // [experts][ctas], null for a single CTA
};
int launch_moe_sort_count(const SortParams& p, void* stream, bool pdl);
int launch_moe_sort_place(const SortParams& p, void* stream, bool pdl);

constexpr int kRowUnits = 4;   // units that a thread of dispatch and combine moves at once where they are not 16 bytes

struct RowsParams {
  const void* x;          // dispatch: tokens; combine: sorted rows; backward: dout
  const void* y;          // backward: sorted rows
  void* out;              // dispatch and backward: sorted rows; combine: tokens
  const void* w;          // combine: weights or null; backward: weights
  void* dw;               // backward
  const int32_t* row;
  const int32_t* offsets;
  const int32_t* counts;
  int64_t ldx, ldy, ldo;
  int64_t hidden;
  int64_t tokens;
  int32_t topk, experts;
  int32_t rows;           // sorted rows
  int32_t w_bf16;
  int32_t token_ctas;     // CTAs that handle tokens; the others clear rows without a token
  int32_t tx;             // threads of a CTA along a row
  int32_t tokens_per_cta;
  int32_t splits;         // combine: CTAs that share a token's columns
};
// bytes: what a thread moves at once, 16, 4 or (bf16) 2
int launch_moe_dispatch(const RowsParams& p, bool bf16, int bytes, int grid, void* stream, bool pdl);
int launch_moe_combine(const RowsParams& p, bool bf16, int bytes, int grid, void* stream, bool pdl);
int launch_moe_backward(const RowsParams& p, bool bf16, int bytes, int grid, void* stream, bool pdl);

}  // namespace muon
