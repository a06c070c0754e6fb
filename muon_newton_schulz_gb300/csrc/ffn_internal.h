// Parameter blocks of the gated feed-forward kernels.
#pragma once

#include <cstdint>
#include <cuda.h>

struct muon_handle_s;

namespace muon {

// Of a handle (defined in muon_api.cpp).
int handle_sm_count(::muon_handle_s* h);
bool handle_withholds_loads(::muon_handle_s* h);   // test hook of the failure path
int handle_ffn_status(::muon_handle_s* h);         // the word that its kernels' waits report to
// A bf16 tensor map with 128-byte swizzle: d0 x d1 elements, d1 lines `ld_bytes`
// apart, and d2 such matrices.  On failure the handle's error says why.
bool encode_operand_map(::muon_handle_s* h, CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                        uint64_t ld_bytes, uint64_t mat_bytes, uint32_t box0, uint32_t box1);

// Status words of a device: kFfnGroups that handles may share, then one for each handle
// in the order in which they are made (beyond 4080 of them two have one).
constexpr int kFfnGroups = 16, kFfnStatusWords = 4096;

constexpr int kFfnSilu = 0, kFfnGelu = 1;

// What the products of one pass read and write.  Rows are the sorted tokens;
// buffers over the ffn width have rows of ldf elements.
enum class FfnProduct : int {
  kGated,   // h = act(x gate^T) * (x up^T)
  kDown,    // y = h down^T
  kSlope,   // dh = dy down; d(gate), d(up) of it
  kInput,   // dx = dg gate + du up
  kWeight,  // dW = p^T q over an expert's rows
};

// A stack of matrices: element (expert, i, j) at p + expert * se + i * si + j * sj.
struct FfnStack {
  void* p;
  int64_t se, si, sj;
};

struct FfnRows {
  const int32_t* offsets;   // null: one expert with all rows
  const int32_t* counts;
  int32_t rows, experts;
};

// What is kept of the forward pass: pre-activations in fp32, or codes of 16 or 8
// bits and scale bytes.
struct FfnSaved {
  void* gate;
  void* up;
  uint8_t* gate_scales;     // null: fp32
  uint8_t* up_scales;
  int32_t bits;             // 0: nothing is kept
};

struct FfnSimtParams {
  FfnRows r;
  FfnStack a[3], b[3];      // product of a's rows with b's rows (kWeight: of each of the jobs)
  int64_t n, k;             // columns of the result, length of the sums
  FfnStack out[3];
  int64_t wm[3], wn[3];     // kWeight: rows and columns of each result
  int32_t jobs;
  bool beside;              // kWeight: the input's gradient is asked for too, in the same grid or in the one before
  FfnSaved saved;           // null pointers: nothing is kept
  void* act;                // h, written by kGated and (8 bits) kSlope
  void* dgate;              // written by kSlope
  void* dup;
  int64_t ldf, ffn;
  int32_t activation;
  int32_t row_tiles, splits, begin[3];   // set by the launch
};
int launch_ffn_simt(FfnProduct what, const FfnSimtParams& p, void* stream, bool pdl);

struct FfnGradsParams {
  FfnSimtParams input, weights;
  int32_t cluster;                           // CTAs of one
  int32_t row_ctas, columns, weight_ctas;    // the input's CTAs along the rows and the columns; the weights' of an expert
  uint32_t first_weight;                     // the first CTA of the weights'
};
// kInput and kWeight in one grid, where both have tiles of one size.
bool ffn_grads_in_one(const FfnSimtParams& input, const FfnSimtParams& weights);
int launch_ffn_grads(const FfnSimtParams& input, const FfnSimtParams& weights, void* stream, bool pdl);

// ---- tensor-core products (bf16)
constexpr int kFfnMaps = 5;          // matrices over the sorted rows that a backward pass reads: x, dy, h, dg, du

struct FfnMapParams {
  CUtensorMap whole[kFfnMaps];
  const void* base[kFfnMaps];
  int64_t ld[kFfnMaps];              // elements
  int32_t used[kFfnMaps];
  FfnRows r;
  CUtensorMap* maps;                 // [kFfnMaps][experts], each of its expert's rows alone
};
int launch_ffn_maps(const FfnMapParams& p, void* stream, bool pdl);

// One weight's gradient: rows of p^T q.
struct FfnJob {
  void* out;
  int64_t se, ld;
  int32_t p, q;                      // numbers of the maps
  int32_t m, n;                      // rows and columns of the result
  int32_t mt, nt;                    // tiles along them
  int32_t begin;                     // first tile of this job among an expert's
  int32_t vec;
};

struct FfnTcParams {
  CUtensorMap a[2], b[2];
  CUtensorMap a_few[2];              // a, 64 rows at a time
  FfnRows r;
  int64_t n;                         // columns of the result
  int32_t nt, nk;                    // column tiles; steps of 64 of the sums (of a segment)
  void* out;
  int64_t ldo;
  int32_t vec;                       // bytes that a store to `out` may have: 32, 16 or 2
  int32_t splits;                    // pairs that share the depth of a tile; more than one leave their sums in part
  float* part;                       // [splits][rows][ldp]
  int64_t ldp;
  int32_t activation;
  FfnSaved saved;
  void* act;
  void* dgate;
  void* dup;
  int64_t ldf;
  // weights' gradients
  const CUtensorMap* maps;
  FfnJob job[3];
  int32_t jobs, tiles_per_expert;
  int32_t withhold_loads;            // test hook: the producer issues no loads, so the waits run out
  int32_t status;                    // the word that tells of waits that ran out
};
// b_mn: the right operand is contiguous along the result's columns
int launch_ffn_tc(FfnProduct what, bool b_mn, const FfnTcParams& p, int sm_count, void* stream, bool pdl);
// out = the sum of the splits' parts, for rows that hold a token.
int launch_ffn_join(const FfnTcParams& p, void* stream, bool pdl);
// The bits of a status word of the current device, which is cleared; `reader` is the handle's
// own word.  A cudaError_t as int.
int read_ffn_status(int word, int reader, uint32_t* bits, void* stream);

// ---- rows of bf16 of any length, to or from rows that begin 16 bytes apart
constexpr int kFfnLines = 5;

struct FfnLines {
  const void* from;
  void* to;
  int64_t from_se, from_ld, to_se, to_ld;
  int64_t begin;                     // first of this job's lines in the launch
  int64_t lines;                     // of an expert
  int32_t length, padded;            // elements that are copied, and up to where zeros follow
  int32_t used_only;                 // experts without a token are left out
};
struct FfnLinesParams {
  FfnRows r;
  FfnLines job[kFfnLines];
  int32_t n;
  int64_t lines;
};
int launch_ffn_lines(const FfnLinesParams& p, void* stream, bool pdl);

// ---- a few rows (bf16)
// Most rows of a call that goes this way.  (us, here and on the pairs of CTAs: one layer of
// 2048 x 8192, 8 rows 23 and 28, 16 rows 30 and 28, 24 rows 47 and 29, 32 rows 49 and 30; 16
// experts of that size, top 2, 16 rows 157 and 154, 20 rows 197 and 221, 32 rows 229 and 236; 512 x
// 2048, one layer of 16 or 32 rows 12 and 19, 8 experts, 16 or 32 rows 17 and 21.)
constexpr int kFfnFewRows = 16;

struct FfnFewParams {
  FfnRows r;
  const void* x;                     // rows of the sorted tokens
  int64_t ldx;
  FfnStack w[2];                     // contiguous along the depth
  int64_t n, k;                      // columns of the result, length of the sums (a multiple of 8)
  int64_t padded;                    // columns that are written, zero behind the result's
  void* out;
  int64_t ldo;
  int32_t rest;                      // from an element of h to what its rounding to bf16 left
  int32_t activation;
};
int launch_ffn_few(bool gated, const FfnFewParams& p, void* stream, bool pdl);

}  // namespace muon
