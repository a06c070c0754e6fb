// Parameter blocks of the kernels of a model's layers: embedding rows,
// activations in 8 bits.
#pragma once

#include <cstdint>

#include "train_internal.h"

namespace muon {

// ---- embedding
constexpr int kIdFew = 512;          // ids that are sorted by counting for each the smaller ones
constexpr int kIdSingle = 2048;      // ids that one CTA sorts by itself
constexpr int kIdPerCta = 1024;      // ids of a CTA of a larger sort, or a multiple of them
constexpr int kIdGrid = 152;         // most CTAs of a larger sort
constexpr int kIdDigitBits = 10;     // most bits of an id sorted in one pass
constexpr int kEmbedChunk = 64;      // most sorted tokens that a group of threads sums
constexpr int kEmbedJoin = 8;        // chunks whose sums a CTA joins

struct EmbedParams {
  const void* ids;
  const void* table;
  void* out;
  int64_t ldt, ldo;
  int64_t tokens, vocab, hidden;
  int32_t ids64;
  int32_t tx;             // threads of a CTA along a row
  int32_t tokens_per_cta;
  int32_t splits;         // CTAs that share a token's columns
  float scale;
};
int launch_embed(const EmbedParams& p, bool bf16, int bytes, int grid, void* stream, bool pdl);

// Rows of dtable that the CTAs of a launch behind the first `first_cta` set to zero.
struct ZeroRows {
  void* p;
  int64_t begin, end;     // rows
  int64_t row_bytes, pitch;
  int32_t first_cta;
};

struct IdSortParams {
  const void* ids;        // the first pass reads these
  const int32_t* key_in;
  const int32_t* at_in;
  int32_t* key_out;       // sorted ids; an id outside the table becomes `vocab`
  int32_t* at_out;        // the tokens that have them
  int32_t* hist;          // [ctas][bins], null for a single CTA
  int32_t* hist_next;     // the next pass's, which this one counts; for the count: cleared
  int64_t clear;          // the count: elements to clear
  int32_t ids64, vocab;
  int32_t n, per_cta, ctas;
  int32_t shift, bins;    // the digit of this pass
  int32_t shift_next;
  ZeroRows zero;
};
int launch_id_sort_few(const IdSortParams& p, void* stream, bool pdl);
int launch_id_sort_count(const IdSortParams& p, void* stream, bool pdl);
int launch_id_sort_place(const IdSortParams& p, void* stream, bool pdl);

struct EmbedGradParams {
  const void* dout;
  void* dtable;
  float* part;            // [chunks][2][ldp]: sums of ids that go on in another chunk
  const int32_t* key;
  const int32_t* at;
  int64_t lddo, lddt, ldp;
  int64_t vocab, hidden;
  int32_t n, chunk, chunks;
  int32_t tx, splits;
  float scale;
};
int launch_embed_grad(const EmbedGradParams& p, bool bf16, int bytes, int grid, void* stream, bool pdl);
int launch_embed_join(const EmbedGradParams& p, bool bf16, void* stream, bool pdl);

// ---- activations in 8 bits
constexpr int kSaved8Block = 32;     // elements of a row that share a scale

struct Saved8Params {
  void* x;                // read by pack, written by unpack
  uint8_t* codes;
  uint8_t* scales;
  int64_t ldx, rows, cols;
  bool special;           // infinities have codes of their own, and zero and finite values none but theirs
};
int launch_pack8(const Saved8Params& p, bool bf16, void* stream, bool pdl);
int launch_unpack8(const Saved8Params& p, bool bf16, void* stream, bool pdl);

}  // namespace muon
