// Parameter blocks of the gated feed-forward kernels.
#pragma once

#include <cstdint>

namespace muon {

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

// What is kept of the forward pass: pre-activations in the inputs' type, or
// codes and scale bytes.
struct FfnSaved {
  void* gate;
  void* up;
  uint8_t* gate_scales;     // null: not in 8 bits
  uint8_t* up_scales;
};

struct FfnSimtParams {
  FfnRows r;
  FfnStack a[2], b[2];      // product of a's rows with b's rows
  int64_t n, k;             // columns of the result, length of the sums (weights: rows of the result in m)
  int64_t m;
  FfnStack out;
  FfnSaved saved;           // null pointers: nothing is kept
  void* act;                // h, written by kGated and (8 bits) kSlope
  void* dgate;              // written by kSlope
  void* dup;
  int64_t ldf, ffn;
  int32_t activation;
};
int launch_ffn_simt(FfnProduct what, const FfnSimtParams& p, bool bf16, void* stream, bool pdl);

struct FfnClearParams {
  FfnRows r;
  void* out;
  int64_t ld, cols;
};
int launch_ffn_clear(const FfnClearParams& p, bool bf16, void* stream, bool pdl);

}  // namespace muon
