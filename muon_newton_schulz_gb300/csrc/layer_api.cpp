// C ABI of the operators of a model's layers (embedding rows and their
// gradient, activations in 8 bits): validation and launches.  See
// include/muon.h for the contract.
#include "muon.h"

#include <nvtx3/nvToolsExt.h>

#include <cmath>

#include "api_common.h"
#include "device_guard.h"
#include "layer_internal.h"

using namespace muon;

namespace {


muon_status invalid(muon_handle h, const std::string& why) { return fail(h, MUON_ERR_INVALID_ARG, why); }

muon_status host_only(muon_handle h) {
  return fail(h, MUON_ERR_UNSUPPORTED, "host-only handle: create it with a device to run");
}

muon_status check_workspace(muon_handle h, const void* ws, size_t ws_bytes, size_t need, std::vector<Span>& spans) {
  if (need == 0) return MUON_OK;
  if (!ws) return fail(h, MUON_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(h, MUON_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < need) return fail(h, MUON_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) + " bytes");
  spans.push_back(span(ws, (int64_t)need, -1, true, "workspace"));
  return MUON_OK;
}

// ---------------------------------------------------------------- embedding

muon_status check_ids(const void* ids, int ids_bits, int64_t tokens, int64_t vocab, std::vector<Span>& spans, std::string& why) {
  if (ids_bits != 32 && ids_bits != 64) { why = "ids_bits must be 32 or 64"; return MUON_ERR_INVALID_ARG; }
  if (tokens < 0 || tokens > kInt32Max) { why = "tokens must be in [0, 2^31)"; return MUON_ERR_INVALID_ARG; }
  if (vocab < 0 || vocab >= kInt32Max) { why = "vocab must be in [0, 2^31 - 1)"; return MUON_ERR_INVALID_ARG; }
  if (tokens > 0 && !ids) { why = "ids must be non-NULL"; return MUON_ERR_INVALID_ARG; }
  if (!aligned(ids, ids_bits / 8)) { why = "ids must be aligned to their size"; return MUON_ERR_INVALID_ARG; }
  spans.push_back(span(ids, tokens * (ids_bits / 8), -1, false, "ids"));
  return MUON_OK;
}

int threads_along(int64_t hidden, int64_t per) {
  int tx = 32;
  while (tx < kThreads256 && tx * per < hidden) tx *= 2;
  return tx;
}

// How the gradient of n tokens is cut up, and where its workspace holds what.
struct GradPlan {
  int32_t per_cta, ctas, passes, digit_bits;   // sort
  int32_t chunk, chunks;
  int64_t ldp;
  size_t key[2], at[2], hist, part, bytes;     // offsets into the workspace
};

GradPlan grad_plan(int64_t n, int64_t vocab, int64_t hidden) {
  GradPlan g{};
  size_t used = 0;
  auto take = [&](size_t bytes) {
    const size_t at = used;
    used += (bytes + 255) / 256 * 256;
    return at;
  };
  int bits = 1;
  while ((vocab >> bits) != 0) ++bits;   // ids and the mark `vocab` itself
  if (n <= kIdFew) {
    g.passes = 0;
  } else {
    g.passes = (int32_t)cdiv(bits, kIdDigitBits);
    g.digit_bits = (int32_t)cdiv(bits, g.passes);
    g.per_cta = n <= kIdSingle ? (int32_t)n : (int32_t)std::min<int64_t>(kInt32Max, cdiv(cdiv(n, kIdGrid), kIdPerCta) * kIdPerCta);
    g.ctas = (int32_t)cdiv(n, g.per_cta);
  }
  for (int i = 0; i < 2; ++i) {
    if (i == 1 && g.passes < 2) break;
    g.key[i] = take((size_t)n * 4);
    g.at[i] = take((size_t)n * 4);
  }
  if (g.ctas > 1) g.hist = take((size_t)g.passes * (size_t)g.ctas << (g.digit_bits + 2));   // one for each pass
  // tokens of a chunk: whole rounds of four CTAs per SM (65536 tokens: two of 54 each,
  // 117 us; with 64, one and two thirds, 122)
  g.chunk = (int32_t)std::clamp<int64_t>(cdiv(n, kSms * 4 * std::max<int64_t>(1, cdiv(n, kSms * 4 * kEmbedChunk))), 8, kEmbedChunk);
  g.chunks = (int32_t)cdiv(n, g.chunk);
  g.ldp = cdiv(hidden, 256) * 256;
  if (g.chunks > 1) g.part = take((size_t)g.chunks * 2 * (size_t)g.ldp * 4);
  g.bytes = used;
  return g;
}

muon_status run_grad(muon_handle h, const GradPlan& g, const void* ids, int ids_bits, int64_t n, const void* dout,
                     int64_t lddout, int64_t vocab, int64_t hidden, int dtype, int bytes, float scale, void* dtable,
                     int64_t lddtable, uint8_t* ws, void* stream) {
  EmbedGradParams p{};
  const int64_t per = bytes / element_size(dtype);
  p.tx = threads_along(hidden, per);
  p.splits = (int32_t)std::min<int64_t>(cdiv(hidden, p.tx * per), 65535);
  const int64_t grid = cdiv(g.chunks, kThreads256 / p.tx) * p.splits;
  const int64_t join = g.chunks > 1 ? cdiv(hidden, 256) * cdiv(g.chunks, kEmbedJoin) : 0;
  if (std::max(grid, join) > kInt32Max) return invalid(h, "tokens: too many for one launch");
  bool pdl = first_pdl(stream);
  int launches = 0, e = 0, sorted = 0;
  auto ints = [&](size_t at) { return reinterpret_cast<int32_t*>(ws + at); };
  const int64_t es = element_size(dtype);
  // which rows each launch of the sort clears: a count takes about a third of a place
  int64_t cleared = 0, weight = 0;
  const int64_t weights = g.passes == 0 ? 1 : 3 * g.passes + (g.ctas > 1 ? 1 : 0);
  auto zero = [&](int ctas, int share, bool last) {
    weight += share;
    const int64_t upto = last ? vocab : vocab * weight / weights;
    const ZeroRows z{dtable, cleared, upto, hidden * es, (vocab > 1 ? lddtable : hidden) * es, ctas};
    cleared = upto;
    return z;
  };
  {
    IdSortParams s{};
    s.ids = ids;
    s.ids64 = ids_bits == 64;
    s.vocab = (int32_t)vocab;
    s.n = (int32_t)n;
    s.per_cta = g.per_cta;
    s.ctas = g.ctas;
    const int64_t counts = (int64_t)g.ctas << g.digit_bits;   // of one pass
    nvtxRangePushA("muon.embed_sort");
    if (g.passes == 0) {
      s.key_out = ints(g.key[0]);
      s.at_out = ints(g.at[0]);
      s.zero = zero(n > 0 ? 1 : 0, 1, true);
      e = launch_id_sort_few(s, stream, pdl);
      launches = 1;
      pdl = kUsePdl;
    }
    for (int i = 0; i < g.passes && !e; ++i) {
      s.shift = i * g.digit_bits;
      s.bins = 1 << g.digit_bits;
      s.key_in = i > 0 ? ints(g.key[sorted]) : nullptr;
      s.at_in = i > 0 ? ints(g.at[sorted]) : nullptr;
      if (i > 0) sorted ^= 1;
      s.key_out = ints(g.key[sorted]);
      s.at_out = ints(g.at[sorted]);
      s.hist = g.ctas > 1 ? ints(g.hist) + i * counts : nullptr;
      s.hist_next = g.ctas > 1 && i + 1 < g.passes ? s.hist + counts : nullptr;
      s.shift_next = s.shift + g.digit_bits;
      if (g.ctas > 1 && i == 0) {
        s.clear = (g.passes - 1) * counts;
        s.zero = zero(g.ctas, 1, false);
        e = launch_id_sort_count(s, stream, pdl);
        pdl = kUsePdl;
        ++launches;
      }
      s.zero = zero(g.ctas, 3, i + 1 == g.passes);
      if (!e) e = launch_id_sort_place(s, stream, pdl);
      pdl = kUsePdl;
      ++launches;
    }
    nvtxRangePop();
    if (e) return cuda_fail(h, "muon_embed_backward", e);
  }
  p.dout = dout;
  p.dtable = dtable;
  p.part = g.chunks > 1 ? reinterpret_cast<float*>(ws + g.part) : nullptr;
  p.key = ints(g.key[sorted]);
  p.at = ints(g.at[sorted]);
  p.lddo = lddout;
  p.lddt = lddtable;
  p.ldp = g.ldp;
  p.vocab = vocab;
  p.hidden = hidden;
  p.n = (int32_t)n;
  p.chunk = g.chunk;
  p.chunks = g.chunks;
  p.scale = scale;
  if (n == 0) {
    count_launches(h, launches);
    return MUON_OK;
  }
  nvtxRangePushA("muon.embed_grad");
  e = launch_embed_grad(p, dtype == MUON_BF16, bytes, (int)grid, stream, pdl);
  if (!e && g.chunks > 1) e = launch_embed_join(p, dtype == MUON_BF16, stream, kUsePdl);
  nvtxRangePop();
  if (e) return cuda_fail(h, "muon_embed_backward", e);
  count_launches(h, launches + (g.chunks > 1 ? 2 : 1));
  return MUON_OK;
}

// ---------------------------------------------------------------- activations in 8 bits

muon_status check_saved8(const void* x, int64_t ldx, int64_t rows, int64_t cols, int dtype, const void* codes, const void* scales,
                         bool pack, std::string& why) {
  if (rows < 0 || cols < 0 || (cols > 0 && rows > kMaxElements / cols)) { why = "rows and cols must be >= 0 and rows * cols at most 2^40"; return MUON_ERR_INVALID_ARG; }
  const int64_t n = rows * cols;
  if (!known_dtype(dtype)) { why = "dtype must be MUON_F32 or MUON_BF16"; return MUON_ERR_INVALID_ARG; }
  if (n == 0) return MUON_OK;
  if (!x || !codes || !scales) { why = "x, codes and scales must be non-NULL"; return MUON_ERR_INVALID_ARG; }
  if (!aligned(x, element_size(dtype))) { why = "x must be aligned to its element size"; return MUON_ERR_INVALID_ARG; }
  if (ldx < cols || ldx > kMaxElements / rows) { why = "ldx must be >= cols, and rows * ldx at most 2^40"; return MUON_ERR_INVALID_ARG; }
  const std::vector<Span> spans = {matrix_span(x, rows, cols, ldx, element_size(dtype), -1, !pack, "x"),
                                   span(codes, n, -1, pack, "codes"),
                                   span(scales, rows * cdiv(cols, kSaved8Block), -1, pack, "scales")};
  return find_overlap(spans, why) ? MUON_ERR_INVALID_ARG : MUON_OK;
}

muon_status run_saved8(muon_handle h, const void* x, int64_t ldx, int64_t rows, int64_t cols, int dtype, bool special,
                       const void* codes, const void* scales, bool pack, void* stream) {
  const Saved8Params p{const_cast<void*>(x), static_cast<uint8_t*>(const_cast<void*>(codes)),
                       static_cast<uint8_t*>(const_cast<void*>(scales)), ldx, rows, cols, special};
  nvtxRangePushA(pack ? "muon.pack8" : "muon.unpack8");
  const int e = (pack ? launch_pack8 : launch_unpack8)(p, dtype == MUON_BF16, stream, first_pdl(stream));
  nvtxRangePop();
  if (e) return cuda_fail(h, pack ? "muon_pack8" : "muon_unpack8", e);
  count_launches(h, 1);
  return MUON_OK;
}

muon_status saved8(muon_handle h, const void* x, int64_t ldx, int64_t rows, int64_t cols, int dtype, const void* codes,
                   const void* scales, bool pack, void* stream) {
  return guarded(h, [&]() -> muon_status {
    std::string why;
    const bool special = (dtype & MUON_SAVED8_SPECIAL) != 0;
    const int kind = dtype & ~MUON_SAVED8_SPECIAL;
    const muon_status st = check_saved8(x, ldx, rows, cols, kind, codes, scales, pack, why);
    if (st != MUON_OK) return fail(h, st, why);
    if (rows == 0 || cols == 0) return MUON_OK;
    if (handle_device(h) < 0) return host_only(h);
    DeviceGuard guard(handle_device(h));
    return run_saved8(h, x, ldx, rows, cols, kind, special, codes, scales, pack, stream);
  });
}

}  // namespace

extern "C" {

muon_status muon_embed(muon_handle h, const void* ids, int ids_bits, int64_t tokens, const void* table, int64_t ldtable,
                       int64_t vocab, int64_t hidden, int dtype, double scale, void* out, int64_t ldout, void* stream) {
  return guarded(h, [&]() -> muon_status {
    std::string why;
    std::vector<Span> spans;
    muon_status st = check_ids(ids, ids_bits, tokens, vocab, spans, why);
    if (st != MUON_OK) return fail(h, st, why);
    int bytes = 0;
    const Mat mats[2] = {{table, vocab, ldtable, false, "table"}, {out, tokens, ldout, true, "out"}};
    st = check_rows(hidden, dtype, mats, 2, spans, bytes, why);
    if (st != MUON_OK) return fail(h, st, why);
    if (tokens == 0 || hidden == 0) return MUON_OK;
    if (handle_device(h) < 0) return host_only(h);
    DeviceGuard guard(handle_device(h));
    EmbedParams p{};
    p.ids = ids;
    p.ids64 = ids_bits == 64;
    p.table = table;
    p.ldt = ldtable;
    p.out = out;
    p.ldo = ldout;
    p.tokens = tokens;
    p.vocab = vocab;
    p.hidden = hidden;
    p.scale = (float)scale;
    const int64_t per = (bytes == 16 ? 1 : kRowUnits) * bytes / element_size(dtype);   // elements that a thread takes at once
    p.tx = threads_along(hidden, per);
    // four tokens of every row of threads where they fill the SMs, else one
    const int64_t rows_of_threads = kThreads256 / p.tx;
    p.tokens_per_cta = (int32_t)(tokens >= rows_of_threads * 4 * kSms * 2 ? rows_of_threads * 4 : rows_of_threads);
    const int64_t token_ctas = cdiv(tokens, p.tokens_per_cta);
    p.splits = (int32_t)std::clamp<int64_t>(kSms / token_ctas, 1, cdiv(hidden, p.tx * per));
    nvtxRangePushA("muon.embed");
    const int e = launch_embed(p, dtype == MUON_BF16, bytes, (int)(token_ctas * p.splits), stream, first_pdl(stream));
    nvtxRangePop();
    if (e) return cuda_fail(h, "muon_embed", e);
    count_launches(h, 1);
    return MUON_OK;
  });
}

muon_status muon_embed_backward_workspace_size(int64_t tokens, int64_t vocab, int64_t hidden, size_t* bytes) {
  if (!bytes || tokens < 0 || tokens > kInt32Max || vocab < 0 || vocab >= kInt32Max || hidden < 0 || hidden > kMaxElements)
    return MUON_ERR_INVALID_ARG;
  const GradPlan g = grad_plan(tokens, vocab, hidden);
  if ((int64_t)g.bytes < 0 || (hidden > 0 && (int64_t)g.chunks * 8 > kMaxElements / hidden)) return MUON_ERR_INVALID_ARG;
  *bytes = g.bytes;
  return MUON_OK;
}

muon_status muon_embed_backward(muon_handle h, const void* ids, int ids_bits, int64_t tokens, const void* dout, int64_t lddout,
                                int64_t vocab, int64_t hidden, int dtype, double scale, void* dtable, int64_t lddtable,
                                void* ws, size_t ws_bytes, void* stream) {
  return guarded(h, [&]() -> muon_status {
    std::string why;
    std::vector<Span> spans;
    muon_status st = check_ids(ids, ids_bits, tokens, vocab, spans, why);
    if (st != MUON_OK) return fail(h, st, why);
    int bytes = 0;
    const Mat mats[2] = {{dout, tokens, lddout, false, "dout"}, {dtable, vocab, lddtable, true, "dtable"}};
    st = check_rows(hidden, dtype, mats, 2, spans, bytes, why);
    if (st != MUON_OK) return fail(h, st, why);
    size_t need = 0;
    st = muon_embed_backward_workspace_size(tokens, vocab, hidden, &need);
    if (st != MUON_OK) return fail(h, st, "tokens times hidden is too large");
    if (vocab == 0 || hidden == 0) return MUON_OK;
    st = check_workspace(h, ws, ws_bytes, need, spans);
    if (st != MUON_OK) return st;
    if (find_overlap(spans, why)) return invalid(h, why);
    if (handle_device(h) < 0) return host_only(h);
    DeviceGuard guard(handle_device(h));
    return run_grad(h, grad_plan(tokens, vocab, hidden), ids, ids_bits, tokens, dout, lddout, vocab, hidden, dtype, bytes,
                    (float)scale, dtable, lddtable, static_cast<uint8_t*>(ws), stream);
  });
}

muon_status muon_pack8(muon_handle h, const void* x, int64_t ldx, int64_t rows, int64_t cols, int dtype, uint8_t* codes,
                       uint8_t* scales, void* stream) {
  return saved8(h, x, ldx, rows, cols, dtype, codes, scales, true, stream);
}

muon_status muon_unpack8(muon_handle h, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* x,
                         int64_t ldx, int dtype, void* stream) {
  return saved8(h, x, ldx, rows, cols, dtype, codes, scales, false, stream);
}

}  // extern "C"
