// C ABI of the training-step operators around the Muon step (AdamW, gradient
// clipping, tokens by expert): validation and launches.  See include/muon.h
// for the contract.
#include "muon.h"

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>
#include <memory>
#include <new>
#include <string>
#include <utility>
#include <vector>

#include "api_common.h"
#include "device_guard.h"
#include "muon_internal.h"
#include "train_internal.h"

using namespace muon;

namespace {

uint64_t splitmix64(uint64_t x) {
  x += 0x9E3779B97F4A7C15ull;
  x = (x ^ (x >> 30)) * 0xBF58476D1CE4E5B9ull;
  x = (x ^ (x >> 27)) * 0x94D049BB133111EBull;
  return x ^ (x >> 31);
}

// ---------------------------------------------------------------- AdamW

muon_status check_adamw(const muon_adamw_config& c, const muon_adamw_desc* d, int n, std::string& why) {
  if (!(c.beta1 >= 0.0 && c.beta1 < 1.0) || !(c.beta2 >= 0.0 && c.beta2 < 1.0)) {
    why = "config: beta1 and beta2 must be in [0, 1)";
    return MUON_ERR_INVALID_ARG;
  }
  if (!(c.eps >= 0.0) || !std::isfinite(c.eps)) { why = "config: eps must be finite and >= 0"; return MUON_ERR_INVALID_ARG; }
  if (n < 0) { why = "n must be >= 0"; return MUON_ERR_INVALID_ARG; }
  if (n > 0 && !d) { why = "descs is NULL"; return MUON_ERR_INVALID_ARG; }
  std::vector<Span> spans;
  spans.reserve((size_t)n * 5);
  for (int i = 0; i < n; ++i) {
    const muon_adamw_desc& x = d[i];
    auto bad = [&](const char* what) {
      why = "desc " + std::to_string(i) + ": " + what;
      return MUON_ERR_INVALID_ARG;
    };
    if (x.n < 0 || x.n > kMaxElements) return bad("n must be in [0, 2^40]");
    if (x.n == 0) continue;
    if (!known_dtype(x.p_dtype) || !known_dtype(x.g_dtype)) return bad("p_dtype and g_dtype must be MUON_F32 or MUON_BF16");
    if (x.state_bits != 32 && x.state_bits != 8) return bad("state_bits must be 32 or 8");
    if (x.reserved != 0) return bad("reserved must be 0");
    if (!x.P || !x.G || !x.M || !x.V) return bad("P, G, M and V must be non-NULL");
    if (!aligned(x.P, element_size(x.p_dtype))) return bad("P must be aligned to its element size");
    if (!aligned(x.G, element_size(x.g_dtype))) return bad("G must be aligned to its element size");
    const int64_t se = x.state_bits / 8;
    if (!aligned(x.M, se) || !aligned(x.V, se)) return bad("M and V must be aligned to their element size");
    if (x.state_bits == 8) {
      if (!x.scales) return bad("scales must be non-NULL for 8-bit states");
      if (!aligned(x.scales, 2)) return bad("scales must be 2-byte aligned");
    } else if (x.scales) {
      return bad("scales must be NULL for 32-bit states");
    }
    if (x.step < 1) return bad("step must be >= 1");
    if (!std::isfinite(x.lr) || !std::isfinite(x.weight_decay)) return bad("lr and weight_decay must be finite");
    spans.push_back(span(x.P, x.n * element_size(x.p_dtype), i, true, "P"));
    spans.push_back(span(x.G, x.n * element_size(x.g_dtype), i, false, "G"));
    spans.push_back(span(x.M, x.n * se, i, true, "M"));
    spans.push_back(span(x.V, x.n * se, i, true, "V"));
    if (x.scales) spans.push_back(span(x.scales, 2 * cdiv(x.n, kStateBlock), i, true, "scales"));
  }
  return find_overlap(spans, why) ? MUON_ERR_INVALID_ARG : MUON_OK;
}

// Elements between the vector boundary (four elements) at or before p and p.
int lead(const void* p, int64_t es) { return (int)(reinterpret_cast<uintptr_t>(p) / (uintptr_t)es % 4); }

// 1 - beta^t of a step number; most tensors of a call share it.  In double:
// 1 - beta^t loses most of its digits in fp32 for small t.
struct BiasCorrections {
  int64_t step = 0;
  double first = 0.0, second = 0.0;
  void at(const muon_adamw_config& c, int64_t t) {
    if (t == step) return;
    step = t;
    first = 1.0 - std::pow(c.beta1, (double)t);
    second = 1.0 - std::pow(c.beta2, (double)t);
  }
};

// Adds one tensor to a launch.
void add_tensor(AdamParams& a, BiasCorrections& bias, const muon_adamw_config& c, const muon_adamw_desc& x) {
  AdamTensor& t = a.t[a.n++];
  t = AdamTensor{};
  t.P = x.P;
  t.G = x.G;
  t.M = x.M;
  t.V = x.V;
  t.scales = x.scales;
  t.n = x.n;
  t.chunk_begin = a.chunks;
  t.p_bf16 = x.p_dtype == MUON_BF16;
  t.g_bf16 = x.g_dtype == MUON_BF16;
  const int64_t ps = element_size(x.p_dtype), gs = element_size(x.g_dtype);
  if (x.state_bits == 32) {
    // tensors packed one after another in flat buffers all start the same
    // number of elements past a boundary: they still move whole vectors
    const int l = lead(x.M, 4);
    t.shift = (uint8_t)l;
    t.vec = (uint8_t)((lead(x.P, ps) == l ? kVecP : 0) | (lead(x.G, gs) == l ? kVecG : 0) | (lead(x.V, 4) == l ? kVecV : 0));
  } else {
    t.vec = aligned(x.P, 16) && aligned(x.G, 16) && aligned(x.M, 16) && aligned(x.V, 16);
  }
  bias.at(c, x.step);
  t.decay = (float)(1.0 - x.lr * x.weight_decay);
  t.step_size = (float)(x.lr / bias.first);
  t.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(bias.second));
  const uint64_t key = splitmix64(x.seed + (uint64_t)x.step * 0x9E3779B97F4A7C15ull);
  t.key_lo = (uint32_t)key;
  t.key_hi = (uint32_t)(key >> 32);
  a.chunks += (uint32_t)cdiv(x.n + t.shift, a.chunk);
}

// Elements per CTA for 8-bit states: its eight warps take up to 32 blocks
// each, one after another, where there are enough of them for every SM (268 M
// bf16 elements, before later steps: 510 us with 4 blocks, 486 with 8, 471 with
// 16, 466 with 32).
int adamw8_chunk(const muon_adamw_desc* d, int n) {
  constexpr int64_t kRound = 8 * kStateBlock;   // a block for each warp
  int64_t rounds = 0;
  for (int i = 0; i < n; ++i)
    if (d[i].state_bits == 8) rounds += cdiv(d[i].n, kRound);
  return (int)(kRound * std::clamp<int64_t>(rounds / (kSms * 8), 1, 32));
}

muon_status run_adamw(muon_handle h, const muon_adamw_config& c, const muon_adamw_desc* d, int n, void* stream) {
  const bool pdl = first_pdl(stream);
  BiasCorrections bias;
  std::unique_ptr<AdamParams> a(new AdamParams);
  a->beta1 = (float)c.beta1;
  a->one_minus_beta1 = (float)(1.0 - c.beta1);
  a->beta2 = (float)c.beta2;
  a->one_minus_beta2 = (float)(1.0 - c.beta2);
  a->eps = (float)c.eps;
  a->minus_zero = -0.f;
  for (const int bits : {32, 8}) {
    a->n = 0;
    a->chunks = 0;
    a->chunk = bits == 32 ? kAdamChunk : adamw8_chunk(d, n);
    auto flush = [&]() -> muon_status {
      if (a->n == 0) return MUON_OK;
      nvtxRangePushA(bits == 32 ? "muon.adamw32" : "muon.adamw8");
      const int e = bits == 32 ? launch_adamw32(*a, stream, pdl) : launch_adamw8(*a, stream, pdl);
      nvtxRangePop();
      if (e) return cuda_fail(h, "muon_adamw_step", e);
      count_launches(h, 1);
      a->n = 0;
      a->chunks = 0;
      return MUON_OK;
    };
    for (int i = 0; i < n; ++i) {
      if (d[i].n == 0 || d[i].state_bits != bits) continue;
      const int64_t chunks = cdiv(d[i].n + 3, a->chunk);
      if (a->n == kAdamTensors || a->chunks + chunks > kInt32Max) {
        const muon_status st = flush();
        if (st != MUON_OK) return st;
      }
      add_tensor(*a, bias, c, d[i]);
    }
    const muon_status st = flush();
    if (st != MUON_OK) return st;
  }
  return MUON_OK;
}

// ---------------------------------------------------------------- clipping

struct ClipView {   // a descriptor with its defaults filled in
  const void* G;
  void* out;
  int64_t rows, cols, ldg, ldo;
  int g_dtype, o_dtype;
};

muon_status check_clip(const muon_clip_desc* d, int n, bool write, const float* norm, const void* ws,
                       std::vector<ClipView>& views, std::string& why) {
  if (n < 0) { why = "n must be >= 0"; return MUON_ERR_INVALID_ARG; }
  if (n > 0 && !d) { why = "descs is NULL"; return MUON_ERR_INVALID_ARG; }
  if (!norm || !aligned(norm, 4)) { why = "norm must be a 4-byte aligned device pointer"; return MUON_ERR_INVALID_ARG; }
  std::vector<Span> spans;
  spans.reserve((size_t)n * 2 + 2);
  views.reserve((size_t)n);
  spans.push_back(span(norm, 4, -1, true, "norm"));
  spans.push_back(span(ws, MUON_CLIP_WORKSPACE_BYTES, -1, true, "workspace"));
  for (int i = 0; i < n; ++i) {
    const muon_clip_desc& x = d[i];
    auto bad = [&](const char* what) {
      why = "desc " + std::to_string(i) + ": " + what;
      return MUON_ERR_INVALID_ARG;
    };
    if (x.rows < 0 || x.cols < 0) return bad("rows and cols must be >= 0");
    if (x.rows == 0 || x.cols == 0) continue;
    if (x.cols > kMaxElements || x.rows > kMaxElements / x.cols) return bad("rows * cols must be at most 2^40");
    if (!x.G) return bad("G must be non-NULL");
    if (!known_dtype(x.g_dtype)) return bad("g_dtype must be MUON_F32 or MUON_BF16");
    const bool in_place = !x.out || x.out == x.G;
    ClipView v{x.G, in_place ? x.G : x.out, x.rows, x.cols, x.ldg, in_place ? x.ldg : x.ldo,
               x.g_dtype, in_place ? x.g_dtype : x.out_dtype};
    if (!known_dtype(v.o_dtype)) return bad("out_dtype must be MUON_F32 or MUON_BF16");
    const int64_t ges = element_size(v.g_dtype), oes = element_size(v.o_dtype);
    if (!aligned(v.G, ges) || !aligned(v.out, oes)) return bad("G and out must be aligned to their element size");
    if (v.rows == 1) v.ldg = v.ldo = v.cols;
    if (v.ldg < v.cols || v.ldo < v.cols) return bad("ldg and ldo must be >= cols");
    if (v.rows > 1 && (v.ldg > kMaxElements / v.rows || v.ldo > kMaxElements / v.rows))
      return bad("rows times the leading dimension must be at most 2^40");
    spans.push_back(matrix_span(v.G, v.rows, v.cols, v.ldg, ges, i, write && in_place, "G"));
    if (write && !in_place) spans.push_back(matrix_span(v.out, v.rows, v.cols, v.ldo, oes, i, true, "out"));
    if (v.ldg == v.cols && v.ldo == v.cols) {
      v.cols *= v.rows;
      v.rows = 1;
      v.ldg = v.ldo = v.cols;
    }
    views.push_back(v);
  }
  return find_overlap(spans, why) ? MUON_ERR_INVALID_ARG : MUON_OK;
}

int64_t add_tensor(ClipParams& p, const ClipView& v) {
  ClipTensor& t = p.t[p.n];
  t = ClipTensor{};
  t.G = v.G;
  t.out = v.out;
  t.ldg = v.ldg;
  t.ldo = v.ldo;
  t.rows = v.rows;
  t.cols = v.cols;
  t.g_bf16 = v.g_dtype == MUON_BF16;
  t.o_bf16 = v.o_dtype == MUON_BF16;
  const int64_t ges = element_size(v.g_dtype), oes = element_size(v.o_dtype);
  const int l = lead(v.G, ges);
  if (v.rows == 1) {
    t.vec = 1;
    t.vec_out = lead(v.out, oes) == l;
    t.shift = (uint8_t)l;
  } else {
    t.vec = l == 0 && v.ldg % 4 == 0;
    t.vec_out = lead(v.out, oes) == 0 && v.ldo % 4 == 0;
  }
  t.seg = (int32_t)std::min<int64_t>(v.cols + t.shift, kClipChunk);
  t.segs_per_row = cdiv(v.cols + t.shift, t.seg);
  t.rows_per_chunk = (int32_t)std::min<int64_t>(v.rows, std::max<int64_t>(1, kClipChunk / t.seg));
  t.chunk_begin = p.chunks;
  return cdiv(v.rows, t.rows_per_chunk) * t.segs_per_row;
}

muon_status run_clip(muon_handle h, const std::vector<ClipView>& views, double max_norm, float* norm, void* ws,
                     void* stream) {
  // tensors of each launch, at most kClipTensors
  std::vector<std::unique_ptr<ClipParams>> launches;
  for (const ClipView& v : views) {
    if (launches.empty() || launches.back()->n == kClipTensors) {
      launches.emplace_back(new ClipParams);
      launches.back()->n = 0;
      launches.back()->chunks = 0;
    }
    ClipParams* p = launches.back().get();
    int64_t chunks = add_tensor(*p, v);
    if (chunks > kInt32Max) return fail(h, MUON_ERR_INVALID_ARG, "a gradient has too many rows");
    if (p->chunks + chunks > kInt32Max) {
      launches.emplace_back(new ClipParams);
      p = launches.back().get();
      p->n = 0;
      p->chunks = 0;
      chunks = add_tensor(*p, v);
    }
    p->n += 1;
    p->chunks += (uint32_t)chunks;
  }
  if (launches.empty()) {   // nothing but the norm, 0
    launches.emplace_back(new ClipParams);
    launches.back()->n = 0;
    launches.back()->chunks = 0;
  }
  if ((int64_t)launches.size() > kClipPartials) return fail(h, MUON_ERR_INVALID_ARG, "too many gradients in one call");
  const int most = std::max<int>(1, std::min<int>(kClipPartials / (int)launches.size(), kSms * 8));
  int partials = 0;
  for (auto& p : launches) {
    p->partial_begin = partials;
    partials += (int)std::min<int64_t>(std::max<int64_t>(p->chunks, 1), most);
  }
  bool first = true;
  for (auto& p : launches) {
    p->partials = partials;
    p->write_norm = p == launches.front();
    p->max_norm = (float)max_norm;
    p->partial = static_cast<double*>(ws);
    p->norm = norm;
    const int grid = (int)std::min<int64_t>(std::max<int64_t>(p->chunks, 1), most);
    nvtxRangePushA("muon.clip_sumsq");
    const int e = launch_clip_sumsq(*p, grid, stream, first ? first_pdl(stream) : kUsePdl);
    nvtxRangePop();
    if (e) return cuda_fail(h, "muon_clip_grads", e);
    count_launches(h, 1);
    first = false;
  }
  const bool write = std::isfinite(max_norm);
  for (auto& p : launches) {
    if (!write) p->chunks = 0;   // the norm alone
    const int grid = (int)std::min<int64_t>(std::max<int64_t>(p->chunks, 1), kSms * 8);
    nvtxRangePushA("muon.clip_scale");
    const int e = launch_clip_scale(*p, grid, stream, kUsePdl);
    nvtxRangePop();
    if (e) return cuda_fail(h, "muon_clip_grads", e);
    count_launches(h, 1);
    if (!write) break;
  }
  return MUON_OK;
}

// ---------------------------------------------------------------- tokens by expert

muon_status check_shape(const muon_moe_shape* s, int64_t& rows, std::string& why) {
  auto bad = [&](const char* what) {
    why = std::string("shape: ") + what;
    return MUON_ERR_INVALID_ARG;
  };
  if (!s) return bad("NULL");
  if (s->topk < 1 || s->topk > kMoeMaxTopk) return bad("topk must be in [1, 64]");
  if (s->experts < 1 || s->experts > kMoeMaxExperts) return bad("experts must be in [1, 1024]");
  if (s->tokens < 0 || s->tokens > kInt32Max / s->topk) return bad("tokens must be >= 0 and tokens * topk < 2^31");
  if (s->capacity < 0) return bad("capacity must be >= 0");
  if (s->align < 1) return bad("align must be >= 1");
  if (s->capacity > 0 && s->align != 1) return bad("align must be 1 when capacity > 0");
  if (s->capacity > 0) rows = (int64_t)s->experts * s->capacity;
  else rows = cdiv(s->tokens * s->topk + (int64_t)s->experts * (s->align - 1), s->align) * s->align;
  if (rows > kInt32Max) return bad("the sorted rows must number less than 2^31");
  return MUON_OK;
}

int sort_ctas(const muon_moe_shape& s, int& per_cta) {
  const int64_t slots = s.tokens * s.topk;
  if (slots <= kSortSingle) {
    per_cta = (int)slots;
    return 1;
  }
  // whole rounds of the CTA's threads
  per_cta = (int)std::min<int64_t>(kInt32Max, cdiv(cdiv(slots, kSortGrid), kSortThreads) * kSortThreads);
  return (int)cdiv(slots, per_cta);
}

size_t sort_bytes(const muon_moe_shape& s) {
  int per_cta = 0;
  const int ctas = sort_ctas(s, per_cta);
  return ctas == 1 ? 0 : (size_t)ctas * (size_t)s.experts * sizeof(int32_t);
}

muon_status check_index(const muon_moe_shape& s, const int32_t* row, const int32_t* offsets, const int32_t* counts,
                        bool segments, bool written, std::vector<Span>& spans, std::string& why) {
  if (s.tokens > 0 && !row) { why = "row must be non-NULL"; return MUON_ERR_INVALID_ARG; }
  if (segments && (!offsets || !counts)) { why = "offsets and counts must be non-NULL"; return MUON_ERR_INVALID_ARG; }
  if (!aligned(row, 4) || !aligned(offsets, 4) || !aligned(counts, 4)) {
    why = "row, offsets and counts must be 4-byte aligned";
    return MUON_ERR_INVALID_ARG;
  }
  spans.push_back(span(row, s.tokens * s.topk * 4, -1, written, "row"));
  if (segments) {
    spans.push_back(span(offsets, ((int64_t)s.experts + 1) * 4, -1, written, "offsets"));
    spans.push_back(span(counts, (int64_t)s.experts * 4, -1, written, "counts"));
  }
  return MUON_OK;
}

// Elements that a thread of a row kernel takes at once: 16 bytes, or `units`
// units of 4 bytes or one element.
int64_t elements_at_once(int bytes, int dtype, int units) { return (bytes == 16 ? 1 : units) * bytes / element_size(dtype); }

RowsParams rows_params(const muon_moe_shape& s, int64_t rows, int64_t hidden, int dtype, int bytes, int units, bool staged,
                       int64_t& token_ctas) {
  RowsParams p{};
  p.hidden = hidden;
  p.tokens = s.tokens;
  p.topk = s.topk;
  p.experts = s.experts;
  p.rows = (int32_t)rows;
  const int64_t per = elements_at_once(bytes, dtype, units);
  p.tx = 32;
  while (p.tx < kThreads256 && p.tx * per < hidden) p.tx *= 2;
  const int64_t rows_of_threads = kThreads256 / p.tx;
  if (staged) {
    // tokens of a CTA: what its threads take at once, several times over when
    // there are many tokens (16384 tokens of 8 choices, 2048 wide: combine 107 us
    // and backward 184 with 6 times, 119 and 235 with once, 116 and 195 with 13
    // times); the shared memory for their rows, weights and sums stays within
    // 32 KB
    const int64_t at_once = rows_of_threads * std::max<int64_t>(1, 4 / s.topk);
    const int64_t room = 32768 / ((int64_t)s.topk * (8 + p.tx / 8));
    const int64_t passes = std::clamp<int64_t>(s.tokens / (at_once * kSms * 16), 1, 8);
    p.tokens_per_cta = (int32_t)std::clamp<int64_t>(std::min(at_once * passes, cdiv(s.tokens, kSms)), 1, room);
  } else {
    p.tokens_per_cta = (int32_t)rows_of_threads;
  }
  token_ctas = cdiv(s.tokens, p.tokens_per_cta);
  p.token_ctas = (int32_t)token_ctas;
  return p;
}

// CTAs that clear rows without a token: a few per SM at most, and no more than
// one row per warp needs.
int64_t clear_ctas(int64_t rows) { return std::min<int64_t>(cdiv(rows, kThreads256 / 32), kSms * 2); }

}  // namespace

extern "C" {

void muon_adamw_config_default(muon_adamw_config* c) {
  if (!c) return;
  c->beta1 = 0.9;
  c->beta2 = 0.95;
  c->eps = 1e-8;
}

muon_status muon_adamw_step(muon_handle h, const muon_adamw_config* cfg, const muon_adamw_desc* descs, int n,
                            void* stream) {
  return guarded(h, [&]() -> muon_status {
    muon_adamw_config c;
    if (cfg) c = *cfg; else muon_adamw_config_default(&c);
    std::string why;
    const muon_status st = check_adamw(c, descs, n, why);
    if (st != MUON_OK) return fail(h, st, why);
    bool any = false;
    for (int i = 0; i < n; ++i) any = any || descs[i].n > 0;
    if (!any) return MUON_OK;
    if (handle_device(h) < 0) return fail(h, MUON_ERR_UNSUPPORTED, "host-only handle: create it with a device to run steps");
    DeviceGuard guard(handle_device(h));
    return run_adamw(h, c, descs, n, stream);
  });
}

muon_status muon_clip_grads(muon_handle h, const muon_clip_desc* descs, int n, double max_norm, float* norm, void* ws,
                            size_t ws_bytes, void* stream) {
  return guarded(h, [&]() -> muon_status {
    if (!(max_norm > 0.0)) return fail(h, MUON_ERR_INVALID_ARG, "max_norm must be > 0");
    std::vector<ClipView> views;
    std::string why;
    const muon_status st = check_clip(descs, n, std::isfinite(max_norm), norm, ws, views, why);
    if (st != MUON_OK) return fail(h, st, why);
    if (!ws) return fail(h, MUON_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(ws, 256)) return fail(h, MUON_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (ws_bytes < MUON_CLIP_WORKSPACE_BYTES)
      return fail(h, MUON_ERR_WORKSPACE, "workspace too small: need " + std::to_string(MUON_CLIP_WORKSPACE_BYTES) + " bytes");
    if (handle_device(h) < 0) return fail(h, MUON_ERR_UNSUPPORTED, "host-only handle: create it with a device to run steps");
    DeviceGuard guard(handle_device(h));
    return run_clip(h, views, max_norm, norm, ws, stream);
  });
}

muon_status muon_moe_rows(const muon_moe_shape* shape, int64_t* rows) {
  if (!rows) return MUON_ERR_INVALID_ARG;
  try {
    std::string why;
    return check_shape(shape, *rows, why);
  } catch (...) {   // no memory for the text
    return MUON_ERR_INVALID_ARG;
  }
}

muon_status muon_moe_sort_workspace_size(const muon_moe_shape* shape, size_t* bytes) {
  int64_t rows = 0;
  if (!bytes) return MUON_ERR_INVALID_ARG;
  const muon_status st = muon_moe_rows(shape, &rows);
  if (st == MUON_OK) *bytes = sort_bytes(*shape);
  return st;
}

muon_status muon_moe_sort(muon_handle h, const muon_moe_shape* shape, const void* ids, int ids_bits, int32_t* row,
                          int32_t* offsets, int32_t* counts, void* ws, size_t ws_bytes, void* stream) {
  return guarded(h, [&]() -> muon_status {
    std::string why;
    int64_t rows = 0;
    muon_status st = check_shape(shape, rows, why);
    if (st != MUON_OK) return fail(h, st, why);
    if (ids_bits != 32 && ids_bits != 64) return fail(h, MUON_ERR_INVALID_ARG, "ids_bits must be 32 or 64");
    const int64_t slots = shape->tokens * shape->topk;
    if (slots > 0 && !ids) return fail(h, MUON_ERR_INVALID_ARG, "ids must be non-NULL");
    if (!aligned(ids, ids_bits / 8)) return fail(h, MUON_ERR_INVALID_ARG, "ids must be aligned to their size");
    std::vector<Span> spans;
    st = check_index(*shape, row, offsets, counts, true, true, spans, why);
    if (st != MUON_OK) return fail(h, st, why);
    spans.push_back(span(ids, slots * (ids_bits / 8), -1, false, "ids"));
    const size_t need = sort_bytes(*shape);
    if (need > 0) {
      if (!ws) return fail(h, MUON_ERR_WORKSPACE, "workspace is NULL");
      if (!aligned(ws, 256)) return fail(h, MUON_ERR_WORKSPACE, "workspace must be 256-byte aligned");
      if (ws_bytes < need) return fail(h, MUON_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) + " bytes");
      spans.push_back(span(ws, (int64_t)need, -1, true, "workspace"));
    }
    if (find_overlap(spans, why)) return fail(h, MUON_ERR_INVALID_ARG, why);
    if (handle_device(h) < 0) return fail(h, MUON_ERR_UNSUPPORTED, "host-only handle: create it with a device to run");
    DeviceGuard guard(handle_device(h));
    SortParams p{};
    p.ids = ids;
    p.ids64 = ids_bits == 64;
    p.slots = (int32_t)slots;
    p.ctas = sort_ctas(*shape, p.per_cta);
    p.experts = shape->experts;
    p.capacity = shape->capacity;
    p.align = shape->align;
    p.row = row;
    p.offsets = offsets;
    p.counts = counts;
    p.hist = need > 0 ? static_cast<int32_t*>(ws) : nullptr;
    int e = 0;
    nvtxRangePushA("muon.moe_sort");
    const bool pdl = first_pdl(stream);
    if (need > 0) e = launch_moe_sort_count(p, stream, pdl);
    if (!e) e = launch_moe_sort_place(p, stream, need > 0 ? kUsePdl : pdl);
    nvtxRangePop();
    if (e) return cuda_fail(h, "muon_moe_sort", e);
    count_launches(h, need > 0 ? 2 : 1);
    return MUON_OK;
  });
}

muon_status muon_moe_dispatch(muon_handle h, const muon_moe_shape* shape, const int32_t* row, const int32_t* offsets,
                              const int32_t* counts, const void* x, int64_t ldx, void* xs, int64_t ldxs,
                              int64_t hidden, int dtype, void* stream) {
  return guarded(h, [&]() -> muon_status {
    std::string why;
    int64_t rows = 0;
    muon_status st = check_shape(shape, rows, why);
    if (st != MUON_OK) return fail(h, st, why);
    std::vector<Span> spans;
    st = check_index(*shape, row, offsets, counts, true, false, spans, why);
    if (st != MUON_OK) return fail(h, st, why);
    int bytes = 0;
    const Mat mats[2] = {{x, shape->tokens, ldx, false, "x"}, {xs, rows, ldxs, true, "xs"}};
    st = check_rows(hidden, dtype, mats, 2, spans, bytes, why);
    if (st != MUON_OK) return fail(h, st, why);
    if (rows == 0 || hidden == 0) return MUON_OK;
    if (handle_device(h) < 0) return fail(h, MUON_ERR_UNSUPPORTED, "host-only handle: create it with a device to run");
    DeviceGuard guard(handle_device(h));
    int64_t token_ctas = 0;
    RowsParams p = rows_params(*shape, rows, hidden, dtype, bytes, kRowUnits, false, token_ctas);
    p.x = x;
    p.ldx = ldx;
    p.out = xs;
    p.ldo = ldxs;
    p.row = row;
    p.offsets = offsets;
    p.counts = counts;
    const int64_t grid = token_ctas + clear_ctas(rows);
    if (grid > kInt32Max) return fail(h, MUON_ERR_INVALID_ARG, "tokens: too many for one launch");
    nvtxRangePushA("muon.moe_dispatch");
    const int e = launch_moe_dispatch(p, dtype == MUON_BF16, bytes, (int)grid, stream, first_pdl(stream));
    nvtxRangePop();
    if (e) return cuda_fail(h, "muon_moe_dispatch", e);
    count_launches(h, 1);
    return MUON_OK;
  });
}

muon_status muon_moe_combine(muon_handle h, const muon_moe_shape* shape, const int32_t* row, const void* ys,
                             int64_t ldys, const void* weights, int w_dtype, void* out, int64_t ldout, int64_t hidden,
                             int dtype, void* stream) {
  return guarded(h, [&]() -> muon_status {
    std::string why;
    int64_t rows = 0;
    muon_status st = check_shape(shape, rows, why);
    if (st != MUON_OK) return fail(h, st, why);
    std::vector<Span> spans;
    st = check_index(*shape, row, nullptr, nullptr, false, false, spans, why);
    if (st != MUON_OK) return fail(h, st, why);
    if (weights) {
      if (!known_dtype(w_dtype)) return fail(h, MUON_ERR_INVALID_ARG, "w_dtype must be MUON_F32 or MUON_BF16");
      if (!aligned(weights, element_size(w_dtype)))
        return fail(h, MUON_ERR_INVALID_ARG, "weights must be aligned to their element size");
      spans.push_back(span(weights, shape->tokens * shape->topk * element_size(w_dtype), -1, false, "weights"));
    }
    int bytes = 0;
    const Mat mats[2] = {{ys, rows, ldys, false, "ys"}, {out, shape->tokens, ldout, true, "out"}};
    st = check_rows(hidden, dtype, mats, 2, spans, bytes, why);
    if (st != MUON_OK) return fail(h, st, why);
    if (shape->tokens == 0 || hidden == 0) return MUON_OK;
    if (handle_device(h) < 0) return fail(h, MUON_ERR_UNSUPPORTED, "host-only handle: create it with a device to run");
    DeviceGuard guard(handle_device(h));
    int64_t token_ctas = 0;
    RowsParams p = rows_params(*shape, rows, hidden, dtype, bytes, kRowUnits, true, token_ctas);
    p.x = ys;
    p.ldx = ldys;
    p.out = out;
    p.ldo = ldout;
    p.row = row;
    p.w = weights;
    p.w_bf16 = w_dtype == MUON_BF16;
    // a few tokens: their columns are spread over the SMs (5 tokens, 6144 wide: 5.1 us
    // against 7.5)
    const int64_t columns = cdiv(hidden, p.tx * elements_at_once(bytes, dtype, kRowUnits));
    p.splits = (int32_t)std::clamp<int64_t>(kSms / token_ctas, 1, columns);
    nvtxRangePushA("muon.moe_combine");
    const int e = launch_moe_combine(p, dtype == MUON_BF16, bytes, (int)(token_ctas * p.splits), stream, first_pdl(stream));
    nvtxRangePop();
    if (e) return cuda_fail(h, "muon_moe_combine", e);
    count_launches(h, 1);
    return MUON_OK;
  });
}

muon_status muon_moe_combine_backward(muon_handle h, const muon_moe_shape* shape, const int32_t* row,
                                      const int32_t* offsets, const int32_t* counts, const void* dout, int64_t lddout,
                                      const void* ys, int64_t ldys, const void* weights, int w_dtype, void* dys,
                                      int64_t lddys, void* dweights, int64_t hidden, int dtype, void* stream) {
  return guarded(h, [&]() -> muon_status {
    std::string why;
    int64_t rows = 0;
    muon_status st = check_shape(shape, rows, why);
    if (st != MUON_OK) return fail(h, st, why);
    std::vector<Span> spans;
    st = check_index(*shape, row, offsets, counts, true, false, spans, why);
    if (st != MUON_OK) return fail(h, st, why);
    if (!known_dtype(w_dtype)) return fail(h, MUON_ERR_INVALID_ARG, "w_dtype must be MUON_F32 or MUON_BF16");
    const int64_t wes = element_size(w_dtype);
    if (shape->tokens > 0 && (!weights || !dweights))
      return fail(h, MUON_ERR_INVALID_ARG, "weights and dweights must be non-NULL");
    if (!aligned(weights, wes) || !aligned(dweights, wes))
      return fail(h, MUON_ERR_INVALID_ARG, "weights and dweights must be aligned to their element size");
    spans.push_back(span(weights, shape->tokens * shape->topk * wes, -1, false, "weights"));
    spans.push_back(span(dweights, shape->tokens * shape->topk * wes, -1, true, "dweights"));
    int bytes = 0;
    const Mat mats[3] = {{dout, shape->tokens, lddout, false, "dout"}, {ys, rows, ldys, false, "ys"},
                         {dys, rows, lddys, true, "dys"}};
    st = check_rows(hidden, dtype, mats, 3, spans, bytes, why);
    if (st != MUON_OK) return fail(h, st, why);
    if (handle_device(h) < 0) return fail(h, MUON_ERR_UNSUPPORTED, "host-only handle: create it with a device to run");
    DeviceGuard guard(handle_device(h));
    int64_t token_ctas = 0;
    RowsParams p = rows_params(*shape, rows, hidden, dtype, bytes, 1, true, token_ctas);
    p.x = dout;
    p.ldx = lddout;
    p.y = ys;
    p.ldy = ldys;
    p.out = dys;
    p.ldo = lddys;
    p.w = weights;
    p.dw = dweights;
    p.w_bf16 = w_dtype == MUON_BF16;
    p.row = row;
    p.offsets = offsets;
    p.counts = counts;
    const int64_t grid = token_ctas + clear_ctas(rows);
    if (grid == 0) return MUON_OK;
    if (grid > kInt32Max) return fail(h, MUON_ERR_INVALID_ARG, "tokens: too many for one launch");
    nvtxRangePushA("muon.moe_combine_backward");
    const int e = launch_moe_backward(p, dtype == MUON_BF16, bytes, (int)grid, stream, first_pdl(stream));
    nvtxRangePop();
    if (e) return cuda_fail(h, "muon_moe_combine_backward", e);
    count_launches(h, 1);
    return MUON_OK;
  });
}

}  // extern "C"
