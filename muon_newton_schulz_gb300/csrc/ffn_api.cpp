// C ABI of the gated feed-forward block: validation, workspace and launches.
// See include/muon.h for the contract.
#include "muon.h"

#include <nvtx3/nvToolsExt.h>

#include "api_common.h"
#include "device_guard.h"
#include "ffn_internal.h"
#include "layer_internal.h"
#include "muon_internal.h"

using namespace muon;

namespace {

constexpr int64_t kMaxWidth = 1ll << 21;

// Row length of buffers over the ffn width: whole words of four scale bytes.
int64_t ld_of(int64_t ffn) { return cdiv(ffn, 128) * 128; }
// Row length of the workspace's copy of x.
int64_t ld_x(int64_t hidden) { return cdiv(hidden, 8) * 8; }

muon_status check_shape(const muon_ffn_shape* s, std::string& why) {
  auto bad = [&](const char* what) {
    why = std::string("shape: ") + what;
    return MUON_ERR_INVALID_ARG;
  };
  if (!s) return bad("NULL");
  if (s->rows < 0 || s->rows > kInt32Max) return bad("rows must be in [0, 2^31)");
  if (s->hidden < 0 || s->hidden > kMaxWidth || s->ffn < 0 || s->ffn > kMaxWidth) return bad("hidden and ffn must be in [0, 2^21]");
  if (s->experts < 1 || s->experts > kMoeMaxExperts) return bad("experts must be in [1, 1024]");
  if (!known_dtype(s->dtype)) return bad("dtype must be MUON_F32 or MUON_BF16");
  if (s->activation != MUON_SILU && s->activation != MUON_GELU) return bad("activation must be MUON_SILU or MUON_GELU");
  if (s->saved_bits != 0 && s->saved_bits != 8 && s->saved_bits != 8 * element_size(s->dtype))
    return bad("saved_bits must be 0, 8 or the bits of dtype");
  if (s->rows > 0 && (ld_of(s->ffn) > kMaxElements / s->rows || ld_x(s->hidden) > kMaxElements / s->rows))
    return bad("rows times hidden and ffn must be at most 2^40");
  return MUON_OK;
}

// Where the workspace holds what.
struct Space {
  size_t act = 0, dgate = 0, dup = 0, x = 0, maps = 0, bytes = 0;
  // copies whose rows begin 16 bytes apart
  size_t dy = 0, w[3] = {}, y = 0, dw[3] = {};
  size_t part = 0;          // sums of splits
};

int64_t up8(int64_t n) { return cdiv(n, 8) * 8; }

// Pairs of CTAs that share the depth of y's or dx's tiles: where the tiles keep less than half
// of them busy, and eight steps of 64 at least for each (one layer, 2048 x 8192: 64 rows
// forward 34 us against 56, 256 rows 41 against 59).
int splits_for(const muon_ffn_shape& s, int64_t steps) {
  constexpr int64_t kPairs = 76;
  const int64_t tiles = (s.rows / 256 + std::min<int64_t>(s.rows, s.experts)) * cdiv(s.hidden, 256);
  if (s.dtype != MUON_BF16 || tiles == 0 || tiles * 2 > kPairs || steps < 16) return 1;
  const int64_t splits = std::min(kPairs / tiles, steps / 8);
  return (int)cdiv(steps, cdiv(steps, splits));   // none without a step
}
int splits_of(const muon_ffn_shape& s, bool backward) { return splits_for(s, (backward ? 2 : 1) * cdiv(s.ffn, 64)); }
int64_t ld_part(int64_t hidden) { return cdiv(hidden, 32) * 32; }
// Widths whose rows of bf16 do not all begin on 16-byte boundaries: operands are copied.
bool loose(const muon_ffn_shape& s) { return s.dtype == MUON_BF16 && (s.hidden % 8 != 0 || s.ffn % 8 != 0); }

Space space_of(const muon_ffn_shape& s, bool backward) {
  Space w;
  auto take = [&](int64_t elements) {
    const size_t at = w.bytes;
    w.bytes += ((size_t)(elements * element_size(s.dtype)) + 255) / 256 * 256;
    return at;
  };
  const int64_t wide = s.rows * ld_of(s.ffn), narrow = s.rows * ld_x(s.hidden);
  if (loose(s)) {
    if (!backward || s.saved_bits != 8) w.x = take(narrow);
    // a matrix may be contiguous in either direction
    for (size_t& at : w.w) at = take(s.experts * std::max(s.ffn * up8(s.hidden), s.hidden * up8(s.ffn)));
    if (s.hidden % 8 != 0) w.y = take(narrow);   // y or dx
    if (backward) w.dy = take(narrow);
    for (int i = 0; backward && i < 3; ++i)
      if ((i < 2 ? s.hidden : s.ffn) % 8 != 0) w.dw[i] = take(s.experts * (i < 2 ? s.ffn * up8(s.hidden) : s.hidden * up8(s.ffn)));
  }
  const int splits = splits_of(s, backward);
  if (splits > 1) w.part = take(splits * s.rows * ld_part(s.hidden) * (4 / element_size(s.dtype)));
  if (!backward) {
    const bool two_terms = s.saved_bits == 0 && s.dtype == MUON_BF16 && s.rows <= kFfnFewRows;   // of h
    if (s.saved_bits == 0 || s.saved_bits == 8) w.act = take(two_terms ? 2 * wide : wide);
    return w;
  }
  w.dgate = take(wide);
  w.dup = take(wide);
  w.maps = w.bytes;
  if (s.dtype == MUON_BF16) w.bytes += (size_t)s.experts * kFfnMaps * sizeof(CUtensorMap);   // 128 bytes each
  if (s.saved_bits == 8) {
    w.act = take(wide);
    w.x = take(narrow);
  }
  return w;
}

// Everything of one call.
struct Call {
  muon_ffn_shape s;
  FfnRows rows;
  const void *x, *dy;
  int64_t ldx, lddy, ldy, lddx;
  FfnStack w[3], dw[3];     // gate, up, down
  void *y, *dx;
  FfnSaved kept;
  void* act;
  const uint8_t *x_codes, *x_scales;
  Space space;
  uint8_t* ws;
};

muon_status check_stack(const muon_stack* m, const muon_ffn_shape& s, int64_t rows, int64_t cols, bool read, const char* name,
                        std::vector<Span>& spans, FfnStack& out, std::string& why) {
  auto bad = [&](const char* what) {
    why = std::string(name) + what;
    return MUON_ERR_INVALID_ARG;
  };
  out = FfnStack{};
  if (!read && (!m || !m->p)) return MUON_OK;
  if (!m) return bad(" must be non-NULL");
  if (rows == 0 || cols == 0) return MUON_OK;
  if (!m->p) return bad(" must be non-NULL");
  const int64_t es = element_size(s.dtype);
  if (!aligned(m->p, es)) return bad(" must be aligned to its element size");
  int64_t se = m->stride[0], si = m->stride[1], sj = m->stride[2];
  if (s.experts == 1) se = 0;
  if (cols == 1) sj = 1;
  if (sj == 1 && rows == 1) si = cols;
  if (sj != 1 && rows == 1) si = 1;
  const bool wide = sj == 1;
  if (!wide && (si != 1 || !read)) return bad(read ? ": stride[1] or stride[2] must be 1" : ": stride[2] must be 1");
  const int64_t ld = wide ? si : sj, lines = wide ? rows : cols, line = wide ? cols : rows;
  if (ld < line || ld > kMaxElements / lines) return bad(": rows must not overlap, and rows times their distance be at most 2^40");
  const int64_t extent = (lines - 1) * ld + line;
  if (s.experts > 1 && (se < extent || se > kMaxElements / s.experts)) return bad(": stride[0] must span a matrix, and all of them at most 2^40");
  if (read && s.dtype == MUON_BF16 && !loose(s)) {
    if (!aligned(m->p, 16) || (lines > 1 && ld % 8 != 0) || se % 8 != 0) return bad(": rows of bf16 must begin on 16-byte boundaries");
  }
  spans.push_back(span(m->p, ((s.experts - 1) * se + extent) * es, -1, !read, name));
  out = FfnStack{m->p, se, si, sj};
  return MUON_OK;
}

muon_status check_route(const muon_ffn_shape& s, const int32_t* offsets, const int32_t* counts, std::vector<Span>& spans, std::string& why) {
  if (!offsets != !counts) { why = "offsets and counts must both be given, or both be NULL"; return MUON_ERR_INVALID_ARG; }
  if (!offsets && s.experts != 1) { why = "offsets and counts must be non-NULL with several experts"; return MUON_ERR_INVALID_ARG; }
  if (!aligned(offsets, 4) || !aligned(counts, 4)) { why = "offsets and counts must be 4-byte aligned"; return MUON_ERR_INVALID_ARG; }
  if (offsets) {
    spans.push_back(span(offsets, ((int64_t)s.experts + 1) * 4, -1, false, "offsets"));
    spans.push_back(span(counts, (int64_t)s.experts * 4, -1, false, "counts"));
  }
  return MUON_OK;
}

muon_status check_matrix(const muon_ffn_shape& s, const void* p, int64_t ld, bool read, const char* name, std::vector<Span>& spans,
                         std::string& why) {
  int bytes = 0;
  const Mat m[1] = {{p, s.rows, ld, !read, name}};
  const muon_status st = check_rows(s.hidden, s.dtype, m, 1, spans, bytes, why);
  if (st != MUON_OK || s.rows == 0 || s.hidden == 0) return st;
  if (read && s.dtype == MUON_BF16 && !loose(s) && (!aligned(p, 16) || (s.rows > 1 && ld % 8 != 0))) {
    why = std::string(name) + ": rows of bf16 must begin on 16-byte boundaries";
    return MUON_ERR_INVALID_ARG;
  }
  return MUON_OK;
}

muon_status check_saved(const muon_ffn_shape& s, const muon_ffn_saved* v, bool written, std::vector<Span>& spans, Call& c, std::string& why) {
  c.kept = FfnSaved{};
  if (s.saved_bits == 0) {
    if (v) { why = "saved must be NULL when saved_bits is 0"; return MUON_ERR_INVALID_ARG; }
    return MUON_OK;
  }
  if (!v) { why = "saved must be non-NULL"; return MUON_ERR_INVALID_ARG; }
  const bool eight = s.saved_bits == 8, scaled = s.saved_bits != 32;
  const int64_t n = s.rows * ld_of(s.ffn), es = s.saved_bits / 8, nx = s.rows * s.hidden;
  struct Part { const void* p; int64_t bytes; bool needed; const char* name; };
  const Part parts[] = {{v->gate, n * es, true, "saved gate"}, {v->up, n * es, true, "saved up"}, {v->act, n * es, !eight, "saved act"},
                        {v->gate_scales, n / 32, scaled, "saved gate_scales"}, {v->up_scales, n / 32, scaled, "saved up_scales"},
                        {v->x_codes, nx, eight, "saved x_codes"},
                        {v->x_scales, s.rows * cdiv(s.hidden, kSaved8Block), eight, "saved x_scales"}};
  for (const Part& p : parts) {
    if (!p.needed) {
      if (p.p) { why = std::string(p.name) + " must be NULL for these saved_bits"; return MUON_ERR_INVALID_ARG; }
      continue;
    }
    if (p.bytes == 0) continue;
    if (!p.p) { why = std::string(p.name) + " must be non-NULL"; return MUON_ERR_INVALID_ARG; }
    if (!aligned(p.p, 4)) { why = std::string(p.name) + " must be 4-byte aligned"; return MUON_ERR_INVALID_ARG; }
    if (!aligned(p.p, 32) && p.bytes >= n) { why = std::string(p.name) + " must be 32-byte aligned"; return MUON_ERR_INVALID_ARG; }
    spans.push_back(span(p.p, p.bytes, -1, written, p.name));
  }
  c.kept = FfnSaved{v->gate, v->up, v->gate_scales, v->up_scales, s.saved_bits};
  c.act = v->act;
  c.x_codes = v->x_codes;
  c.x_scales = v->x_scales;
  return MUON_OK;
}

muon_status check_space(muon_handle h, Call& c, bool backward, void* ws, size_t ws_bytes, std::vector<Span>& spans) {
  c.space = space_of(c.s, backward);
  c.ws = static_cast<uint8_t*>(ws);
  if (c.space.bytes == 0) return MUON_OK;
  if (!ws) return fail(h, MUON_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(h, MUON_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < c.space.bytes)
    return fail(h, MUON_ERR_WORKSPACE, "workspace too small: need " + std::to_string(c.space.bytes) + " bytes");
  spans.push_back(span(ws, (int64_t)c.space.bytes, -1, true, "workspace"));
  return MUON_OK;
}

// One after another on a stream; the first error stops the rest.
struct Launches {
  muon_handle h;
  void* stream;
  const char* call;
  bool pdl;
  int e = 0;
  Launches(muon_handle h_, void* stream_, const char* call_) : h(h_), stream(stream_), call(call_), pdl(first_pdl(stream_)) {}
  template <typename F>
  void operator()(const char* range, F f) {
    if (e) return;
    nvtxRangePushA(range);
    e = f(pdl);
    nvtxRangePop();
    if (e) return;
    count_launches(h, 1);
    pdl = kUsePdl;
  }
  muon_status done() { return e ? cuda_fail(h, call, e) : MUON_OK; }
};

// One of the products of a pass: a's rows with b's rows, twice for two segments
// (kInput) or two results (kGated).
struct Product {
  FfnProduct what;
  const char* range;
  const void* a[2];
  int64_t lda;              // rows of the sorted tokens
  FfnStack b[2];            // columns of the result x depth
  int64_t n, k;
  void* out;
  int64_t ldo;
  void *act, *dgate, *dup;
};

FfnStack rows_stack(const void* p, int64_t ld) { return FfnStack{const_cast<void*>(p), 0, ld, 1}; }
FfnStack turned(const FfnStack& m) { return FfnStack{m.p, m.se, m.sj, m.si}; }

// Bytes that a store to rows of bf16 may have.
int store_bytes(const void* p, int64_t ld, int64_t more) {
  for (const int n : {32, 16})
    if (aligned(p, n) && ld * 2 % n == 0 && more * 2 % n == 0) return n;
  return 2;
}

bool on_tensor_cores(const muon_ffn_shape& s) { return s.dtype == MUON_BF16; }
// Sums over nothing: every result is 0.
bool nothing(const muon_ffn_shape& s) { return s.rows == 0 || s.hidden == 0 || s.ffn == 0; }

struct Pass {
  muon_handle h;
  const Call& c;
  Launches go;
  bool tc, bad_map = false;
  FfnSimtParams input{};    // of the input's gradient in fp32, until the weights' are known
  Pass(muon_handle h_, const Call& c_, void* stream, const char* call)
      : h(h_), c(c_), go(h_, stream, call), tc(on_tensor_cores(c_.s)) {}

  int64_t ldf() const { return ld_of(c.s.ffn); }

  // Lines of a row operand: cols x rows, one after another `ld` elements.
  bool rows_map(CUtensorMap* map, const void* p, int64_t cols, int64_t ld, uint32_t box1) {
    if (c.s.rows == 1) ld = cdiv(cols, 8) * 8;
    return encode_operand_map(h, map, p, (uint64_t)cols, (uint64_t)c.s.rows, 1, (uint64_t)ld * 2, (uint64_t)ld * 2, 64, box1);
  }
  // Sets a matrix, or each of a stack, to zero.
  void zero(void* p, int64_t rows, int64_t cols, int64_t ld) {
    const size_t es = (size_t)element_size(c.s.dtype);
    if (p && rows > 0 && cols > 0)
      go("muon.ffn_zero", [&](bool) {
        return (int)cudaMemset2DAsync(p, (size_t)ld * es, 0, (size_t)cols * es, (size_t)rows, reinterpret_cast<cudaStream_t>(go.stream));
      });
  }
  void zero(const FfnStack& w, int64_t rows, int64_t cols) {
    if (w.se == rows * w.si || c.s.experts == 1) return zero(w.p, rows * c.s.experts, cols, w.si);
    for (int e = 0; w.p && e < c.s.experts; ++e)
      zero(static_cast<uint8_t*>(w.p) + e * w.se * element_size(c.s.dtype), rows, cols, w.si);
  }
  // A stack whose element (e, i, j) is column i of the result at depth j.
  bool stack_map(CUtensorMap* map, const FfnStack& w, int64_t n, int64_t k, bool mn, uint32_t box) {
    const int64_t inner = mn ? n : k, lines = mn ? k : n, line = mn ? w.sj : w.si;
    const int64_t ld = lines == 1 ? cdiv(inner, 8) * 8 : line, se = c.s.experts == 1 ? ld : w.se;
    return encode_operand_map(h, map, w.p, (uint64_t)inner, (uint64_t)lines, (uint64_t)c.s.experts, (uint64_t)ld * 2, (uint64_t)se * 2, 64,
                              mn ? 64 : box);
  }
  FfnTcParams tc_base() const {
    FfnTcParams p{};
    p.r = c.rows;
    p.ldf = ldf();
    p.activation = c.s.activation;
    p.status = handle_ffn_status(h);
    return p;
  }
  FfnSimtParams simt_base() const {
    FfnSimtParams p{};
    p.r = c.rows;
    p.ldf = ldf();
    p.ffn = c.s.ffn;
    p.activation = c.s.activation;
    return p;
  }

  void product(const Product& q) {
    if (go.e || bad_map) return;
    if (!tc) {
      FfnSimtParams p = simt_base();
      for (int i = 0; i < 2; ++i) {
        p.a[i] = rows_stack(q.a[i], q.lda);
        p.b[i] = q.b[i];
      }
      p.n = q.n;
      p.k = q.k;
      p.out[0] = rows_stack(q.out, q.ldo);
      p.saved = c.kept;
      p.act = q.act;
      p.dgate = q.dgate;
      p.dup = q.dup;
      if (q.what == FfnProduct::kInput && (c.dw[0].p || c.dw[1].p || c.dw[2].p)) input = p;   // with the weights'
      else go(q.range, [&](bool pdl) { return launch_ffn_simt(q.what, p, go.stream, pdl); });
      return;
    }
    FfnTcParams p = tc_base();
    // matrices of one layout: contiguous along the depth, or along the columns
    const bool mn = q.b[0].sj != 1;
    for (int i = 0; i < 2 && !bad_map; ++i) {
      if (q.a[i]) bad_map = !rows_map(&p.a[i], q.a[i], q.k, q.lda, 128) || !rows_map(&p.a_few[i], q.a[i], q.k, q.lda, 64);
      if (q.b[i].p && !bad_map) bad_map = !stack_map(&p.b[i], q.b[i], q.n, q.k, mn, q.what == FfnProduct::kGated ? 64 : 128);
    }
    if (bad_map) return;
    p.n = q.n;
    p.nt = (int32_t)cdiv(q.n, q.what == FfnProduct::kGated ? 128 : 256);
    p.nk = (int32_t)cdiv(q.k, 64);
    p.out = q.out;
    p.ldo = q.ldo;
    p.splits = 1;
    if (q.what == FfnProduct::kDown || q.what == FfnProduct::kInput) {
      p.splits = splits_of(c.s, q.what == FfnProduct::kInput);
      p.part = reinterpret_cast<float*>(c.ws + c.space.part);
      p.ldp = ld_part(q.n);
    }
    p.vec = q.out ? store_bytes(q.out, c.s.rows > 1 ? q.ldo : 0, 0) : 0;
    p.saved = c.kept;
    p.act = q.act;
    p.dgate = q.dgate;
    p.dup = q.dup;
    p.withhold_loads = handle_withholds_loads(h) && q.what == FfnProduct::kGated;
    go(q.range, [&](bool pdl) { return launch_ffn_tc(q.what, mn, p, handle_sm_count(h), go.stream, pdl); });
    if (p.splits > 1) go("muon.ffn_join", [&](bool pdl) { return launch_ffn_join(p, go.stream, pdl); });
  }

  void saved_x(bool pack, const void* x, int64_t ldx) {
    const Saved8Params p{const_cast<void*>(x), const_cast<uint8_t*>(c.x_codes), const_cast<uint8_t*>(c.x_scales), ldx, c.s.rows, c.s.hidden, false};
    const bool bf16 = c.s.dtype == MUON_BF16;
    go(pack ? "muon.pack8" : "muon.unpack8", [&](bool pdl) { return (pack ? launch_pack8 : launch_unpack8)(p, bf16, go.stream, pdl); });
  }

  // Copies of operands, and results, of widths that are not `loose`'s.
  FfnLinesParams lines{};
  void copy(const void* from, int64_t from_se, int64_t from_ld, void* to, int64_t to_se, int64_t to_ld, int64_t n, int64_t length,
            int64_t padded, int experts, bool used_only) {
    FfnLines& j = lines.job[lines.n++];
    j = FfnLines{from, to, from_se, from_ld, to_se, to_ld, lines.lines, n, (int32_t)length, (int32_t)padded, used_only};
    lines.lines += n * experts;
  }
  void copy_all(const char* range) {
    lines.r = c.rows;
    if (lines.n > 0) go(range, [&](bool pdl) { return launch_ffn_lines(lines, go.stream, pdl); });
    lines = FfnLinesParams{};
  }
  // Rows of x or dy on their way into the workspace.
  const void* rows_in(const void* p, int64_t& ld, size_t at) {
    const int64_t h8 = up8(c.s.hidden);
    copy(p, 0, ld, c.ws + at, 0, h8, c.s.rows, c.s.hidden, h8, 1, false);
    ld = h8;
    return c.ws + at;
  }
  FfnStack stack_in(const FfnStack& w, int64_t rows, int64_t cols, size_t at) {
    const bool wide = w.sj == 1;
    const int64_t lines_of = wide ? rows : cols, length = wide ? cols : rows, ld = up8(length);
    copy(w.p, w.se, wide ? w.si : w.sj, c.ws + at, lines_of * ld, ld, lines_of, length, ld, c.s.experts, true);
    return FfnStack{c.ws + at, lines_of * ld, wide ? ld : 1, wide ? 1 : ld};
  }
  // The weights' gradients that are asked for.
  struct Weight {
    const void* p;
    const void* q;
    int64_t ldp, ldq, m, n;
    int mp, mq;             // numbers of their maps
  };
  void weights(const Weight (&w)[3]) {
    if (go.e || bad_map) return;
    if (!tc) {
      FfnSimtParams p = simt_base();
      for (int i = 0; i < 3; ++i) {
        if (!c.dw[i].p) continue;
        const int j = p.jobs++;
        p.a[j] = turned(rows_stack(w[i].p, w[i].ldp));
        p.b[j] = turned(rows_stack(w[i].q, w[i].ldq));
        p.wm[j] = w[i].m;
        p.wn[j] = w[i].n;
        p.out[j] = c.dw[i];
      }
      p.beside = c.dx != nullptr;
      if (p.jobs == 0) return;
      if (p.beside && ffn_grads_in_one(input, p)) {
        go("muon.ffn_input_weight", [&](bool pdl) { return launch_ffn_grads(input, p, go.stream, pdl); });
        return;
      }
      if (p.beside) go("muon.ffn_input", [&](bool pdl) { return launch_ffn_simt(FfnProduct::kInput, input, go.stream, pdl); });
      go("muon.ffn_weight", [&](bool pdl) { return launch_ffn_simt(FfnProduct::kWeight, p, go.stream, pdl); });
      return;
    }
    FfnTcParams p = tc_base();
    p.maps = reinterpret_cast<const CUtensorMap*>(c.ws + c.space.maps);
    int tiles = 0;
    for (int i = 0; i < 3; ++i) {
      if (!c.dw[i].p) continue;
      FfnJob& j = p.job[p.jobs++];
      j.out = c.dw[i].p;
      j.se = c.dw[i].se;
      j.ld = c.dw[i].si;
      j.p = w[i].mp;
      j.q = w[i].mq;
      j.m = (int32_t)w[i].m;
      j.n = (int32_t)w[i].n;
      j.mt = (int32_t)cdiv(w[i].m, 256);
      j.nt = (int32_t)cdiv(w[i].n, 256);
      j.begin = tiles;
      j.vec = store_bytes(j.out, j.m > 1 ? j.ld : 0, c.s.experts > 1 ? j.se : 0);
      tiles += j.mt * j.nt;
    }
    p.tiles_per_expert = tiles;
    if (p.jobs > 0) go("muon.ffn_weight", [&](bool pdl) { return launch_ffn_tc(FfnProduct::kWeight, true, p, handle_sm_count(h), go.stream, pdl); });
  }
  // Tensor maps of each expert's rows, for the weights' gradients.
  void maps(const void* const (&base)[kFfnMaps], const int64_t (&ld)[kFfnMaps], const int64_t (&cols)[kFfnMaps], const bool (&used)[kFfnMaps]) {
    if (!tc || go.e) return;
    FfnMapParams p{};
    bool any = false;
    for (int i = 0; i < kFfnMaps && !bad_map; ++i) {
      p.base[i] = base[i];
      p.ld[i] = ld[i];
      p.used[i] = used[i];
      any = any || used[i];
      if (used[i]) bad_map = !rows_map(&p.whole[i], base[i], cols[i], ld[i], 64);
    }
    if (bad_map || !any) return;
    p.r = c.rows;
    p.maps = reinterpret_cast<CUtensorMap*>(c.ws + c.space.maps);
    go("muon.ffn_maps", [&](bool pdl) { return launch_ffn_maps(p, go.stream, pdl); });
  }

  muon_status done() { return bad_map ? MUON_ERR_CUDA : go.done(); }
};

// A forward pass over a few rows that keeps nothing, with weights contiguous along the depth.
bool few_rows(const Call& c) {
  const muon_ffn_shape& s = c.s;
  return on_tensor_cores(s) && s.saved_bits == 0 && s.rows <= kFfnFewRows && c.w[0].sj == 1 && c.w[2].sj == 1;
}

// Lays out the operands of widths that need it.
void lay_out(Pass& pass, Call& c) {
  if (!loose(c.s)) return;
  const int64_t H = c.s.hidden, F = c.s.ffn;
  if (c.x) c.x = pass.rows_in(c.x, c.ldx, c.space.x);
  if (c.dy) c.dy = pass.rows_in(c.dy, c.lddy, c.space.dy);
  for (int i = 0; i < 3; ++i) c.w[i] = pass.stack_in(c.w[i], i < 2 ? F : H, i < 2 ? H : F, c.space.w[i]);
  pass.copy_all("muon.ffn_lay_out");
}

muon_status run_forward(muon_handle h, Call& c, void* stream) {
  if (!c.act) c.act = c.ws + c.space.act;
  Pass pass(h, c, stream, "muon_ffn_forward");
  const int64_t H = c.s.hidden, F = c.s.ffn, ldf = pass.ldf();
  if (c.s.saved_bits == 8 && H > 0) pass.saved_x(true, c.x, c.ldx);
  if (nothing(c.s)) {
    pass.zero(c.y, c.s.rows, H, c.ldy);
    return pass.done();
  }
  lay_out(pass, c);
  if (few_rows(c)) {
    // the copies of loose widths are padded with zeros, and so is h
    const int32_t rest = (int32_t)(c.s.rows * ldf);
    FfnFewParams p{c.rows, c.x, c.ldx, {c.w[0], c.w[1]}, F, up8(H), up8(F), c.act, ldf, rest, c.s.activation};
    pass.go("muon.ffn_gated", [&](bool pdl) { return launch_ffn_few(true, p, stream, pdl); });
    FfnFewParams q{c.rows, c.act, ldf, {c.w[2], FfnStack{}}, H, up8(F), H, c.y, c.ldy, rest, c.s.activation};
    pass.go("muon.ffn_down", [&](bool pdl) { return launch_ffn_few(false, q, stream, pdl); });
    return pass.done();
  }
  Product q{FfnProduct::kGated, "muon.ffn_gated", {c.x, nullptr}, c.ldx, {c.w[0], c.w[1]}, F, H};
  q.act = c.act;
  pass.product(q);
  const bool copied = loose(c.s) && H % 8 != 0;
  void* y = copied ? c.ws + c.space.y : c.y;
  const int64_t ldy = copied ? up8(H) : c.ldy;
  pass.product({FfnProduct::kDown, "muon.ffn_down", {c.act, nullptr}, ldf, {c.w[2], FfnStack{}}, H, F, y, ldy});
  if (copied) {
    pass.copy(y, 0, ldy, c.y, 0, c.ldy, c.s.rows, H, H, 1, false);
    pass.copy_all("muon.ffn_lay_out");
  }
  return pass.done();
}

muon_status run_backward(muon_handle h, Call& c, void* stream) {
  const bool eight = c.s.saved_bits == 8;
  const int64_t H = c.s.hidden, F = c.s.ffn;
  void *dgate = c.ws + c.space.dgate, *dup = c.ws + c.space.dup;
  const bool need_x = c.dw[0].p || c.dw[1].p;
  Pass pass(h, c, stream, "muon_ffn_backward");
  if (nothing(c.s)) {
    pass.zero(c.dx, c.s.rows, H, c.lddx);
    for (int i = 0; i < 3; ++i) pass.zero(c.dw[i], i < 2 ? F : H, i < 2 ? H : F);
    return pass.done();
  }
  lay_out(pass, c);
  if (eight) {
    c.act = c.ws + c.space.act;
    c.x = c.ws + c.space.x;
    c.ldx = ld_x(H);
    if (need_x) pass.saved_x(false, c.x, c.ldx);
  }
  const int64_t ldf = pass.ldf();
  // results of loose widths come from the workspace
  void* const dx = c.dx;
  const int64_t lddx = c.lddx;
  const FfnStack dw[3] = {c.dw[0], c.dw[1], c.dw[2]};
  if (loose(c.s)) {
    const int64_t h8 = up8(H), f8 = up8(F);
    if (dx && H % 8 != 0) {
      c.dx = c.ws + c.space.y;
      c.lddx = h8;
    }
    for (int i = 0; i < 3; ++i)
      if (dw[i].p && (i < 2 ? H : F) % 8 != 0) c.dw[i] = FfnStack{c.ws + c.space.dw[i], i < 2 ? F * h8 : H * f8, i < 2 ? h8 : f8, 1};
  }
  enum { kX, kDy, kAct, kDGate, kDUp };
  const void* const base[kFfnMaps] = {c.x, c.dy, c.act, dgate, dup};
  const int64_t ld[kFfnMaps] = {c.ldx, c.lddy, ldf, ldf, ldf};
  const int64_t cols[kFfnMaps] = {H, H, F, F, F};
  const bool used[kFfnMaps] = {need_x, c.dw[2].p != nullptr, c.dw[2].p != nullptr, c.dw[0].p != nullptr, c.dw[1].p != nullptr};
  pass.maps(base, ld, cols, used);
  Product q{FfnProduct::kSlope, "muon.ffn_slope", {c.dy, nullptr}, c.lddy, {turned(c.w[2]), FfnStack{}}, F, H};
  q.act = eight ? c.act : nullptr;
  q.dgate = dgate;
  q.dup = dup;
  pass.product(q);
  if (c.dx) pass.product({FfnProduct::kInput, "muon.ffn_input", {dgate, dup}, ldf, {turned(c.w[0]), turned(c.w[1])}, H, F, c.dx, c.lddx});
  pass.weights({{dgate, c.x, ldf, c.ldx, F, H, kDGate, kX}, {dup, c.x, ldf, c.ldx, F, H, kDUp, kX}, {c.dy, c.act, c.lddy, ldf, H, F, kDy, kAct}});
  if (c.dx != dx) pass.copy(c.dx, 0, c.lddx, dx, 0, lddx, c.s.rows, H, H, 1, false);
  for (int i = 0; i < 3; ++i)
    if (c.dw[i].p != dw[i].p)   // also of experts without a token: zeros
      pass.copy(c.dw[i].p, c.dw[i].se, c.dw[i].si, dw[i].p, dw[i].se, dw[i].si, i < 2 ? F : H, i < 2 ? H : F, i < 2 ? H : F, c.s.experts, false);
  pass.copy_all("muon.ffn_lay_out");
  return pass.done();
}

}  // namespace

extern "C" {

muon_status muon_ffn_workspace_size(const muon_ffn_shape* shape, int backward, size_t* bytes) {
  if (!bytes) return MUON_ERR_INVALID_ARG;
  try {
    std::string why;
    const muon_status st = check_shape(shape, why);
    if (st == MUON_OK) *bytes = space_of(*shape, backward != 0).bytes;
    return st;
  } catch (...) {   // no memory for the text
    return MUON_ERR_INVALID_ARG;
  }
}

muon_status muon_ffn_forward(muon_handle h, const muon_ffn_shape* shape, const int32_t* offsets, const int32_t* counts,
                             const void* x, int64_t ldx, const muon_stack* gate, const muon_stack* up,
                             const muon_stack* down, void* y, int64_t ldy, const muon_ffn_saved* saved, void* ws,
                             size_t ws_bytes, void* stream) {
  return guarded(h, [&]() -> muon_status {
    std::string why;
    Call c{};
    muon_status st = check_shape(shape, why);
    if (st != MUON_OK) return fail(h, st, why);
    const muon_ffn_shape& s = c.s = *shape;
    c.rows = FfnRows{offsets, counts, (int32_t)s.rows, s.experts};
    c.x = x; c.ldx = ldx; c.y = y; c.ldy = ldy;
    std::vector<Span> spans;
    if (st == MUON_OK) st = check_route(s, offsets, counts, spans, why);
    if (st == MUON_OK) st = check_matrix(s, x, ldx, true, "x", spans, why);
    if (st == MUON_OK) st = check_matrix(s, y, ldy, false, "y", spans, why);
    if (st == MUON_OK) st = check_stack(gate, s, s.ffn, s.hidden, true, "gate", spans, c.w[0], why);
    if (st == MUON_OK) st = check_stack(up, s, s.ffn, s.hidden, true, "up", spans, c.w[1], why);
    if (st == MUON_OK) st = check_stack(down, s, s.hidden, s.ffn, true, "down", spans, c.w[2], why);
    if (st == MUON_OK && on_tensor_cores(s) && (c.w[0].sj == 1) != (c.w[1].sj == 1)) {
      why = "gate and up of bf16 must be contiguous in one direction";
      st = MUON_ERR_INVALID_ARG;
    }
    if (st == MUON_OK) st = check_saved(s, saved, true, spans, c, why);
    if (st != MUON_OK) return fail(h, st, why);
    if (s.rows == 0) return MUON_OK;
    st = check_space(h, c, false, ws, ws_bytes, spans);
    if (st != MUON_OK) return st;
    if (find_overlap(spans, why)) return fail(h, MUON_ERR_INVALID_ARG, why);
    if (handle_device(h) < 0) return fail(h, MUON_ERR_UNSUPPORTED, "host-only handle: create it with a device to run");
    DeviceGuard guard(handle_device(h));
    return run_forward(h, c, stream);
  });
}

muon_status muon_ffn_backward(muon_handle h, const muon_ffn_shape* shape, const int32_t* offsets, const int32_t* counts,
                              const void* dy, int64_t lddy, const void* x, int64_t ldx, const muon_stack* gate,
                              const muon_stack* up, const muon_stack* down, const muon_ffn_saved* saved, void* dx,
                              int64_t lddx, const muon_stack* dgate, const muon_stack* dup, const muon_stack* ddown,
                              void* ws, size_t ws_bytes, void* stream) {
  return guarded(h, [&]() -> muon_status {
    std::string why;
    Call c{};
    muon_status st = check_shape(shape, why);
    if (st != MUON_OK) return fail(h, st, why);
    const muon_ffn_shape& s = c.s = *shape;
    if (s.saved_bits == 0) return fail(h, MUON_ERR_INVALID_ARG, "shape: the backward pass needs saved_bits");
    c.rows = FfnRows{offsets, counts, (int32_t)s.rows, s.experts};
    c.dy = dy; c.lddy = lddy; c.x = x; c.ldx = ldx; c.dx = dx; c.lddx = lddx;
    std::vector<Span> spans;
    if (st == MUON_OK) st = check_route(s, offsets, counts, spans, why);
    if (st == MUON_OK) st = check_matrix(s, dy, lddy, true, "dy", spans, why);
    if (st == MUON_OK && s.saved_bits != 8) st = check_matrix(s, x, ldx, true, "x", spans, why);
    if (st == MUON_OK && s.saved_bits == 8 && x) { why = "x must be NULL when saved_bits is 8"; st = MUON_ERR_INVALID_ARG; }
    if (st == MUON_OK && dx) st = check_matrix(s, dx, lddx, false, "dx", spans, why);
    if (st == MUON_OK) st = check_stack(gate, s, s.ffn, s.hidden, true, "gate", spans, c.w[0], why);
    if (st == MUON_OK) st = check_stack(up, s, s.ffn, s.hidden, true, "up", spans, c.w[1], why);
    if (st == MUON_OK) st = check_stack(down, s, s.hidden, s.ffn, true, "down", spans, c.w[2], why);
    if (st == MUON_OK && on_tensor_cores(s) && (c.w[0].sj == 1) != (c.w[1].sj == 1)) {
      why = "gate and up of bf16 must be contiguous in one direction";
      st = MUON_ERR_INVALID_ARG;
    }
    if (st == MUON_OK) st = check_stack(dgate, s, s.ffn, s.hidden, false, "dgate", spans, c.dw[0], why);
    if (st == MUON_OK) st = check_stack(dup, s, s.ffn, s.hidden, false, "dup", spans, c.dw[1], why);
    if (st == MUON_OK) st = check_stack(ddown, s, s.hidden, s.ffn, false, "ddown", spans, c.dw[2], why);
    if (st == MUON_OK) st = check_saved(s, saved, false, spans, c, why);
    if (st != MUON_OK) return fail(h, st, why);
    if (!(c.dx && s.rows > 0 && s.hidden > 0) && !c.dw[0].p && !c.dw[1].p && !c.dw[2].p) return MUON_OK;
    st = check_space(h, c, true, ws, ws_bytes, spans);
    if (st != MUON_OK) return st;
    if (find_overlap(spans, why)) return fail(h, MUON_ERR_INVALID_ARG, why);
    if (handle_device(h) < 0) return fail(h, MUON_ERR_UNSUPPORTED, "host-only handle: create it with a device to run");
    DeviceGuard guard(handle_device(h));
    return run_backward(h, c, stream);
  });
}

}  // extern "C"
