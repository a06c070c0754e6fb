// What the C entries around the Muon step share: checks of addresses, sizes
// and overlaps, errors, and how a call's first launch may start.
#pragma once

#include "muon.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <limits>
#include <new>
#include <string>
#include <utility>
#include <vector>

#include "muon_internal.h"

namespace muon {

constexpr int64_t kMaxElements = 1ll << 40;
constexpr int64_t kInt32Max = std::numeric_limits<int32_t>::max();
constexpr int kSms = 152;   // of the one device this library is built for

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t element_size(int dtype) { return dtype == MUON_BF16 ? 2 : 4; }
inline bool known_dtype(int dtype) { return dtype == MUON_F32 || dtype == MUON_BF16; }
inline bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

inline muon_status fail(muon_handle h, muon_status s, const std::string& why) {
  set_handle_error(h, why);
  return s;
}

inline muon_status cuda_fail(muon_handle h, const char* what, int e) {
  cudaGetLastError();   // the status says it: whoever asks CUDA next is not told again
  return fail(h, MUON_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString((cudaError_t)e));
}

// Bytes that a call reads or writes: [lo, hi), or rows of `width` bytes in it
// that are `pitch` bytes apart.
struct Span {
  uintptr_t lo, hi;
  uintptr_t pitch, width;
  int32_t desc;
  bool written;
  const char* what;
};

inline Span span(const void* p, int64_t bytes, int desc, bool written, const char* what) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + (uintptr_t)bytes, 0, 0, desc, written, what};
}

inline Span matrix_span(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t es, int desc, bool written,
                 const char* what) {
  Span s = span(p, rows == 0 || cols == 0 ? 0 : ((rows - 1) * ld + cols) * es, desc, written, what);
  if (rows > 1 && ld > cols) {
    s.pitch = (uintptr_t)(ld * es);
    s.width = (uintptr_t)(cols * es);
  }
  return s;
}

inline std::string named(const Span& s) {
  return s.desc < 0 ? std::string(s.what) : "desc " + std::to_string(s.desc) + " " + s.what;
}

// Whether two spans share a byte, a starting no later than b and ending behind
// b's start.  Matrices that are column ranges of one buffer do not, nor does
// what lies between two rows.
inline bool share(const Span& a, const Span& b) {
  if (a.pitch == 0 || (b.pitch != 0 && a.pitch != b.pitch)) return true;
  const uintptr_t at = (b.lo - a.lo) % a.pitch;
  const uintptr_t bytes = b.pitch ? b.width : std::min(a.hi, b.hi) - b.lo;
  return at < a.width || at + bytes > a.pitch;
}

// A written span may share no byte with any other.
inline bool find_overlap(const std::vector<Span>& v, std::string& why) {
  std::vector<std::pair<uintptr_t, const Span*>> order;   // by address
  order.reserve(v.size());
  for (const Span& s : v)
    if (s.lo != s.hi) order.emplace_back(s.lo, &s);
  std::sort(order.begin(), order.end(), [](const auto& a, const auto& b) { return a.first < b.first; });
  std::vector<const Span*> open;   // earlier spans that may reach further
  for (const auto& at : order) {
    const Span& s = *at.second;
    size_t kept = 0;
    for (const Span* o : open) {
      if (o->hi <= s.lo) continue;
      open[kept++] = o;
      if ((o->written || s.written) && share(*o, s)) {
        why = "buffers overlap: " + named(*o) + " and " + named(s);
        return true;
      }
    }
    open.resize(kept);
    open.push_back(&s);
  }
  return false;
}

// Runs f, turning a failed host allocation into a status: no exception leaves
// a C entry.
template <typename F>
inline muon_status guarded(muon_handle h, F f) {
  if (!h) return MUON_ERR_INVALID_ARG;
  try {
    set_handle_error(h, "");
    return f();
  } catch (const std::bad_alloc&) {
    return MUON_ERR_CUDA;
  } catch (...) {
    return MUON_ERR_CUDA;
  }
}

// Whether a call's first launch may be a programmatic dependent of whatever
// the stream holds before it.  Every kernel here waits for its predecessor
// before it touches global memory, so only the launch itself overlaps.  Not
// while the stream is being captured: the node before may be of any kind.
inline bool first_pdl(void* stream) {
  cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(reinterpret_cast<cudaStream_t>(stream), &st) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return kUsePdl && st == cudaStreamCaptureStatusNone;
}

// A matrix argument of a row operator.
struct Mat {
  const void* p;
  int64_t rows, ld;
  bool written;
  const char* name;
};

// Also finds the bytes that a thread can move at once: 16, 4 or one element.
inline muon_status check_rows(int64_t hidden, int dtype, const Mat* mats, int nm, std::vector<Span>& spans, int& bytes,
                       std::string& why) {
  if (hidden < 0 || hidden > kMaxElements) { why = "hidden must be in [0, 2^40]"; return MUON_ERR_INVALID_ARG; }
  if (!known_dtype(dtype)) { why = "dtype must be MUON_F32 or MUON_BF16"; return MUON_ERR_INVALID_ARG; }
  const int64_t es = element_size(dtype);
  auto multiple = [&](int64_t n) { return hidden * es % n == 0; };
  bytes = multiple(16) ? 16 : multiple(4) ? 4 : 2;
  for (int i = 0; i < nm; ++i) {
    const Mat& m = mats[i];
    if (m.rows == 0 || hidden == 0) continue;
    if (!m.p) { why = std::string(m.name) + " must be non-NULL"; return MUON_ERR_INVALID_ARG; }
    if (!aligned(m.p, es)) { why = std::string(m.name) + " must be aligned to its element size"; return MUON_ERR_INVALID_ARG; }
    if (m.ld < hidden) { why = std::string("ld of ") + m.name + " must be >= hidden"; return MUON_ERR_INVALID_ARG; }
    if (m.ld > kMaxElements / m.rows) {
      why = std::string("rows of ") + m.name + " times its ld must be at most 2^40";
      return MUON_ERR_INVALID_ARG;
    }
    const int at = aligned(m.p, 16) && m.ld * es % 16 == 0 ? 16 : aligned(m.p, 4) && m.ld * es % 4 == 0 ? 4 : 2;
    bytes = std::min(bytes, at);
    spans.push_back(matrix_span(m.p, m.rows, hidden, m.ld, es, -1, m.written, m.name));
  }
  return find_overlap(spans, why) ? MUON_ERR_INVALID_ARG : MUON_OK;
}

}  // namespace muon
