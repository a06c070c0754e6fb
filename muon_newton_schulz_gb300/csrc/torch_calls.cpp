// The torch layer's part of a call that is too slow in Python: checks of the
// call's tensors, their descriptors, the results' allocation and the library's
// call itself.  A function returns None when a check fails, and leaves it to
// the caller to say which, or the library's status when that is not MUON_OK.
// (In Python the checks take 1.6 us per parameter, here 0.1 us: a step over the
// 49 norm gains of a model was 100 us on the host and 4 us on the GPU.)
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/TracerMode.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/as_strided.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <vector>

#include "muon.h"

namespace {

constexpr int64_t kStateBlock = 256;

// The tensor that an object holds, or null.
const at::Tensor* tensor_of(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool dtype_of(const at::Tensor& t, int32_t& dtype) {
  const auto k = t.scalar_type();
  if (k != at::kFloat && k != at::kBFloat16) return false;
  dtype = k == at::kBFloat16 ? MUON_BF16 : MUON_F32;
  return true;
}

bool on(const at::Tensor& t, long index) {
  return t.layout() == at::kStrided && t.is_cuda() && t.get_device() == index;
}

// The same elements in the same order of memory.
bool alike(const at::Tensor& a, const at::Tensor& b) {
  return a.sizes() == b.sizes() && (a.strides() == b.strides() || (a.is_contiguous() && b.is_contiguous()));
}

// Lets other Python threads run for the length of a scope: allocations and
// launches can wait for the device, and that for a thread that needs the lock.
// Nothing of Python may be touched in it.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// The items of a list or tuple argument, held: another thread may change the list.
struct Items {
  PyObject* seq = nullptr;
  ~Items() { Py_XDECREF(seq); }
  bool take(PyObject* o) {
    seq = PySequence_Tuple(o);
    return seq != nullptr;
  }
  Py_ssize_t size() const { return PyTuple_GET_SIZE(seq); }
  PyObject* at(Py_ssize_t i) const { return PyTuple_GET_ITEM(seq, i); }
};

// A number for all tensors, or a list of one for each.
struct Numbers {
  PyObject* o;
  PyObject* at(Py_ssize_t i) const { return PyList_Check(o) ? PyList_GET_ITEM(o, i) : o; }
  bool fits(Py_ssize_t n) const { return !PyList_Check(o) || PyList_GET_SIZE(o) == n; }
};

// Whether torch records operations (torch.jit.trace, make_fx): a tracer would
// see a result's allocation and not the kernel that fills it.
bool traced() {
  using c10::impl::TorchDispatchModeTLS;
  return at::tracer::impl::is_dispatch_enabled() ||
         TorchDispatchModeTLS::get_mode(c10::impl::TorchDispatchModeKey::PROXY).has_value();
}

// The calls allocate and view plain results: nothing for autograd to record.
// Exceptions become the Python errors that torch's own operators raise.
template <typename F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  if (traced()) {
    PyErr_SetString(PyExc_RuntimeError, "the library's calls cannot be traced: their kernels are not torch operations");
    return nullptr;
  }
  at::AutoDispatchBelowADInplaceOrView below;
  return f();
  END_HANDLE_TH_ERRORS
}

// The library's functions, whose addresses the caller hands over: it decides
// which build of the library is loaded.
decltype(&muon_adamw_step) fn_adamw = nullptr;
decltype(&muon_clip_grads) fn_clip = nullptr;
decltype(&muon_moe_sort) fn_sort = nullptr;
decltype(&muon_moe_dispatch) fn_dispatch = nullptr;
decltype(&muon_moe_combine) fn_combine = nullptr;
decltype(&muon_moe_combine_backward) fn_backward = nullptr;

PyObject* bind(PyObject*, PyObject* args) {
  Py_ssize_t f[6];
  if (!PyArg_ParseTuple(args, "nnnnnn", f, f + 1, f + 2, f + 3, f + 4, f + 5)) return nullptr;
  fn_adamw = reinterpret_cast<decltype(fn_adamw)>(f[0]);
  fn_clip = reinterpret_cast<decltype(fn_clip)>(f[1]);
  fn_sort = reinterpret_cast<decltype(fn_sort)>(f[2]);
  fn_dispatch = reinterpret_cast<decltype(fn_dispatch)>(f[3]);
  fn_combine = reinterpret_cast<decltype(fn_combine)>(f[4]);
  fn_backward = reinterpret_cast<decltype(fn_backward)>(f[5]);
  Py_RETURN_NONE;
}

decltype(&muon_embed) fn_embed = nullptr;
decltype(&muon_embed_backward_workspace_size) fn_embed_bytes = nullptr;
decltype(&muon_embed_backward) fn_embed_backward = nullptr;
decltype(&muon_pack8) fn_pack8 = nullptr;
decltype(&muon_unpack8) fn_unpack8 = nullptr;
decltype(&muon_ffn_workspace_size) fn_ffn_bytes = nullptr;
decltype(&muon_ffn_forward) fn_ffn_forward = nullptr;
decltype(&muon_ffn_backward) fn_ffn_backward = nullptr;

PyObject* bind_layers(PyObject*, PyObject* args) {
  Py_ssize_t f[8];
  if (!PyArg_ParseTuple(args, "nnnnnnnn", f, f + 1, f + 2, f + 3, f + 4, f + 5, f + 6, f + 7)) return nullptr;
  fn_embed = reinterpret_cast<decltype(fn_embed)>(f[0]);
  fn_embed_bytes = reinterpret_cast<decltype(fn_embed_bytes)>(f[1]);
  fn_embed_backward = reinterpret_cast<decltype(fn_embed_backward)>(f[2]);
  fn_pack8 = reinterpret_cast<decltype(fn_pack8)>(f[3]);
  fn_unpack8 = reinterpret_cast<decltype(fn_unpack8)>(f[4]);
  fn_ffn_bytes = reinterpret_cast<decltype(fn_ffn_bytes)>(f[5]);
  fn_ffn_forward = reinterpret_cast<decltype(fn_ffn_forward)>(f[6]);
  fn_ffn_backward = reinterpret_cast<decltype(fn_ffn_backward)>(f[7]);
  Py_RETURN_NONE;
}

// Tells autograd that a call has written t, through its address.
void written(PyObject* o) {
  const at::Tensor* t = tensor_of(o);
  if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();   // those of inference mode have no version
}
// Whether a call that ended with st may have written anything.
bool launched(muon_status st) { return st == MUON_OK || st == MUON_ERR_CUDA; }

// What a call returns: its result, or the status when that is not MUON_OK.
PyObject* result(muon_status st, std::initializer_list<at::Tensor> out) {
  if (st != MUON_OK || out.size() == 0) return PyLong_FromLong((long)st);
  if (out.size() == 1) return THPVariable_Wrap(*out.begin());
  PyObject* t = PyTuple_New((Py_ssize_t)out.size());
  Py_ssize_t i = 0;
  for (const at::Tensor& x : out) PyTuple_SET_ITEM(t, i++, THPVariable_Wrap(x));
  return t;
}

// adamw(params, grads, ms, vs, scales, index, lr, weight_decay, step, seed,
// beta1, beta2, eps, handle, stream): the status.  scales: None, or a list of
// None and tensors.
PyObject* adamw(PyObject*, PyObject* args) {
  PyObject *op, *og, *om, *ov, *os;
  long index;
  Numbers lr, decay, step, seed;
  muon_adamw_config cfg;
  Py_ssize_t handle_at, stream_at;
  if (!PyArg_ParseTuple(args, "OOOOOlOOOOdddnn", &op, &og, &om, &ov, &os, &index, &lr.o, &decay.o, &step.o, &seed.o,
                        &cfg.beta1, &cfg.beta2, &cfg.eps, &handle_at, &stream_at))
    return nullptr;
  return guarded([&]() -> PyObject* {
    Items ps, gs, ms, vs, ss;
    if (!ps.take(op) || !gs.take(og) || !ms.take(om) || !vs.take(ov) || (os != Py_None && !ss.take(os))) return nullptr;
    const Py_ssize_t n = ps.size();
    if (gs.size() != n || ms.size() != n || vs.size() != n || (ss.seq && ss.size() != n) || !lr.fits(n) ||
        !decay.fits(n) || !step.fits(n) || !seed.fits(n))
      Py_RETURN_NONE;
    std::vector<muon_adamw_desc> d((size_t)n);
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor *p = tensor_of(ps.at(i)), *g = tensor_of(gs.at(i)), *m = tensor_of(ms.at(i)),
                       *v = tensor_of(vs.at(i));
      if (!p || !g || !m || !v) Py_RETURN_NONE;
      muon_adamw_desc& x = d[(size_t)i];
      if (!on(*p, index) || !on(*g, index) || !on(*m, index) || !on(*v, index) || !alike(*p, *g) || !alike(*p, *m) ||
          !alike(*p, *v) || !p->is_non_overlapping_and_dense() || !dtype_of(*p, x.p_dtype) || !dtype_of(*g, x.g_dtype))
        Py_RETURN_NONE;
      x.n = p->numel();
      PyObject* so = ss.seq ? ss.at(i) : Py_None;
      if (so == Py_None) {
        if (m->scalar_type() != at::kFloat || v->scalar_type() != at::kFloat) Py_RETURN_NONE;
        x.state_bits = 32;
        x.scales = nullptr;
      } else {
        const at::Tensor* s = tensor_of(so);
        if (!s || !on(*s, index) || !s->is_contiguous() || s->scalar_type() != at::kFloat8_e8m0fnu ||
            s->numel() != 2 * ((x.n + kStateBlock - 1) / kStateBlock) || m->scalar_type() != at::kFloat8_e4m3fn ||
            v->scalar_type() != at::kFloat8_e5m2)
          Py_RETURN_NONE;
        x.state_bits = 8;
        x.scales = static_cast<uint8_t*>(s->data_ptr());
      }
      x.P = p->data_ptr();
      x.G = g->data_ptr();
      x.M = m->data_ptr();
      x.V = v->data_ptr();
      x.reserved = 0;
      x.lr = PyFloat_AsDouble(lr.at(i));
      x.weight_decay = PyFloat_AsDouble(decay.at(i));
      x.step = PyLong_AsLongLong(step.at(i));
      x.seed = PyLong_AsUnsignedLongLongMask(seed.at(i)) + (PyList_Check(seed.o) ? 0u : (uint64_t)i);
      if (PyErr_Occurred()) return nullptr;
    }
    muon_status st;
    {
      Unlocked unlocked;
      st = fn_adamw(reinterpret_cast<muon_handle>(handle_at), &cfg, d.data(), (int)n, reinterpret_cast<void*>(stream_at));
    }
    for (Py_ssize_t i = 0; launched(st) && i < n; ++i) {
      for (PyObject* o : {ps.at(i), ms.at(i), vs.at(i)}) written(o);
      if (d[(size_t)i].scales) written(ss.at(i));
    }
    return result(st, {});
  });
}

// clip(grads, outs, index, max_norm, handle, stream): the norm.
PyObject* clip(PyObject*, PyObject* args) {
  PyObject *og, *oo;
  long index;
  double max_norm;
  Py_ssize_t handle_at, stream_at;
  if (!PyArg_ParseTuple(args, "OOldnn", &og, &oo, &index, &max_norm, &handle_at, &stream_at)) return nullptr;
  return guarded([&]() -> PyObject* {
    Items gs, outs;
    if (!gs.take(og) || !outs.take(oo)) return nullptr;
    const Py_ssize_t n = gs.size();
    if (outs.size() != n) Py_RETURN_NONE;
    std::vector<muon_clip_desc> d((size_t)n);
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor *g = tensor_of(gs.at(i)), *o = tensor_of(outs.at(i));
      if (!g || !o) Py_RETURN_NONE;
      muon_clip_desc& x = d[(size_t)i];
      if (!on(*g, index) || !on(*o, index) || !dtype_of(*g, x.g_dtype) || !dtype_of(*o, x.out_dtype)) Py_RETURN_NONE;
      if (alike(*g, *o) && g->is_non_overlapping_and_dense()) {
        x.rows = 1;
        x.cols = x.ldg = x.ldo = g->numel();
      } else if (g->dim() == 2 && g->sizes() == o->sizes() && (g->size(1) == 1 || (g->stride(1) == 1 && o->stride(1) == 1))) {
        x.rows = g->size(0);
        x.cols = g->size(1);
        x.ldg = g->stride(0);
        x.ldo = o->stride(0);
      } else {
        Py_RETURN_NONE;
      }
      x.G = g->data_ptr();
      x.out = o->data_ptr();
    }
    const auto options = tensor_of(gs.at(0))->options().dtype(at::kFloat);
    at::Tensor norm;   // by itself: a program may keep it
    muon_status st;
    {
      Unlocked unlocked;
      norm = at::empty({}, options);
      const at::Tensor ws = at::empty({MUON_CLIP_WORKSPACE_BYTES / 4}, options);
      st = fn_clip(reinterpret_cast<muon_handle>(handle_at), d.data(), (int)n, max_norm, static_cast<float*>(norm.data_ptr()),
                   ws.data_ptr(), MUON_CLIP_WORKSPACE_BYTES, reinterpret_cast<void*>(stream_at));
    }
    for (Py_ssize_t i = 0; std::isfinite(max_norm) && launched(st) && i < n; ++i) written(outs.at(i));
    return result(st, {norm});
  });
}

// ---- tokens by expert

// What every token operator gets: the route, the library's handle and stream.
struct Route {
  const at::Tensor *row, *offsets, *counts;
  const muon_moe_shape* shape;
  int64_t rows;
  muon_handle handle;
  void* stream;

  bool take(PyObject* row_o, PyObject* offsets_o, PyObject* counts_o, Py_ssize_t shape_at, int64_t rows_n,
            Py_ssize_t handle_at, Py_ssize_t stream_at) {
    row = tensor_of(row_o);
    offsets = tensor_of(offsets_o);
    counts = tensor_of(counts_o);
    shape = reinterpret_cast<const muon_moe_shape*>(shape_at);
    rows = rows_n;
    handle = reinterpret_cast<muon_handle>(handle_at);
    stream = reinterpret_cast<void*>(stream_at);
    if (!row || !offsets || !counts || !row->is_cuda()) return false;
    for (const at::Tensor* t : {row, offsets, counts})
      if (t->scalar_type() != at::kInt || !t->is_contiguous() || !on(*t, row->get_device())) return false;
    return row->dim() == 2 && row->size(0) == shape->tokens && row->size(1) == shape->topk &&
           counts->numel() == shape->experts && offsets->numel() == shape->experts + 1;
  }
  const int32_t* ints(const at::Tensor* t) const { return static_cast<const int32_t*>(t->data_ptr()); }
};

// A matrix of the route's device with `rows` rows.
bool matrix(PyObject* o, int64_t rows, const Route& r, at::Tensor& t, int32_t& dtype) {
  const at::Tensor* p = tensor_of(o);
  if (!p || p->dim() != 2 || p->size(0) != rows || !on(*p, r.row->get_device()) || !dtype_of(*p, dtype)) return false;
  t = *p;
  return true;
}
// Gives it unit column stride by a copy, where it has another.
void lay_out(at::Tensor& t) {
  if ((t.size(1) > 1 && t.stride(1) != 1) || (t.size(0) > 1 && t.stride(0) < t.size(1))) t = t.contiguous();
}
int64_t ld(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : std::max<int64_t>(t.size(1), 1); }

bool weights_of(PyObject* o, const Route& r, at::Tensor& w, int32_t& dtype) {
  const at::Tensor* p = tensor_of(o);
  if (!p || p->sizes() != r.row->sizes() || !on(*p, r.row->get_device()) || !dtype_of(*p, dtype)) return false;
  w = *p;
  return true;
}

// sort(ids, shape, need, handle, stream): (row, offsets, counts)
PyObject* sort(PyObject*, PyObject* args) {
  PyObject* oi;
  Py_ssize_t shape_at, need, handle_at, stream_at;
  if (!PyArg_ParseTuple(args, "Onnnn", &oi, &shape_at, &need, &handle_at, &stream_at)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor* p = tensor_of(oi);
    const auto* shape = reinterpret_cast<const muon_moe_shape*>(shape_at);
    if (!p || p->dim() != 2 || !p->is_cuda() || p->layout() != at::kStrided || p->size(0) != shape->tokens ||
        p->size(1) != shape->topk || (p->scalar_type() != at::kInt && p->scalar_type() != at::kLong))
      Py_RETURN_NONE;
    const int64_t e = shape->experts;
    at::Tensor ids = *p, row, ends;
    muon_status st;
    {
      Unlocked unlocked;
      ids = ids.contiguous();
      const auto ints = ids.options().dtype(at::kInt);
      row = at::empty({shape->tokens, shape->topk}, ints);
      ends = at::empty({2 * e + 1}, ints);
      at::Tensor ws;
      if (need > 0) ws = at::empty({(int64_t)need}, ids.options().dtype(at::kByte));
      int32_t* at_ends = static_cast<int32_t*>(ends.data_ptr());
      st = fn_sort(reinterpret_cast<muon_handle>(handle_at), shape, ids.data_ptr(), ids.scalar_type() == at::kLong ? 64 : 32,
                   static_cast<int32_t*>(row.data_ptr()), at_ends, at_ends + e + 1, need > 0 ? ws.data_ptr() : nullptr,
                   (size_t)need, reinterpret_cast<void*>(stream_at));
    }
    if (st != MUON_OK) return PyLong_FromLong((long)st);
    return result(st, {row, at::as_strided(ends, {e + 1}, {1}, 0), at::as_strided(ends, {e}, {1}, e + 1)});
  });
}

// dispatch(x, row, offsets, counts, shape, rows, handle, stream): xs
PyObject* dispatch(PyObject*, PyObject* args) {
  PyObject *ox, *a, *b, *c;
  Py_ssize_t shape_at, rows, handle_at, stream_at;
  if (!PyArg_ParseTuple(args, "OOOOnnnn", &ox, &a, &b, &c, &shape_at, &rows, &handle_at, &stream_at)) return nullptr;
  return guarded([&]() -> PyObject* {
    Route r;
    at::Tensor x;
    int32_t dtype;
    if (!r.take(a, b, c, shape_at, rows, handle_at, stream_at) || !matrix(ox, r.shape->tokens, r, x, dtype)) Py_RETURN_NONE;
    const int64_t h = x.size(1);
    at::Tensor xs;
    muon_status st;
    {
      Unlocked unlocked;
      lay_out(x);
      xs = at::empty({r.rows, h}, x.options());
      st = fn_dispatch(r.handle, r.shape, r.ints(r.row), r.ints(r.offsets), r.ints(r.counts), x.data_ptr(), ld(x),
                       xs.data_ptr(), std::max<int64_t>(h, 1), h, dtype, r.stream);
    }
    return result(st, {xs});
  });
}

// combine(y, weights or None, row, offsets, counts, shape, rows, handle, stream): out
PyObject* combine(PyObject*, PyObject* args) {
  PyObject *oy, *ow, *a, *b, *c;
  Py_ssize_t shape_at, rows, handle_at, stream_at;
  if (!PyArg_ParseTuple(args, "OOOOOnnnn", &oy, &ow, &a, &b, &c, &shape_at, &rows, &handle_at, &stream_at)) return nullptr;
  return guarded([&]() -> PyObject* {
    Route r;
    at::Tensor y, w;
    int32_t dtype, w_dtype = MUON_F32;
    if (!r.take(a, b, c, shape_at, rows, handle_at, stream_at) || !matrix(oy, r.rows, r, y, dtype) ||
        (ow != Py_None && !weights_of(ow, r, w, w_dtype)))
      Py_RETURN_NONE;
    const int64_t h = y.size(1);
    at::Tensor out;
    muon_status st;
    {
      Unlocked unlocked;
      lay_out(y);
      if (w.defined()) w = w.contiguous();
      out = at::empty({r.shape->tokens, h}, y.options());
      st = fn_combine(r.handle, r.shape, r.ints(r.row), y.data_ptr(), ld(y), w.defined() ? w.data_ptr() : nullptr, w_dtype,
                      out.data_ptr(), std::max<int64_t>(h, 1), h, dtype, r.stream);
    }
    return result(st, {out});
  });
}

// combine_backward(dout, y, weights, row, offsets, counts, shape, rows, handle, stream): (dy, dweights)
PyObject* combine_backward(PyObject*, PyObject* args) {
  PyObject *od, *oy, *ow, *a, *b, *c;
  Py_ssize_t shape_at, rows, handle_at, stream_at;
  if (!PyArg_ParseTuple(args, "OOOOOOnnnn", &od, &oy, &ow, &a, &b, &c, &shape_at, &rows, &handle_at, &stream_at))
    return nullptr;
  return guarded([&]() -> PyObject* {
    Route r;
    at::Tensor d, y, w;
    int32_t d_dtype, dtype, w_dtype;
    if (!r.take(a, b, c, shape_at, rows, handle_at, stream_at) || !matrix(od, r.shape->tokens, r, d, d_dtype) ||
        !matrix(oy, r.rows, r, y, dtype) || d_dtype != dtype || d.size(1) != y.size(1) || !weights_of(ow, r, w, w_dtype))
      Py_RETURN_NONE;
    const int64_t h = y.size(1);
    at::Tensor dy, dw;
    muon_status st;
    {
      Unlocked unlocked;
      lay_out(d);
      lay_out(y);
      w = w.contiguous();
      dy = at::empty({r.rows, h}, y.options());
      dw = at::empty(w.sizes(), w.options());
      st = fn_backward(r.handle, r.shape, r.ints(r.row), r.ints(r.offsets), r.ints(r.counts), d.data_ptr(), ld(d),
                       y.data_ptr(), ld(y), w.data_ptr(), w_dtype, dy.data_ptr(), std::max<int64_t>(h, 1), dw.data_ptr(), h,
                       dtype, r.stream);
    }
    return result(st, {dy, dw});
  });
}

// ---- embedding

// Ids of any shape on a device, their shape followed by `more` in `shape`.
bool ids_of(PyObject* o, at::Tensor& ids, std::vector<int64_t>& shape) {
  const at::Tensor* p = tensor_of(o);
  if (!p || !p->is_cuda() || p->layout() != at::kStrided || (p->scalar_type() != at::kInt && p->scalar_type() != at::kLong))
    return false;
  ids = *p;
  shape.assign(p->sizes().begin(), p->sizes().end());
  return true;
}
int bits_of(const at::Tensor& ids) { return ids.scalar_type() == at::kLong ? 64 : 32; }

// embed(ids, table, scale, handle, stream): out
PyObject* embed(PyObject*, PyObject* args) {
  PyObject *oi, *ot;
  double scale;
  Py_ssize_t handle_at, stream_at;
  if (!PyArg_ParseTuple(args, "OOdnn", &oi, &ot, &scale, &handle_at, &stream_at)) return nullptr;
  return guarded([&]() -> PyObject* {
    at::Tensor ids, table, out;
    std::vector<int64_t> shape;
    const at::Tensor* pt = tensor_of(ot);
    int32_t dtype;
    if (!ids_of(oi, ids, shape) || !pt || pt->dim() != 2 || !on(*pt, ids.get_device()) || !dtype_of(*pt, dtype)) Py_RETURN_NONE;
    muon_status st;
    {
      Unlocked unlocked;
      table = *pt;
      lay_out(table);
      ids = ids.contiguous();
      const int64_t h = table.size(1);
      shape.push_back(h);
      out = at::empty(shape, table.options());
      st = fn_embed(reinterpret_cast<muon_handle>(handle_at), ids.data_ptr(), bits_of(ids), ids.numel(), table.data_ptr(),
                    ld(table), table.size(0), h, dtype, scale, out.data_ptr(), std::max<int64_t>(h, 1),
                    reinterpret_cast<void*>(stream_at));
    }
    return result(st, {out});
  });
}

// embed_backward(dout, ids, vocab, scale, handle, stream): dtable
PyObject* embed_backward(PyObject*, PyObject* args) {
  PyObject *od, *oi;
  long long vocab;
  double scale;
  Py_ssize_t handle_at, stream_at;
  if (!PyArg_ParseTuple(args, "OOLdnn", &od, &oi, &vocab, &scale, &handle_at, &stream_at)) return nullptr;
  return guarded([&]() -> PyObject* {
    at::Tensor ids, dout, dtable, ws;
    std::vector<int64_t> shape;
    const at::Tensor* pd = tensor_of(od);
    int32_t dtype;
    if (!ids_of(oi, ids, shape) || !pd || pd->dim() != (int64_t)shape.size() + 1 || !on(*pd, ids.get_device()) ||
        !dtype_of(*pd, dtype) || !std::equal(shape.begin(), shape.end(), pd->sizes().begin()) || vocab < 0)
      Py_RETURN_NONE;
    muon_status st;
    {
      Unlocked unlocked;
      ids = ids.contiguous();
      const int64_t n = ids.numel(), h = pd->size(pd->dim() - 1);
      dout = pd->dim() == 2 ? *pd : pd->reshape({n, h});
      lay_out(dout);
      size_t need = 0;
      st = fn_embed_bytes(n, vocab, h, &need);
      if (st == MUON_OK) {
        dtable = at::empty({(int64_t)vocab, h}, dout.options());
        ws = at::empty({(int64_t)need}, dout.options().dtype(at::kByte));
        st = fn_embed_backward(reinterpret_cast<muon_handle>(handle_at), ids.data_ptr(), bits_of(ids), n, dout.data_ptr(), ld(dout),
                               vocab, h, dtype, scale, dtable.data_ptr(), std::max<int64_t>(h, 1), ws.data_ptr(), need,
                               reinterpret_cast<void*>(stream_at));
      }
    }
    return result(st, {dtable});
  });
}

// ---- activations in 8 bits

constexpr int64_t kSavedBlock = 32;

// pack8(x, handle, stream, special = False): (codes, scales)
PyObject* pack8(PyObject*, PyObject* args) {
  PyObject* ox;
  Py_ssize_t handle_at, stream_at;
  int special = 0;
  if (!PyArg_ParseTuple(args, "Onn|p", &ox, &handle_at, &stream_at, &special)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor* p = tensor_of(ox);
    int32_t dtype;
    if (!p || p->dim() < 1 || !p->is_cuda() || p->layout() != at::kStrided || !dtype_of(*p, dtype)) Py_RETURN_NONE;
    at::Tensor x = *p, codes, scales;
    muon_status st;
    {
      Unlocked unlocked;
      const int64_t cols = x.size(-1);
      std::vector<int64_t> shape(x.sizes().begin(), x.sizes().end());
      codes = at::empty(shape, x.options().dtype(at::kFloat8_e4m3fn));
      shape.back() = (cols + kSavedBlock - 1) / kSavedBlock;
      scales = at::empty(shape, x.options().dtype(at::kFloat8_e8m0fnu));
      if (x.dim() != 2) x = x.contiguous().reshape({cols ? x.numel() / cols : 0, cols});
      lay_out(x);
      st = fn_pack8(reinterpret_cast<muon_handle>(handle_at), x.data_ptr(), ld(x), x.size(0), cols,
                    dtype | (special ? MUON_SAVED8_SPECIAL : 0),
                    static_cast<uint8_t*>(codes.data_ptr()), static_cast<uint8_t*>(scales.data_ptr()),
                    reinterpret_cast<void*>(stream_at));
    }
    return result(st, {codes, scales});
  });
}

// unpack8(codes, scales, bf16, handle, stream, special = False): x
PyObject* unpack8(PyObject*, PyObject* args) {
  PyObject *oc, *os;
  int bf16, special = 0;
  Py_ssize_t handle_at, stream_at;
  if (!PyArg_ParseTuple(args, "OOpnn|p", &oc, &os, &bf16, &handle_at, &stream_at, &special)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor *c = tensor_of(oc), *s = tensor_of(os);
    if (!c || !s || c->dim() < 1 || !c->is_cuda() || !on(*c, c->get_device()) || !on(*s, c->get_device()) ||
        c->scalar_type() != at::kFloat8_e4m3fn || s->scalar_type() != at::kFloat8_e8m0fnu || !c->is_contiguous() ||
        !s->is_contiguous())
      Py_RETURN_NONE;
    const int64_t cols = c->size(-1), rows = cols ? c->numel() / cols : 0;
    std::vector<int64_t> shape(c->sizes().begin(), c->sizes().end());
    shape.back() = (cols + kSavedBlock - 1) / kSavedBlock;
    if (s->sizes() != at::IntArrayRef(shape)) Py_RETURN_NONE;
    at::Tensor x;
    muon_status st;
    {
      Unlocked unlocked;
      x = at::empty(c->sizes(), c->options().dtype(bf16 ? at::kBFloat16 : at::kFloat));
      st = fn_unpack8(reinterpret_cast<muon_handle>(handle_at), static_cast<const uint8_t*>(c->data_ptr()),
                      static_cast<const uint8_t*>(s->data_ptr()), rows, cols, x.data_ptr(), std::max<int64_t>(cols, 1),
                      (bf16 ? MUON_BF16 : MUON_F32) | (special ? MUON_SAVED8_SPECIAL : 0), reinterpret_cast<void*>(stream_at));
    }
    return result(st, {x});
  });
}

// ---- gated feed-forward block

// Whether a 16-byte boundary begins every line of bf16 (fp32 needs none).
bool on_lines(const at::Tensor& t, int64_t line_stride, int64_t more_stride) {
  return t.element_size() == 4 || (reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0 && line_stride % 8 == 0 && more_stride % 8 == 0);
}
// A copy whose rows of the last dimension begin on 16-byte boundaries.
at::Tensor spread(const at::Tensor& t) {
  std::vector<int64_t> shape(t.sizes().begin(), t.sizes().end());
  const int64_t cols = shape.back();
  shape.back() = (cols + 7) / 8 * 8;
  at::Tensor to = at::empty(shape, t.options()).narrow(-1, 0, cols);
  to.copy_(t);
  return to;
}
void lay_out_rows(at::Tensor& t, bool on_boundaries) {
  lay_out(t);
  if (on_boundaries && t.numel() > 0 && !on_lines(t, t.size(0) > 1 ? t.stride(0) : 0, 0)) t = spread(t);
}

// A stack of matrices, experts x rows x cols, or rows x cols of the one expert
// there is without a route.
struct Stack {
  at::Tensor t;
  muon_stack m;
  bool take(PyObject* o, int64_t experts, int64_t rows, int64_t cols, bool routed, long index, at::ScalarType kind) {
    const at::Tensor* p = tensor_of(o);
    if (!p || p->dim() != (routed ? 3 : 2) || !on(*p, index) || p->scalar_type() != kind || p->size(-2) != rows ||
        p->size(-1) != cols || (routed && p->size(0) != experts))
      return false;
    t = *p;
    return true;
  }
  void lay_out(bool on_boundaries) {
    const bool many = t.dim() == 3 && t.size(0) > 1;
    const int64_t rows = t.size(-2), cols = t.size(-1);
    if (t.numel() > 0) {
      int64_t si = rows > 1 ? t.stride(-2) : cols, sj = cols > 1 ? t.stride(-1) : 1;
      if (sj != 1 && rows == 1) si = 1;
      const bool lines = (sj == 1 && si >= cols) || (si == 1 && sj >= rows);
      const int64_t extent = sj == 1 ? (rows - 1) * si + cols : (cols - 1) * sj + rows;
      if (!lines || (many && t.stride(0) < extent) ||
          (on_boundaries && !on_lines(t, sj != 1 ? sj : rows > 1 ? si : 0, many ? t.stride(0) : 0)))
        t = spread(t);
    }
    m.p = t.data_ptr();
    m.stride[0] = t.dim() == 3 ? t.stride(0) : 0;
    m.stride[1] = rows > 1 ? t.stride(-2) : std::max<int64_t>(cols, 1);
    m.stride[2] = cols > 1 ? t.stride(-1) : 1;
    if (m.stride[2] != 1 && rows == 1) m.stride[1] = 1;
  }
  void make(int64_t experts, int64_t rows, int64_t cols, bool routed, const at::TensorOptions& options) {
    t = routed ? at::empty({experts, rows, cols}, options) : at::empty({rows, cols}, options);
    m = muon_stack{t.data_ptr(), {rows * cols, cols, 1}};
  }
};

// The inputs that the forward and the backward pass share.
struct Ffn {
  muon_ffn_shape shape{};
  const int32_t *offsets = nullptr, *counts = nullptr;
  bool routed = false;
  long index = -1;
  at::ScalarType kind;
  Stack gate, up, down;
  int64_t ld = 0;

  // rows: x or dy
  bool take(PyObject* orows, PyObject* og, PyObject* ou, PyObject* od, PyObject* oo, PyObject* oc, int activation, int saved_bits,
            at::Tensor& rows) {
    const at::Tensor *p = tensor_of(orows), *g = tensor_of(og);
    if (!p || p->dim() != 2 || !p->is_cuda() || !on(*p, p->get_device()) || !dtype_of(*p, shape.dtype) || !g || g->dim() < 2) return false;
    rows = *p;
    index = p->get_device();
    kind = p->scalar_type();
    routed = oo != Py_None;
    shape.rows = p->size(0);
    shape.hidden = p->size(1);
    shape.ffn = g->size(-2);
    shape.experts = 1;
    shape.activation = activation;
    shape.saved_bits = saved_bits;
    if (routed) {
      const at::Tensor *o = tensor_of(oo), *c = tensor_of(oc);
      if (!o || !c) return false;
      for (const at::Tensor* t : {o, c})
        if (t->scalar_type() != at::kInt || !t->is_contiguous() || !on(*t, index)) return false;
      if (o->numel() != c->numel() + 1 || c->numel() < 1 || c->numel() > 1 << 20) return false;
      shape.experts = (int32_t)c->numel();
      offsets = static_cast<const int32_t*>(o->data_ptr());
      counts = static_cast<const int32_t*>(c->data_ptr());
    }
    ld = (shape.ffn + 127) / 128 * 128;
    return gate.take(og, shape.experts, shape.ffn, shape.hidden, routed, index, kind) &&
           up.take(ou, shape.experts, shape.ffn, shape.hidden, routed, index, kind) &&
           down.take(od, shape.experts, shape.hidden, shape.ffn, routed, index, kind);
  }
  void lay_out() {
    gate.lay_out(on_boundaries());
    up.lay_out(on_boundaries());
    down.lay_out(on_boundaries());
    if ((gate.m.stride[2] == 1) != (up.m.stride[2] == 1)) {   // both the same way
      gate.t = spread(gate.t);
      up.t = spread(up.t);
      gate.lay_out(on_boundaries());
      up.lay_out(on_boundaries());
    }
  }
  // Whether the library takes rows on 16-byte boundaries alone; others it copies itself.
  bool on_boundaries() const { return shape.hidden % 8 == 0 && shape.ffn % 8 == 0; }
};

// What is kept: pre (2 x rows x ld: g and u) and act (rows x ld) in 32 bits; pre, its
// scale bytes and act in 16; pre, its scale bytes and x in 8.
struct Kept {
  at::Tensor pre, act, scales, x_codes, x_scales;
  muon_ffn_saved s{};
  // The tensors, in the order in which they are handed over.
  std::vector<at::Tensor*> parts(int bits) {
    if (bits == 8) return {&pre, &scales, &x_codes, &x_scales};
    if (bits == 16) return {&pre, &scales, &act};
    return {&pre, &act};
  }
  static at::ScalarType kind_of(int bits, size_t i) {
    if (bits == 8) return i % 2 ? at::kFloat8_e8m0fnu : at::kFloat8_e4m3fn;
    if (bits == 16) return i == 0 ? at::kHalf : i == 1 ? at::kFloat8_e8m0fnu : at::kBFloat16;
    return at::kFloat;
  }
  static std::vector<int64_t> shape_of(int bits, size_t i, const Ffn& f) {
    const int64_t rows = f.shape.rows, h = f.shape.hidden;
    if (i == 0) return {2, rows, f.ld};
    if (bits != 32 && i == 1) return {2, rows, f.ld / kSavedBlock};
    if (bits != 8) return {rows, f.ld};
    return {rows, i == 2 ? h : (h + kSavedBlock - 1) / kSavedBlock};
  }
  void fill(const Ffn& f) {
    const int64_t n = f.shape.rows * f.ld;
    const int bits = f.shape.saved_bits;
    uint8_t* p = static_cast<uint8_t*>(pre.data_ptr());
    s.gate = p;
    s.up = p ? p + n * pre.element_size() : nullptr;
    if (bits != 8) s.act = act.data_ptr();
    if (bits != 32) {
      s.gate_scales = static_cast<uint8_t*>(scales.data_ptr());
      s.up_scales = s.gate_scales ? s.gate_scales + n / kSavedBlock : nullptr;
    }
    if (bits == 8) {
      s.x_codes = static_cast<uint8_t*>(x_codes.data_ptr());
      s.x_scales = static_cast<uint8_t*>(x_scales.data_ptr());
    }
  }
};

// ffn_forward(x, gate, up, down, offsets, counts, activation, saved_bits, handle, stream): y, or y and what is
// kept
PyObject* ffn_forward(PyObject*, PyObject* args) {
  PyObject *ox, *og, *ou, *od, *oo, *oc;
  int activation, saved_bits;
  Py_ssize_t handle_at, stream_at;
  if (!PyArg_ParseTuple(args, "OOOOOOiinn", &ox, &og, &ou, &od, &oo, &oc, &activation, &saved_bits, &handle_at, &stream_at))
    return nullptr;
  return guarded([&]() -> PyObject* {
    Ffn f;
    at::Tensor x, y, ws;
    if (!f.take(ox, og, ou, od, oo, oc, activation, saved_bits, x)) Py_RETURN_NONE;
    Kept k;
    muon_status st;
    {
      Unlocked unlocked;
      const auto options = x.options();
      const int64_t rows = f.shape.rows, h = f.shape.hidden;
      lay_out_rows(x, f.on_boundaries());
      f.lay_out();
      y = at::empty({rows, h}, options);
      if (saved_bits != 0) {
        const auto parts = k.parts(saved_bits);
        for (size_t i = 0; i < parts.size(); ++i)
          *parts[i] = at::empty(Kept::shape_of(saved_bits, i, f), options.dtype(Kept::kind_of(saved_bits, i)));
      }
      if (saved_bits != 0) k.fill(f);
      size_t need = 0;
      st = fn_ffn_bytes(&f.shape, 0, &need);
      if (st == MUON_OK) {
        ws = at::empty({(int64_t)need}, options.dtype(at::kByte));
        st = fn_ffn_forward(reinterpret_cast<muon_handle>(handle_at), &f.shape, f.offsets, f.counts, x.data_ptr(), ld(x), &f.gate.m,
                            &f.up.m, &f.down.m, y.data_ptr(), std::max<int64_t>(h, 1), saved_bits ? &k.s : nullptr, ws.data_ptr(),
                            need, reinterpret_cast<void*>(stream_at));
      }
    }
    if (saved_bits == 0) return result(st, {y});
    if (saved_bits == 8) return result(st, {y, k.pre, k.scales, k.x_codes, k.x_scales});
    if (saved_bits == 16) return result(st, {y, k.pre, k.scales, k.act});
    return result(st, {y, k.pre, k.act});
  });
}

// ffn_backward(dy, x or None, gate, up, down, offsets, counts, kept, activation, saved_bits, want, handle, stream): dx,
// dgate, dup, ddown, each None where its bit of `want` is not set.  kept: what ffn_forward returned behind y.
PyObject* ffn_backward(PyObject*, PyObject* args) {
  PyObject *ody, *ox, *og, *ou, *od, *oo, *oc, *ok;
  int activation, saved_bits, want;
  Py_ssize_t handle_at, stream_at;
  if (!PyArg_ParseTuple(args, "OOOOOOOOiiinn", &ody, &ox, &og, &ou, &od, &oo, &oc, &ok, &activation, &saved_bits, &want, &handle_at,
                        &stream_at))
    return nullptr;
  return guarded([&]() -> PyObject* {
    Ffn f;
    Kept k;
    Items kept;
    at::Tensor dy, x, dx, ws;
    Stack dw[3];
    const bool eight = saved_bits == 8;
    if (!kept.take(ok)) return nullptr;
    if (saved_bits != 8 && saved_bits != 16 && saved_bits != 32) Py_RETURN_NONE;
    const auto parts = k.parts(saved_bits);
    if (!f.take(ody, og, ou, od, oo, oc, activation, saved_bits, dy) || kept.size() != (Py_ssize_t)parts.size()) Py_RETURN_NONE;
    const int64_t rows = f.shape.rows, h = f.shape.hidden;
    for (size_t i = 0; i < parts.size(); ++i) {
      const at::Tensor* p = tensor_of(kept.at((Py_ssize_t)i));
      if (!p || !on(*p, f.index) || !p->is_contiguous() || p->scalar_type() != Kept::kind_of(saved_bits, i) ||
          p->sizes() != at::IntArrayRef(Kept::shape_of(saved_bits, i, f)))
        Py_RETURN_NONE;
      *parts[i] = *p;
    }
    if (!eight) {
      const at::Tensor* p = tensor_of(ox);
      if (!p || p->sizes() != dy.sizes() || !on(*p, f.index) || p->scalar_type() != f.kind) Py_RETURN_NONE;
      x = *p;
    }
    muon_status st;
    {
      Unlocked unlocked;
      const auto options = dy.options();
      lay_out_rows(dy, f.on_boundaries());
      if (!eight) lay_out_rows(x, f.on_boundaries());
      f.lay_out();
      k.fill(f);
      if (want & 1) dx = at::empty({rows, h}, options);
      for (int i = 0; i < 3; ++i) {
        dw[i].m = muon_stack{};
        if (want & (2 << i)) dw[i].make(f.shape.experts, i < 2 ? f.shape.ffn : h, i < 2 ? h : f.shape.ffn, f.routed, options);
      }
      size_t need = 0;
      st = fn_ffn_bytes(&f.shape, 1, &need);
      if (st == MUON_OK) {
        ws = at::empty({(int64_t)need}, options.dtype(at::kByte));
        st = fn_ffn_backward(reinterpret_cast<muon_handle>(handle_at), &f.shape, f.offsets, f.counts, dy.data_ptr(), ld(dy),
                             eight ? nullptr : x.data_ptr(), eight ? 0 : ld(x), &f.gate.m, &f.up.m, &f.down.m, &k.s,
                             want & 1 ? dx.data_ptr() : nullptr, std::max<int64_t>(h, 1), &dw[0].m, &dw[1].m, &dw[2].m,
                             ws.data_ptr(), need, reinterpret_cast<void*>(stream_at));
      }
    }
    if (st != MUON_OK) return PyLong_FromLong((long)st);
    const at::Tensor out[4] = {dx, dw[0].t, dw[1].t, dw[2].t};
    PyObject* t = PyTuple_New(4);
    for (Py_ssize_t i = 0; i < 4; ++i) {
      if (want & (1 << i)) {
        PyTuple_SET_ITEM(t, i, THPVariable_Wrap(out[i]));
      } else {
        Py_INCREF(Py_None);
        PyTuple_SET_ITEM(t, i, Py_None);
      }
    }
    return t;
  });
}

PyMethodDef methods[] = {
    {"ffn_forward", ffn_forward, METH_VARARGS, "muon_ffn_forward into new tensors."},
    {"ffn_backward", ffn_backward, METH_VARARGS, "muon_ffn_backward into new tensors."},
    {"bind", bind, METH_VARARGS, "Takes the addresses of the library's functions."},
    {"bind_layers", bind_layers, METH_VARARGS, "Takes the addresses of the library's functions for a model's layers."},
    {"embed", embed, METH_VARARGS, "muon_embed into a new tensor."},
    {"embed_backward", embed_backward, METH_VARARGS, "muon_embed_backward into a new tensor."},
    {"pack8", pack8, METH_VARARGS, "muon_pack8 into new tensors."},
    {"unpack8", unpack8, METH_VARARGS, "muon_unpack8 into a new tensor."},
    {"sort", sort, METH_VARARGS, "muon_moe_sort on new tensors."},
    {"dispatch", dispatch, METH_VARARGS, "muon_moe_dispatch into a new tensor."},
    {"combine", combine, METH_VARARGS, "muon_moe_combine into a new tensor."},
    {"combine_backward", combine_backward, METH_VARARGS, "muon_moe_combine_backward into new tensors."},
    {"adamw", adamw, METH_VARARGS, "muon_adamw_step on lists of tensors."},
    {"clip", clip, METH_VARARGS, "muon_clip_grads on lists of tensors."},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
