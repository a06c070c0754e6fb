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

PyObject* bind_layers(PyObject*, PyObject* args) {
  Py_ssize_t f[5];
  if (!PyArg_ParseTuple(args, "nnnnn", f, f + 1, f + 2, f + 3, f + 4)) return nullptr;
  fn_embed = reinterpret_cast<decltype(fn_embed)>(f[0]);
  fn_embed_bytes = reinterpret_cast<decltype(fn_embed_bytes)>(f[1]);
  fn_embed_backward = reinterpret_cast<decltype(fn_embed_backward)>(f[2]);
  fn_pack8 = reinterpret_cast<decltype(fn_pack8)>(f[3]);
  fn_unpack8 = reinterpret_cast<decltype(fn_unpack8)>(f[4]);
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

// pack8(x, handle, stream): (codes, scales)
PyObject* pack8(PyObject*, PyObject* args) {
  PyObject* ox;
  Py_ssize_t handle_at, stream_at;
  if (!PyArg_ParseTuple(args, "Onn", &ox, &handle_at, &stream_at)) return nullptr;
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
      st = fn_pack8(reinterpret_cast<muon_handle>(handle_at), x.data_ptr(), ld(x), x.size(0), cols, dtype,
                    static_cast<uint8_t*>(codes.data_ptr()), static_cast<uint8_t*>(scales.data_ptr()),
                    reinterpret_cast<void*>(stream_at));
    }
    return result(st, {codes, scales});
  });
}

// unpack8(codes, scales, bf16, handle, stream): x
PyObject* unpack8(PyObject*, PyObject* args) {
  PyObject *oc, *os;
  int bf16;
  Py_ssize_t handle_at, stream_at;
  if (!PyArg_ParseTuple(args, "OOpnn", &oc, &os, &bf16, &handle_at, &stream_at)) return nullptr;
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
                      bf16 ? MUON_BF16 : MUON_F32, reinterpret_cast<void*>(stream_at));
    }
    return result(st, {x});
  });
}

PyMethodDef methods[] = {
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
