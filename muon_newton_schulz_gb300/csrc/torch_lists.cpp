// Descriptors of lists of torch tensors, for the torch layer of AdamW and
// gradient clipping: checks a call's tensors and writes muon_adamw_desc or
// muon_clip_desc arrays.  The checks are the torch layer's; each function
// returns None when one fails and leaves it to the caller to say which.  (In
// Python the same checks take 1.6 us per parameter, here 0.1 us: a step over
// the 49 norm gains of a model was 100 us on the host and 4 us on the GPU.)
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <exception>
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

// A list or tuple argument, its items borrowed.
struct Items {
  PyObject* seq = nullptr;
  ~Items() { Py_XDECREF(seq); }
  bool take(PyObject* o) {
    seq = PySequence_Fast(o, "a list of tensors is expected");
    return seq != nullptr;
  }
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
  PyObject* at(Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
};

// A number for all tensors, or a list of one for each.
struct Numbers {
  PyObject* o;
  PyObject* at(Py_ssize_t i) const { return PyList_Check(o) ? PyList_GET_ITEM(o, i) : o; }
  bool fits(Py_ssize_t n) const { return !PyList_Check(o) || PyList_GET_SIZE(o) == n; }
};

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// adamw(params, grads, ms, vs, scales, index, lr, weight_decay, step, seed):
// the bytes of a muon_adamw_desc array.  scales: None, or a list of None and
// tensors.
PyObject* adamw(PyObject*, PyObject* args) {
  PyObject *op, *og, *om, *ov, *os;
  long index;
  Numbers lr, decay, step, seed;
  if (!PyArg_ParseTuple(args, "OOOOOlOOOO", &op, &og, &om, &ov, &os, &index, &lr.o, &decay.o, &step.o, &seed.o))
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
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(d.data()), n * (Py_ssize_t)sizeof(muon_adamw_desc));
  });
}

// clip(grads, outs, index): the bytes of a muon_clip_desc array.
PyObject* clip(PyObject*, PyObject* args) {
  PyObject *og, *oo;
  long index;
  if (!PyArg_ParseTuple(args, "OOl", &og, &oo, &index)) return nullptr;
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
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(d.data()), n * (Py_ssize_t)sizeof(muon_clip_desc));
  });
}

PyMethodDef methods[] = {
    {"adamw", adamw, METH_VARARGS, "The bytes of a muon_adamw_desc array, or None when a check fails."},
    {"clip", clip, METH_VARARGS, "The bytes of a muon_clip_desc array, or None when a check fails."},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_lists", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_lists() { return PyModule_Create(&module); }
