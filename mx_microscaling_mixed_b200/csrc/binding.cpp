// binding.cpp -- the serving calls' arguments from Python to libmxs in one
// step, for their ordinary form: CUDA tensors on the current device, outputs
// and partial results made by the call, the current stream.  A function
// returns what the call gives, the status (an int) where it was refused, or
// None where the arguments are of another form: the binding in capi.py then
// takes them, and says what is wrong with them if something is.
//   A decode step makes a handful of these calls of a few microseconds each;
// through ctypes and torch's Python functions one takes 9 us on the host,
// from here 4, the launch included.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mxs.h"

namespace {

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// On CUDA device `dev`, an ordinary dense or strided tensor.
bool here(const at::Tensor &t, int dev) { return t.is_cuda() && t.get_device() == dev && t.layout() == at::kStrided; }

// bf16 or fp32, (tokens, heads, d) with unit stride along d.
bool heads_ok(const at::Tensor &t) {
  const auto st = t.scalar_type();
  return t.dim() == 3 && (st == at::kBFloat16 || st == at::kFloat) && (t.stride(2) == 1 || t.size(2) <= 1);
}
bool index_ok(const at::Tensor &t, int64_t n, int dev) {
  return here(t, dev) && t.scalar_type() == at::kLong && t.dim() == 1 && t.numel() == n && t.is_contiguous();
}
mxs_dtype type_of(const at::Tensor &t) { return t.scalar_type() == at::kFloat ? MXS_F32 : MXS_BF16; }
void *stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

at::Tensor empty(at::IntArrayRef shape, at::ScalarType st, int dev) {
  return at::empty(shape, at::TensorOptions().dtype(st).device(at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev))));
}

template <typename F>
PyObject *guarded(F f) {
  try {
    return f();
  } catch (const std::exception &e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
PyObject *other_form() { Py_RETURN_NONE; }
PyObject *status(mxs_status st) { return PyLong_FromLong(st); }

// 0: bf16, 1: fp32, -1: neither.
int type_code(PyObject *dtype) {
  if (!THPDtype_Check(dtype)) return -1;
  const auto st = reinterpret_cast<THPDtype *>(dtype)->scalar_type;
  return st == at::kBFloat16 ? 0 : st == at::kFloat ? 1 : -1;
}
at::ScalarType scalar(int code) { return code ? at::kFloat : at::kBFloat16; }

// rope(x, pos, plan address, inverse, dtype or None)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 5) return other_form();
    const at::Tensor *x = tensor(a[0]), *pos = tensor(a[1]);
    if (!x || !pos || !x->is_cuda()) return other_form();
    const int dev = c10::cuda::current_device();
    if (!here(*x, dev) || !heads_ok(*x) || !index_ok(*pos, x->size(0), dev)) return other_form();
    int code = type_of(*x) == MXS_F32;
    if (a[4] != Py_None && (code = type_code(a[4])) < 0) return other_form();
    const int inverse = PyObject_IsTrue(a[3]);
    const auto *plan = static_cast<const mxs_rope_plan *>(PyLong_AsVoidPtr(a[2]));
    if (inverse < 0 || PyErr_Occurred()) return nullptr;
    const int64_t T = x->size(0), heads = x->size(1), d = x->size(2);
    at::Tensor out = empty({T, heads, d}, scalar(code), dev);
    const mxs_status st = mxs_rope(x->data_ptr(), type_of(*x), T, heads, d, x->stride(0), x->stride(1),
                                   static_cast<const int64_t *>(pos->data_ptr()), plan, inverse, out.data_ptr(),
                                   code ? MXS_F32 : MXS_BF16, heads * d, d, stream_of(dev));
    return st == MXS_OK ? THPVariable_Wrap(out) : status(st);
  });
}

// (asked with a device index of a tensor: CUDA is up then)
bool current(int dev) { return dev >= 0 && dev == c10::cuda::current_device(); }

struct Cache {
  const mxs_kv_cache *c;
  int dev;
};
// The cache's address and device index (-1: not a CUDA device).
bool cache_of(PyObject *address, PyObject *index, Cache *out) {
  out->c = static_cast<const mxs_kv_cache *>(PyLong_AsVoidPtr(address));
  out->dev = static_cast<int>(PyLong_AsLong(index));
  return !PyErr_Occurred();
}

// kv_write(k, v, cache address, device, slot, pos or None, plan address or None)
PyObject *kv_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 7) return other_form();
    const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *slot = tensor(a[4]);
    Cache c;
    if (!cache_of(a[2], a[3], &c)) return nullptr;
    const bool turn = a[5] != Py_None;
    const at::Tensor *pos = turn ? tensor(a[5]) : nullptr;
    if (!k || !v || !slot || (turn && !pos) || turn != (a[6] != Py_None)) return other_form();
    if (!k->is_cuda() || !current(c.dev)) return other_form();
    if (!here(*k, c.dev) || !here(*v, c.dev) || !heads_ok(*k) || !heads_ok(*v) || k->sizes() != v->sizes() ||
        k->scalar_type() != v->scalar_type() || k->size(1) != c.c->n_kvh || k->size(2) != c.c->K.lay.K)
      return other_form();
    const int64_t T = k->size(0);
    if (!index_ok(*slot, T, c.dev) || (turn && !index_ok(*pos, T, c.dev))) return other_form();
    const void *plan = turn ? PyLong_AsVoidPtr(a[6]) : nullptr;
    if (PyErr_Occurred()) return nullptr;
    return status(mxs_kv_write(k->data_ptr(), k->stride(0), k->stride(1), v->data_ptr(), v->stride(0), v->stride(1),
                               type_of(*k), T, static_cast<const int64_t *>(slot->data_ptr()),
                               turn ? static_cast<const int64_t *>(pos->data_ptr()) : nullptr,
                               static_cast<const mxs_rope_plan *>(plan), c.c, stream_of(c.dev)));
  });
}

// kv_read(cache address, device, slot, dtype)
PyObject *kv_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 4) return other_form();
    Cache c;
    if (!cache_of(a[0], a[1], &c)) return nullptr;
    const at::Tensor *slot = tensor(a[2]);
    const int code = type_code(a[3]);
    if (!slot || code < 0 || !slot->is_cuda() || !current(c.dev) || slot->dim() != 1 ||
        !index_ok(*slot, slot->numel(), c.dev))
      return other_form();
    const int64_t T = slot->numel(), h = c.c->n_kvh, d = c.c->K.lay.K;
    at::Tensor k = empty({T, h, d}, scalar(code), c.dev), v = empty({T, h, d}, scalar(code), c.dev);
    const mxs_status st = mxs_kv_read(c.c, T, static_cast<const int64_t *>(slot->data_ptr()), k.data_ptr(), h * d, d,
                                      v.data_ptr(), h * d, d, code ? MXS_F32 : MXS_BF16, stream_of(c.dev));
    if (st != MXS_OK) return status(st);
    PyObject *ko = THPVariable_Wrap(k), *vo = THPVariable_Wrap(v);
    PyObject *both = ko && vo ? PyTuple_Pack(2, ko, vo) : nullptr;
    Py_XDECREF(ko);
    Py_XDECREF(vo);
    return both;
  });
}

// attn_tree(q, cache address, device, batch address, batch's device, scale, dtype, lse wanted, workspace or None)
PyObject *attn_tree(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    if (n != 9) return other_form();
    const at::Tensor *q = tensor(a[0]);
    Cache c;
    if (!cache_of(a[1], a[2], &c)) return nullptr;
    const auto *batch = static_cast<const mxs_tree_batch *>(PyLong_AsVoidPtr(a[3]));
    const long batch_dev = PyLong_AsLong(a[4]);
    const double scale = PyFloat_AsDouble(a[5]);
    const int code = type_code(a[6]), want_lse = PyObject_IsTrue(a[7]);
    if (PyErr_Occurred()) return nullptr;
    if (!q || code < 0 || !q->is_cuda() || !current(c.dev) || batch_dev != c.dev || !here(*q, c.dev) ||
        !heads_ok(*q) || q->scalar_type() != at::kBFloat16 || q->size(2) != c.c->K.lay.K)
      return other_form();
    const int64_t rows = q->size(0), n_qh = q->size(1), d = q->size(2);
    mxs_tree_batch t = *batch;
    if (t.mask && t.rows != rows) return other_form();
    t.rows = rows;                                   // a chain's batch covers the rows that q has
    const mxs_dtype ot = code ? MXS_F32 : MXS_BF16;
    const at::Tensor *ws = nullptr;
    at::Tensor own;
    if (a[8] != Py_None) {
      ws = tensor(a[8]);
      if (!ws || !here(*ws, c.dev) || !ws->is_contiguous()) return other_form();
    } else {
      size_t need = 0;
      const mxs_status st = mxs_attn_tree_workspace_bytes(c.c, &t, n_qh, ot, &need);
      if (st != MXS_OK) return status(st);
      own = empty({static_cast<int64_t>(need) + 256}, at::kByte, c.dev);
      ws = &own;
    }
    const uintptr_t base = reinterpret_cast<uintptr_t>(ws->data_ptr()), p = (base + 255) / 256 * 256;
    const size_t bytes = ws->numel() * ws->element_size();
    at::Tensor out = empty({rows, n_qh, d}, scalar(code), c.dev), lse;
    if (want_lse) lse = empty({rows, n_qh}, at::kFloat, c.dev);
    const mxs_status st = mxs_attn_tree(q->data_ptr(), n_qh, q->stride(0), q->stride(1), c.c, &t, static_cast<float>(scale),
                                        out.data_ptr(), ot, n_qh * d, d,
                                        want_lse ? static_cast<float *>(lse.data_ptr()) : nullptr,
                                        reinterpret_cast<void *>(p), bytes > p - base ? bytes - (p - base) : 0,
                                        stream_of(c.dev));
    if (st != MXS_OK) return status(st);
    if (!want_lse) return THPVariable_Wrap(out);
    PyObject *oo = THPVariable_Wrap(out), *lo = THPVariable_Wrap(lse);
    PyObject *both = oo && lo ? PyTuple_Pack(2, oo, lo) : nullptr;
    Py_XDECREF(oo);
    Py_XDECREF(lo);
    return both;
  });
}

template <typename F>
PyCFunction method(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {
    {"rope", method(rope), METH_FASTCALL, nullptr},
    {"kv_write", method(kv_write), METH_FASTCALL, nullptr},
    {"kv_read", method(kv_read), METH_FASTCALL, nullptr},
    {"attn_tree", method(attn_tree), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
