// Native half of the Python binding for the recurrent block's entry points
// (include/ttt.h): fills the ttt_tensor descriptors from torch tensors and
// calls the C function, about 1 us instead of the 15 us that building a dozen
// descriptors in Python takes. A single-token call is 7 to 9 us in all.
//
// call(function, tensors, split, scalar, stream, name) -> status. `function` is the
// C function's address (from the loaded library), `tensors` a tuple of tensors
// or None, the scalar argument goes behind the first `split` of them. `stream`
// is None for the tensors' device's current stream, or a stream's handle.
//
// Whatever torch throws (a tensor without memory of its own, as inside
// torch.func's transforms; an allocation that fails) becomes the Python
// exception that torch itself raises for it.
#include <ATen/ATen.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <array>
#include <utility>
#include <vector>

#include "../../include/ttt.h"

namespace {

constexpr size_t kMost = 24;

template <size_t NA, size_t NB, typename S, size_t... A, size_t... B>
ttt_status invoke(void* f, ttt_tensor* const* t, S scalar, void* stream, std::index_sequence<A...>,
                  std::index_sequence<B...>) {
  using At = const ttt_tensor*;
  using F = ttt_status (*)(decltype((void)A, At())..., S, decltype((void)B, At())..., void*);
  return reinterpret_cast<F>(f)(t[A]..., scalar, t[NA + B]..., stream);
}
template <size_t NA, size_t NB, typename S>
ttt_status invoke(void* f, ttt_tensor* const* t, S scalar, void* stream) {
  return invoke<NA, NB, S>(f, t, scalar, stream, std::make_index_sequence<NA>(), std::make_index_sequence<NB>());
}

PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 6 || !PyTuple_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "call(function, tensors, split, scalar, stream, name)");
    return nullptr;
  }
  void* fn = PyLong_AsVoidPtr(args[0]);
  const Py_ssize_t n = PyTuple_GET_SIZE(args[1]);
  const long split = PyLong_AsLong(args[2]);
  const bool real = PyFloat_Check(args[3]);
  const double fs = real ? PyFloat_AS_DOUBLE(args[3]) : 0.0;
  const long is = real ? 0 : PyLong_AsLong(args[3]);
  void* given = args[4] == Py_None ? nullptr : PyLong_AsVoidPtr(args[4]);
  const char* name = PyUnicode_AsUTF8(args[5]);
  if (PyErr_Occurred()) return nullptr;
  if (!name || !fn || n > (Py_ssize_t)kMost) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no such call");
    return nullptr;
  }
  ttt_tensor desc[kMost];
  ttt_tensor* t[kMost] = {};
  int device = -1;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = PyTuple_GET_ITEM(args[1], i);
    if (o == Py_None) continue;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "%s: argument %zd is not a tensor", name, i);
      return nullptr;
    }
    const at::Tensor& v = THPVariable_Unpack(o);
    const int on = v.is_cuda() ? v.get_device() : -1;
    if (on < 0 || (device >= 0 && on != device)) {
      PyErr_Format(PyExc_ValueError, "%s: tensors have to be on one CUDA device", name);
      return nullptr;
    }
    device = on;
    if (v.layout() != at::kStrided || v.dim() > 4) {
      PyErr_Format(PyExc_ValueError, "%s: tensors have to be strided, of at most 4 dimensions", name);
      return nullptr;
    }
    if (v.is_neg()) {  // its memory holds the values with the other sign
      PyErr_Format(PyExc_ValueError, "%s: argument %zd is a negated view: resolve_neg() first", name, i);
      return nullptr;
    }
    ttt_tensor& d = desc[i];
    switch (v.scalar_type()) {
      case at::kFloat: d.dtype = TTT_F32; break;
      case at::kBFloat16: d.dtype = TTT_BF16; break;
      case at::kInt: d.dtype = TTT_I32; break;
      case at::kFloat8_e4m3fn: d.dtype = TTT_E4M3; break;
      default:
        PyErr_Format(PyExc_TypeError, "%s: unsupported dtype (argument %zd)", name, i);
        return nullptr;
    }
    d.data = v.numel() ? v.data_ptr() : nullptr;
    d.ndim = (int32_t)v.dim();
    for (int k = 0; k < 4; ++k) {
      d.shape[k] = k < d.ndim ? v.size(k) : 0;
      d.stride[k] = k < d.ndim ? v.stride(k) : 0;
    }
    t[i] = &d;
  }
  if (device < 0) {
    PyErr_Format(PyExc_TypeError, "%s: no tensor", name);
    return nullptr;
  }
  ttt_status st = TTT_ERR_ARG;
  bool known = true;
  {
    const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)device));
    void* s = args[4] == Py_None ? (void*)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream() : given;
    Py_BEGIN_ALLOW_THREADS
    const float f = (float)fs;
    const int32_t k = (int32_t)is;
    if (real && split == 3 && n == 6) st = invoke<3, 3>(fn, t, f, s);
    else if (real && split == 4 && n == 6) st = invoke<4, 2>(fn, t, f, s);
    else if (!real && split == 5 && n == 6) st = invoke<5, 1>(fn, t, k, s);
    else if (!real && split == 5 && n == 7) st = invoke<5, 2>(fn, t, k, s);
    else if (!real && split == 5 && n == 11) st = invoke<5, 6>(fn, t, k, s);
    else if (!real && split == 10 && n == 11) st = invoke<10, 1>(fn, t, k, s);
    else if (!real && split == 10 && n == 12) st = invoke<10, 2>(fn, t, k, s);
    else if (!real && split == 10 && n == 21) st = invoke<10, 11>(fn, t, k, s);
    else known = false;
    Py_END_ALLOW_THREADS
  }
  if (!known) {
    PyErr_Format(PyExc_ValueError, "%s: no such call", name);
    return nullptr;
  }
  return PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// Layout of a new token tensor [B,H,T,d]: x's order of storage (heads before or
// behind tokens), its rows a multiple of 16 bytes apart.
struct Rows {
  std::array<int64_t, 4> size, stride;
  int64_t count;
  Rows(const at::Tensor& x, int64_t d, int64_t element) {
    const int64_t B = x.size(0), H = x.size(1), T = x.size(2);
    const int64_t per = 16 / element, row = (d + per - 1) / per * per;
    const bool behind = H > 1 && T > 1 && x.stride(1) < x.stride(2);
    size = {B, H, T, d};
    stride = {H * T * row, behind ? row : T * row, behind ? H * row : row, 1};
    count = B * H * T * row;
  }
};

PyObject* like_tokens(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 4 || !THPVariable_Check(args[0]) || !THPDtype_Check(args[2])) {
    PyErr_SetString(PyExc_TypeError, "like_tokens(x, d, dtype, zero)");
    return nullptr;
  }
  const at::Tensor& x = THPVariable_Unpack(args[0]);
  const int64_t d = PyLong_AsLongLong(args[1]);
  const auto type = reinterpret_cast<THPDtype*>(args[2])->scalar_type;
  const int zero = PyObject_IsTrue(args[3]);
  if (PyErr_Occurred()) return nullptr;
  if (x.dim() != 4 || d < 0) {
    PyErr_SetString(PyExc_ValueError, "tokens are [B,H,T,d]");
    return nullptr;
  }
  const Rows r(x, d, (int64_t)c10::elementSize(type));
  const auto opt = x.options().dtype(type).requires_grad(false);
  const at::Tensor t = zero ? at::zeros({r.count}, opt) : at::empty({r.count}, opt);
  return THPVariable_Wrap(t.as_strided(r.size, r.stride));
  END_HANDLE_TH_ERRORS
}

// New zero tensors like each of a tuple of token tensors of one type (None gives
// None), in one allocation with one fill.
PyObject* zeros_like_tokens(PyObject*, PyObject* arg) {
  HANDLE_TH_ERRORS
  if (!PyTuple_Check(arg)) {
    PyErr_SetString(PyExc_TypeError, "zeros_like_tokens((x, ...))");
    return nullptr;
  }
  const Py_ssize_t n = PyTuple_GET_SIZE(arg);
  std::vector<Rows> rows;
  const at::Tensor* first = nullptr;
  int64_t total = 0;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = PyTuple_GET_ITEM(arg, i);
    if (o == Py_None) continue;
    if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 4) {
      PyErr_SetString(PyExc_ValueError, "tokens are [B,H,T,d]");
      return nullptr;
    }
    const at::Tensor& x = THPVariable_Unpack(o);
    if (!first) first = &x;
    rows.emplace_back(x, x.size(3), (int64_t)x.element_size());
    total += rows.back().count;
  }
  THPObjectPtr out(PyTuple_New(n));
  if (!out) return nullptr;
  at::Tensor all;
  if (first) all = at::zeros({total}, first->options().requires_grad(false));
  int64_t at_ = 0;
  size_t k = 0;
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (PyTuple_GET_ITEM(arg, i) == Py_None) {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(out.get(), i, Py_None);
      continue;
    }
    PyTuple_SET_ITEM(out.get(), i, THPVariable_Wrap(all.as_strided(rows[k].size, rows[k].stride, at_)));
    at_ += rows[k++].count;
  }
  return out.release();
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"like_tokens", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(like_tokens)), METH_FASTCALL,
     "like_tokens(x, d, dtype, zero) -> tensor"},
    {"zeros_like_tokens", zeros_like_tokens, METH_O, "zeros_like_tokens((x, ...)) -> tensors"},
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(call)), METH_FASTCALL,
     "call(function, tensors, split, scalar, stream, name) -> status"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: what the module was compiled against (build.py's binding_key())
PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", TTT_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
