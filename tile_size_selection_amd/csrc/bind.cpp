// The entry points of tss.h as Python functions, for the calls whose time on
// the host counts: a tensor argument becomes its data's address, the current
// stream of the tensors' GPU is added as the last argument, and that GPU is
// current for the call.  Python code checks shapes and types before (with
// `fits`, which says whether a tensor is contiguous and has a given shape and
// element type); here every tensor must be on one GPU.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <type_traits>
#include <utility>
#include <vector>

#include "tss.h"

extern "C" int hipGetDevice(int *);
extern "C" int hipSetDevice(int);

namespace {

constexpr int kMostArgs = 24;
PyObject *raw_stream;  // device index -> the current stream's handle

struct Slot {
  long long i = 0;
  double d = 0;
};

// The GPU that all of the call's tensors are on: -1 before the first one.
bool place(const at::Tensor &t, int &device) {
  const int at = t.is_cuda() ? int(t.get_device()) : -2;
  if (device == -1) device = at;
  if (at < 0 || at != device) {
    PyErr_SetString(PyExc_ValueError, "every tensor must be on the same GPU");
    return false;
  }
  return true;
}

bool take(PyObject *o, Slot &s, int &device) {
  if (o == Py_None) return true;
  if (THPVariable_Check(o)) {
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!place(t, device)) return false;
    s.i = reinterpret_cast<long long>(t.data_ptr());
    return true;
  }
  if (PyBytes_Check(o)) {
    s.i = reinterpret_cast<long long>(PyBytes_AS_STRING(o));
    return true;
  }
  if (PyFloat_Check(o)) {
    s.d = PyFloat_AS_DOUBLE(o);
    return true;
  }
  PyObject *n = PyNumber_Index(o);
  if (!n) return false;
  s.i = PyLong_AsLongLong(n);
  Py_DECREF(n);
  s.d = double(s.i);
  return !(s.i == -1 && PyErr_Occurred());
}

template <typename T>
T as(const Slot &s) {
  if constexpr (std::is_pointer_v<T>) return reinterpret_cast<T>(s.i);
  else if constexpr (std::is_floating_point_v<T>) return T(s.d);
  else return T(s.i);
}

template <typename T>
bool fits_arg(const Slot &s) {
  if constexpr (std::is_integral_v<T> && sizeof(T) == 4) return s.i >= INT32_MIN && s.i <= INT32_MAX;
  else return true;
}

// f(), with what it throws as a Python error.
template <typename F>
PyObject *guarded(F f) {
  try {
    return f();
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <auto F>
struct Entry;
template <typename... A, int32_t (*F)(A...)>
struct Entry<F> {
  static constexpr int kArgs = sizeof...(A);
  static_assert(kArgs <= kMostArgs);
  template <size_t... I>
  static int32_t run(const Slot *s, std::index_sequence<I...>) {
    return F(as<A>(s[I])...);
  }
  template <size_t... I>
  static bool in_range(const Slot *s, std::index_sequence<I...>) {
    return (fits_arg<A>(s[I]) && ...);
  }
  // Every argument but the stream.
  static PyObject *call(PyObject *const *args, Py_ssize_t n) {
    if (n != kArgs - 1) return PyErr_Format(PyExc_TypeError, "%d arguments, not %d", int(n), kArgs - 1);
    Slot s[kArgs];
    int device = -1;
    for (int i = 0; i < kArgs - 1; ++i)
      if (!take(args[i], s[i], device)) return nullptr;
    if (device < 0) return PyErr_Format(PyExc_ValueError, "no tensor on a GPU");
    if (!in_range(s, std::make_index_sequence<kArgs>())) return PyErr_Format(PyExc_OverflowError, "an argument does not fit 32 bits");
    PyObject *index = PyLong_FromLong(device);
    if (!index) return nullptr;
    PyObject *handle = PyObject_CallOneArg(raw_stream, index);
    Py_DECREF(index);
    if (!handle) return nullptr;
    s[kArgs - 1].i = reinterpret_cast<long long>(PyLong_AsVoidPtr(handle));
    Py_DECREF(handle);
    if (PyErr_Occurred()) return nullptr;
    int now = device;
    hipGetDevice(&now);
    if (now != device) hipSetDevice(device);
    const int32_t st = run(s, std::make_index_sequence<kArgs>());
    if (now != device) hipSetDevice(now);
    return PyLong_FromLong(st);
  }
};

// A workspace's size: no tensor, no stream.
template <auto F>
struct Size;
template <typename... A, int64_t (*F)(A...)>
struct Size<F> {
  template <size_t... I>
  static int64_t run(const Slot *s, std::index_sequence<I...>) {
    return F(as<A>(s[I])...);
  }
  static PyObject *call(PyObject *const *args, Py_ssize_t n) {
    constexpr int kArgs = sizeof...(A);
    if (n != kArgs) return PyErr_Format(PyExc_TypeError, "%d arguments, not %d", int(n), kArgs);
    Slot s[kArgs];
    int device = -1;
    for (int i = 0; i < kArgs; ++i)
      if (!take(args[i], s[i], device)) return nullptr;
    return PyLong_FromLongLong(run(s, std::make_index_sequence<kArgs>()));
  }
};

// fits(tensor, dtype, size, ...): contiguous, of this element type and shape.
PyObject *fits(PyObject *const *args, Py_ssize_t n) {
  if (n < 2 || !THPVariable_Check(args[0]) || !THPDtype_Check(args[1]))
    return PyErr_Format(PyExc_TypeError, "fits(tensor, dtype, size, ...)");
  const at::Tensor &t = THPVariable_Unpack(args[0]);
  bool ok = t.scalar_type() == reinterpret_cast<THPDtype *>(args[1])->scalar_type && t.dim() == n - 2 && t.is_contiguous();
  for (Py_ssize_t i = 2; ok && i < n; ++i) {
    const long long v = PyLong_AsLongLong(args[i]);
    if (v == -1 && PyErr_Occurred()) return nullptr;
    ok = t.size(i - 2) == v;
  }
  return PyBool_FromLong(ok);
}

// table(list of tensors, out list or None, types): (addresses, elements, type
// numbers, outputs' addresses or None, GPU) with types a dict of element types
// to numbers; None if a tensor's type is not among them, it has gaps, or an
// output is not like its tensor (the caller then finds out which).
PyObject *table(PyObject *const *args, Py_ssize_t nargs) {
  if (nargs != 3 || !PyList_Check(args[0]) || !(args[1] == Py_None || PyList_Check(args[1])) || !PyDict_Check(args[2]))
    return PyErr_Format(PyExc_TypeError, "table(list, list or None, dict)");
  const Py_ssize_t n = PyList_GET_SIZE(args[0]);
  const bool out = args[1] != Py_None;
  if (out && PyList_GET_SIZE(args[1]) != n) Py_RETURN_NONE;
  std::vector<int64_t> at(n), size(n), to(n);
  std::vector<int32_t> type(n);
  int device = -1;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject *o = PyList_GET_ITEM(args[0], i), *w = out ? PyList_GET_ITEM(args[1], i) : o;
    if (!THPVariable_Check(o) || !THPVariable_Check(w)) Py_RETURN_NONE;
    const at::Tensor &t = THPVariable_Unpack(o), &v = THPVariable_Unpack(w);
    if (!place(t, device) || (w != o && !place(v, device))) return nullptr;
    if (!t.is_non_overlapping_and_dense()) Py_RETURN_NONE;
    if (w != o && (v.scalar_type() != t.scalar_type() || v.sizes() != t.sizes() || v.strides() != t.strides())) Py_RETURN_NONE;
    PyObject *d = reinterpret_cast<PyObject *>(torch::getTHPDtype(t.scalar_type()));
    PyObject *number = PyDict_GetItemWithError(args[2], d);
    if (!number) {
      if (PyErr_Occurred()) return nullptr;
      Py_RETURN_NONE;
    }
    type[i] = int32_t(PyLong_AsLong(number));
    at[i] = reinterpret_cast<int64_t>(t.data_ptr());
    to[i] = reinterpret_cast<int64_t>(v.data_ptr());
    size[i] = t.numel();
  }
  auto bytes = [](const auto &v) {
    return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(v.data()), Py_ssize_t(v.size() * sizeof(v[0])));
  };
  return out ? Py_BuildValue("NNNNi", bytes(at), bytes(size), bytes(type), bytes(to), device)
             : Py_BuildValue("NNNOi", bytes(at), bytes(size), bytes(type), Py_None, device);
}

template <auto F>
PyObject *method(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&] { return F(args, n); });
}

#define TSS_METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&f)), METH_FASTCALL, nullptr}
#define TSS_ENTRY(name) TSS_METHOD(#name, method<Entry<name>::call>)
#define TSS_SIZE(name) TSS_METHOD(#name, method<Size<name>::call>)
PyMethodDef methods[] = {
    TSS_SIZE(tss_layer_norm_backward_workspace_size),
    TSS_SIZE(tss_gemm_int8_workspace_size),
    TSS_SIZE(tss_clip_grad_norm_workspace_size),
    TSS_SIZE(tss_sort_by_expert_workspace_size),
    TSS_METHOD("fits", method<fits>),
    TSS_METHOD("table", method<table>),
    TSS_ENTRY(tss_layer_norm),
    TSS_ENTRY(tss_layer_norm_backward),
    TSS_ENTRY(tss_quantize_int8),
    TSS_ENTRY(tss_gemm_int8),
    TSS_ENTRY(tss_clip_grad_norm),
    TSS_ENTRY(tss_sort_by_expert),
    TSS_ENTRY(tss_gather_rows),
    TSS_ENTRY(tss_combine_rows),
    TSS_ENTRY(tss_combine_rows_backward),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() {
  PyObject *m = PyModule_Create(&module);
  if (!m) return nullptr;
  PyObject *torch = PyImport_ImportModule("torch._C");
  raw_stream = torch ? PyObject_GetAttrString(torch, "_cuda_getCurrentRawStream") : nullptr;
  Py_XDECREF(torch);
  if (!raw_stream) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
