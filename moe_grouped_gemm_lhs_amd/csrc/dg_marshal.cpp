// dg_marshal.cpp -- the Python module _marshal: what the binding of the gate, the adapters
// and the feed-forward operators does for every argument of every call, in C++.  A decode
// step makes these calls once a layer with a few microseconds of GPU work each; checking ten
// tensors through their Python attributes and a ctypes call of twenty arguments took 7 us of
// the host's 12 (one token of dg_lora_bf16, two launches).
//
// vector() and rows() return at once for the usual argument; whatever else it may be goes to
// the Python functions given to use_slow(), which find out what is wrong and say so.  The
// calls of include/dg.h have their C names and arguments; None is a null pointer.
#include <Python.h>

#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <tuple>
#include <type_traits>
#include <utility>

#include "dg.h"

namespace {

PyObject *slow_vector, *slow_rows;

// Whether args (t, name, dtype, shape, device) are a tensor of just this dtype, shape, device.
bool matches(PyObject* const* args) {
  if (!THPVariable_Check(args[0]) || !THPDtype_Check(args[2]) || !PyTuple_Check(args[3]) ||
      !THPDevice_Check(args[4]))
    return false;
  const at::Tensor& t = THPVariable_Unpack(args[0]);
  if (t.layout() != at::kStrided || t.scalar_type() != ((THPDtype*)args[2])->scalar_type ||
      t.device() != ((THPDevice*)args[4])->device || t.dim() != PyTuple_GET_SIZE(args[3]))
    return false;
  for (int64_t i = 0; i < t.dim(); ++i) {
    const long long n = PyLong_AsLongLong(PyTuple_GET_ITEM(args[3], i));
    if (n == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      return false;
    }
    if (t.size(i) != n) return false;
  }
  return true;
}

// Pointer of an optional dense argument (None: a null pointer).
PyObject* vector(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "vector(t, name, dtype, shape, device)");
    return nullptr;
  }
  if (args[0] == Py_None) Py_RETURN_NONE;
  try {
    if (matches(args)) {
      const at::Tensor& t = THPVariable_Unpack(args[0]);
      if (t.is_contiguous()) return PyLong_FromVoidPtr(t.data_ptr());
    }
  } catch (...) {                            // a tensor without memory of its own
  }
  return PyObject_Vectorcall(slow_vector, args, n, nullptr);
}

// Pointer and row stride of a matrix whose rows are dense but may lie apart.  Of no or one row
// the row stride says nothing.
PyObject* rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "rows(t, name, dtype, shape, device)");
    return nullptr;
  }
  try {
    if (matches(args)) {
      const at::Tensor& t = THPVariable_Unpack(args[0]);
      if (t.dim() == 2 && (t.size(0) == 0 || t.size(1) <= 1 || t.stride(1) == 1))
        return Py_BuildValue("(NL)", PyLong_FromVoidPtr(t.data_ptr()),
                             (long long)(t.size(0) <= 1 ? t.size(1) : t.stride(0)));
    }
  } catch (...) {
  }
  return PyObject_Vectorcall(slow_rows, args, n, nullptr);
}

PyObject* use_slow(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 2 || !PyCallable_Check(args[0]) || !PyCallable_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "use_slow(vector, rows)");
    return nullptr;
  }
  Py_INCREF(args[0]);
  Py_INCREF(args[1]);
  Py_XSETREF(slow_vector, args[0]);
  Py_XSETREF(slow_rows, args[1]);
  Py_RETURN_NONE;
}

// ------------------------------------------------------------------------ calls of dg.h
template <class T>
T from(PyObject* v) {
  if constexpr (std::is_pointer_v<T>) {
    return v == Py_None ? nullptr : (T)PyLong_AsVoidPtr(v);
  } else if constexpr (std::is_floating_point_v<T>) {
    return (T)PyFloat_AsDouble(v);
  } else if constexpr (std::is_unsigned_v<T>) {
    return (T)PyLong_AsSize_t(v);
  } else {
    const long long x = PyLong_AsLongLong(v);
    if ((T)x != x) PyErr_SetString(PyExc_OverflowError, "integer argument out of range");
    return (T)x;
  }
}

template <class R, class... A, size_t... I>
PyObject* call(R (*f)(A...), PyObject* const* args, Py_ssize_t n, std::index_sequence<I...>) {
  if (n != (Py_ssize_t)sizeof...(A)) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", (int)sizeof...(A), n);
    return nullptr;
  }
  std::tuple<A...> v{from<A>(args[I])...};
  if (PyErr_Occurred()) return nullptr;
  R r;
  Py_BEGIN_ALLOW_THREADS
  r = f(std::get<I>(v)...);
  Py_END_ALLOW_THREADS
  return std::is_unsigned_v<R> ? PyLong_FromSize_t((size_t)r) : PyLong_FromLong((long)r);
}

template <auto f>
struct Call;
template <class R, class... A, R (*f)(A...)>
struct Call<f> {
  static PyObject* run(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return call(f, args, n, std::index_sequence_for<A...>{});
  }
};

#define DG_METHOD(name, f) {name, (PyCFunction)(void (*)())f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    DG_METHOD("vector", vector),
    DG_METHOD("rows", rows),
    DG_METHOD("use_slow", use_slow),
    DG_METHOD("dg_moe_route_workspace_bytes", Call<dg_moe_route_workspace_bytes>::run),
    DG_METHOD("dg_moe_route", Call<dg_moe_route>::run),
    DG_METHOD("dg_moe_route_backward", Call<dg_moe_route_backward>::run),
    DG_METHOD("dg_lora_workspace_bytes", Call<dg_lora_workspace_bytes>::run),
    DG_METHOD("dg_lora_bf16", Call<dg_lora_bf16>::run),
    DG_METHOD("dg_rms_norm_fp8", Call<dg_rms_norm_fp8>::run),
    DG_METHOD("dg_rms_norm_backward_workspace_bytes", Call<dg_rms_norm_backward_workspace_bytes>::run),
    DG_METHOD("dg_rms_norm_backward", Call<dg_rms_norm_backward>::run),
    DG_METHOD("dg_gated_workspace_bytes", Call<dg_gated_workspace_bytes>::run),
    DG_METHOD("dg_gated_fp8_nt", Call<dg_gated_fp8_nt>::run),
    DG_METHOD("dg_grouped_gated_fp8_contiguous", Call<dg_grouped_gated_fp8_contiguous>::run),
    DG_METHOD("dg_grouped_gated_fp8_masked", Call<dg_grouped_gated_fp8_masked>::run),
    DG_METHOD("dg_gated_backward", Call<dg_gated_backward>::run),
    DG_METHOD("dg_wgrad_workspace_bytes", Call<dg_wgrad_workspace_bytes>::run),
    DG_METHOD("dg_wgrad_fp8", Call<dg_wgrad_fp8>::run),
    DG_METHOD("dg_grouped_wgrad_fp8_contiguous", Call<dg_grouped_wgrad_fp8_contiguous>::run),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
