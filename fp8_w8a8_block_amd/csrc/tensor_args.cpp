// What a call reads of its tensor arguments, in one step each: type, device,
// shape and strides checked, pointer and sizes returned.  A tensor that is not
// as a call expects it gives None, and the binding's Python checks say why.
//
// A call of the attention step takes 7 to 17 tensors; each attribute read from
// Python costs 70 to 130 ns, a whole step's checks more than its kernels where
// those are small.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// The tensor behind o if it is one of this type on this device, which is a GPU.
const at::Tensor* tensor_of(PyObject* o, at::ScalarType type, PyObject* device) {
  if (!THPVariable_Check(o) || !THPDevice_Check(device)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || t.layout() != at::kStrided || t.scalar_type() != type || !t.is_cuda() ||
      t.device() != reinterpret_cast<THPDevice*>(device)->device)
    return nullptr;
  return &t;
}

PyObject* pointer(const at::Tensor& t) { return PyLong_FromVoidPtr(t.data_ptr()); }

// vector(t, dtype, device, n) -> pointer: contiguous, 1-D, of n elements (n < 0: any)
PyObject* vector(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 4 || !THPDtype_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "vector(tensor, dtype, device, n)");
    return nullptr;
  }
  const auto type = reinterpret_cast<THPDtype*>(args[1])->scalar_type;
  const long long n = PyLong_AsLongLong(args[3]);
  if (n == -1 && PyErr_Occurred()) return nullptr;
  const at::Tensor* t = tensor_of(args[0], type, args[2]);
  if (!t || t->dim() != 1 || (n >= 0 && t->size(0) != n) || !t->is_contiguous()) Py_RETURN_NONE;
  return pointer(*t);
}

// heads(t, device) -> (pointer, T, H, D, token stride): bf16 [T, H, D], not empty,
// each token's H D values contiguous
PyObject* heads(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 2) {
    PyErr_SetString(PyExc_TypeError, "heads(tensor, device)");
    return nullptr;
  }
  const at::Tensor* t = tensor_of(args[0], at::kBFloat16, args[1]);
  if (!t || t->dim() != 3 || t->numel() == 0) Py_RETURN_NONE;
  const long long T = t->size(0), H = t->size(1), D = t->size(2);
  if (t->stride(2) != 1 || (H > 1 && t->stride(1) != D)) Py_RETURN_NONE;
  return Py_BuildValue("NLLLL", pointer(*t), T, H, D,
                       T > 1 ? (long long)t->stride(0) : H * D);
}

// table(t, device, rows) -> (pointer, row stride, width): int32 [rows, width], unit
// column stride
PyObject* table(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 3) {
    PyErr_SetString(PyExc_TypeError, "table(tensor, device, rows)");
    return nullptr;
  }
  const long long rows = PyLong_AsLongLong(args[2]);
  if (rows == -1 && PyErr_Occurred()) return nullptr;
  const at::Tensor* t = tensor_of(args[0], at::kInt, args[1]);
  if (!t || t->dim() != 2 || t->size(0) != rows || t->stride(1) != 1) Py_RETURN_NONE;
  const long long width = t->size(1);
  return Py_BuildValue("NLL", pointer(*t), rows > 1 ? (long long)t->stride(0) : width, width);
}

// matrix(t, dtype, device) -> (pointer, rows, columns): contiguous, 2-D
PyObject* matrix(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 3 || !THPDtype_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "matrix(tensor, dtype, device)");
    return nullptr;
  }
  const at::Tensor* t =
      tensor_of(args[0], reinterpret_cast<THPDtype*>(args[1])->scalar_type, args[2]);
  if (!t || t->dim() != 2 || !t->is_contiguous()) Py_RETURN_NONE;
  return Py_BuildValue("NLL", pointer(*t), (long long)t->size(0), (long long)t->size(1));
}

// rows(t, dtype, device) -> (pointer, rows, columns, row stride): 2-D, unit column stride
PyObject* rows(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 3 || !THPDtype_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "rows(tensor, dtype, device)");
    return nullptr;
  }
  const at::Tensor* t =
      tensor_of(args[0], reinterpret_cast<THPDtype*>(args[1])->scalar_type, args[2]);
  if (!t || t->dim() != 2 || (t->size(1) > 1 && t->stride(1) != 1)) Py_RETURN_NONE;
  const long long n = t->size(0), width = t->size(1);
  return Py_BuildValue("NLLL", pointer(*t), n, width, n > 1 ? (long long)t->stride(0) : width);
}

// caches(key, value, device) -> (key pointer, value pointer, blocks, block size, H, D):
// contiguous uint8 [blocks, block size, H, D], of one shape
PyObject* caches(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 3) {
    PyErr_SetString(PyExc_TypeError, "caches(key, value, device)");
    return nullptr;
  }
  const at::Tensor* k = tensor_of(args[0], at::kByte, args[2]);
  const at::Tensor* v = k ? tensor_of(args[1], at::kByte, args[2]) : nullptr;
  if (!v || k->dim() != 4 || !k->is_contiguous() || !v->is_contiguous() ||
      k->sizes() != v->sizes())
    Py_RETURN_NONE;
  return Py_BuildValue("NNLLLL", pointer(*k), pointer(*v), (long long)k->size(0),
                       (long long)k->size(1), (long long)k->size(2), (long long)k->size(3));
}

// Nothing that a tensor's accessors throw leaves a call.
template <PyObject* (*kCall)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  try {
    return kCall(self, args, nargs);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {
    {"vector", (PyCFunction)(void (*)(void))guarded<vector>, METH_FASTCALL, nullptr},
    {"heads", (PyCFunction)(void (*)(void))guarded<heads>, METH_FASTCALL, nullptr},
    {"table", (PyCFunction)(void (*)(void))guarded<table>, METH_FASTCALL, nullptr},
    {"matrix", (PyCFunction)(void (*)(void))guarded<matrix>, METH_FASTCALL, nullptr},
    {"rows", (PyCFunction)(void (*)(void))guarded<rows>, METH_FASTCALL, nullptr},
    {"caches", (PyCFunction)(void (*)(void))guarded<caches>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args(void) { return PyModule_Create(&module); }
