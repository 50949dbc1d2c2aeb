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

// ---- whole calls ---------------------------------------------------------------
// The step's calls with arguments as they should be: read, passed on and made here,
// where even the steps between Python and the library cost more than a small step's
// kernel.  They take the address of the library's function and the stream, and
// return its status, or None if an argument is not as expected.

struct Rows {
  void* p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
};

bool rows_of(PyObject* o, at::ScalarType type, PyObject* device, Rows* r) {
  const at::Tensor* t = tensor_of(o, type, device);
  if (!t || t->dim() != 2 || (t->size(1) > 1 && t->stride(1) != 1)) return false;
  *r = {t->data_ptr(), t->size(0), t->size(1), t->size(0) > 1 ? t->stride(0) : t->size(1)};
  return true;
}

bool rows_of(PyObject* o, at::ScalarType type, PyObject* device, int64_t rows, int64_t cols,
             Rows* r) {
  return rows_of(o, type, device, r) && r->rows == rows && r->cols == cols;
}

bool whole_of(PyObject* o, at::ScalarType type, PyObject* device, int64_t rows, int64_t cols,
              void** p) {
  const at::Tensor* t = tensor_of(o, type, device);
  if (!t || t->dim() != 2 || !t->is_contiguous() || t->size(0) != rows || t->size(1) != cols)
    return false;
  *p = t->data_ptr();
  return true;
}

bool vector_of(PyObject* o, at::ScalarType type, PyObject* device, int64_t n, void** p) {
  const at::Tensor* t = tensor_of(o, type, device);
  if (!t || t->dim() != 1 || t->size(0) != n || !t->is_contiguous()) return false;
  *p = t->data_ptr();
  return true;
}

bool workspace_of(PyObject* o, PyObject* device, void** p, size_t* n) {
  *p = nullptr;
  *n = 0;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor_of(o, at::kByte, device);
  if (!t || !t->is_contiguous()) return false;
  *p = t->data_ptr();
  *n = (size_t)t->numel();
  return true;
}

// [T, H, D] bf16, not empty, each token's heads contiguous
struct Heads {
  void* p = nullptr;
  int64_t T = 0, H = 0, D = 0, ld = 0;
};

bool heads_of(PyObject* o, PyObject* device, Heads* h) {
  const at::Tensor* t = tensor_of(o, at::kBFloat16, device);
  if (!t || t->dim() != 3 || t->numel() == 0) return false;
  *h = {t->data_ptr(), t->size(0), t->size(1), t->size(2),
        t->size(0) > 1 ? t->stride(0) : t->size(1) * t->size(2)};
  return t->stride(2) == 1 && (h->H == 1 || t->stride(1) == h->D);
}

template <typename F, typename... A>
PyObject* made(PyObject* fn, A... args) {
  F f = reinterpret_cast<F>(PyLong_AsVoidPtr(fn));
  if (!f) return nullptr;
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f(args...);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

bool counted(Py_ssize_t nargs, Py_ssize_t want) {
  if (nargs == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

using c_vp = const void*;

// int4_linear(fn, x, codes, scales, zeros, out, workspace, device, stream)
PyObject* int4_linear(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (!counted(nargs, 9)) return nullptr;
  PyObject* dev = args[7];
  Rows x, out;
  if (!rows_of(args[1], at::kBFloat16, dev, &x)) Py_RETURN_NONE;
  const at::Tensor* codes = tensor_of(args[2], at::kByte, dev);
  const at::Tensor* scales = tensor_of(args[3], at::kFloat, dev);
  if (!codes || codes->dim() != 2 || !codes->is_contiguous() || !scales || scales->dim() != 2 ||
      !scales->is_contiguous())
    Py_RETURN_NONE;
  const int64_t n = codes->size(0), k = x.cols, groups = scales->size(1);
  if (codes->size(1) * 2 != k || scales->size(0) != n || groups == 0 || k % groups != 0)
    Py_RETURN_NONE;
  void *zeros = nullptr, *ws;
  size_t ws_bytes;
  if (args[4] != Py_None && !whole_of(args[4], at::kByte, dev, n, groups, &zeros)) Py_RETURN_NONE;
  if (!rows_of(args[5], at::kBFloat16, dev, x.rows, n, &out) ||
      !workspace_of(args[6], dev, &ws, &ws_bytes))
    Py_RETURN_NONE;
  typedef int (*Fn)(c_vp, int64_t, c_vp, c_vp, c_vp, int64_t, void*, int64_t, int64_t, int64_t,
                    int64_t, void*, size_t, void*);
  return made<Fn>(args[0], x.p, x.ld, codes->data_ptr(), scales->data_ptr(), zeros, k / groups, out.p,
                  out.ld, x.rows, n, k, ws, ws_bytes, PyLong_AsVoidPtr(args[8]));
}

// add_rms_norm(fn, x, residual, residual_out, weight, eps, out, q, scales, mode, scale, device,
// stream): residual, residual_out, out, q, scales and scale may be None; mode as in the library
PyObject* add_rms_norm(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (!counted(nargs, 13)) return nullptr;
  PyObject* dev = args[11];
  const double eps = PyFloat_AsDouble(args[5]);
  const long mode = PyLong_AsLong(args[9]);
  if (PyErr_Occurred()) return nullptr;
  Rows x, r, ro, y, q, s;
  if (!rows_of(args[1], at::kBFloat16, dev, &x)) Py_RETURN_NONE;
  const int64_t T = x.rows, H = x.cols;
  if (args[2] != Py_None && (!rows_of(args[2], at::kBFloat16, dev, T, H, &r) ||
                             !rows_of(args[3], at::kBFloat16, dev, T, H, &ro)))
    Py_RETURN_NONE;
  if (args[6] != Py_None && !rows_of(args[6], at::kBFloat16, dev, T, H, &y)) Py_RETURN_NONE;
  if (args[7] != Py_None && !rows_of(args[7], at::kByte, dev, T, H, &q)) Py_RETURN_NONE;
  void *w, *scale = nullptr;
  if (!vector_of(args[4], at::kBFloat16, dev, H, &w)) Py_RETURN_NONE;
  if (args[8] != Py_None) {                       // [T, H / 128], or [T]
    const at::Tensor* t = tensor_of(args[8], at::kFloat, dev);
    if (!t) Py_RETURN_NONE;
    if (t->dim() == 1 && mode == 2 && t->size(0) == T)
      s = {t->data_ptr(), T, 1, T > 1 ? t->stride(0) : 1};
    else if (mode != 0 || !rows_of(args[8], at::kFloat, dev, T, H / 128, &s))
      Py_RETURN_NONE;
  }
  if (args[10] != Py_None && !vector_of(args[10], at::kFloat, dev, 1, &scale)) Py_RETURN_NONE;
  typedef int (*Fn)(c_vp, int64_t, c_vp, int64_t, void*, int64_t, c_vp, float, void*, int64_t, void*,
                    int64_t, void*, int64_t, int, c_vp, int64_t, int64_t, void*);
  return made<Fn>(args[0], x.p, x.ld, r.p, r.ld, ro.p, ro.ld, w, (float)eps, y.p, y.ld, q.p, q.ld, s.p,
                  s.ld, (int)mode, scale, T, H, PyLong_AsVoidPtr(args[12]));
}

// qk_norm_mrope_cache(fn, query, key, value, q_weight, k_weight, eps, cos_sin, interleaved,
// positions, sections, order, slots, query_out, key_cache, value_cache, k_scale, v_scale, device,
// stream): sections a tuple of whole numbers
PyObject* qk_norm_mrope_cache(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (!counted(nargs, 20)) return nullptr;
  PyObject* dev = args[18];
  const double eps = PyFloat_AsDouble(args[6]);
  const long inter = PyLong_AsLong(args[8]), order = PyLong_AsLong(args[11]);
  if (PyErr_Occurred()) return nullptr;
  if (!PyTuple_Check(args[10]) || PyTuple_GET_SIZE(args[10]) > 4) Py_RETURN_NONE;
  const int64_t A = PyTuple_GET_SIZE(args[10]);
  int64_t sections[4] = {};
  for (int64_t i = 0; i < A; ++i) {
    sections[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(args[10], i));
    if (PyErr_Occurred()) return nullptr;
  }
  Heads q, k, v, o;
  if (!heads_of(args[1], dev, &q) || !heads_of(args[2], dev, &k) || !heads_of(args[3], dev, &v) ||
      !heads_of(args[13], dev, &o))
    Py_RETURN_NONE;
  const int64_t T = q.T, Hq = q.H, Hk = k.H, D = q.D;
  if (k.T != T || k.D != D || v.T != T || v.H != Hk || v.D != D || o.T != T || o.H != Hq || o.D != D)
    Py_RETURN_NONE;
  void *qw, *kw, *slots, *ks, *vs;
  if (!vector_of(args[4], at::kBFloat16, dev, D, &qw) || !vector_of(args[5], at::kBFloat16, dev, D, &kw) ||
      !vector_of(args[12], at::kLong, dev, T, &slots) || !vector_of(args[16], at::kFloat, dev, 1, &ks) ||
      !vector_of(args[17], at::kFloat, dev, 1, &vs))
    Py_RETURN_NONE;
  const at::Tensor* cs = tensor_of(args[7], at::kFloat, dev);
  if (!cs || cs->dim() != 2 || !cs->is_contiguous()) Py_RETURN_NONE;
  Rows pos;
  if (!rows_of(args[9], at::kLong, dev, A, T, &pos)) Py_RETURN_NONE;
  const at::Tensor* kc = tensor_of(args[14], at::kByte, dev);
  const at::Tensor* vc = tensor_of(args[15], at::kByte, dev);
  if (!kc || !vc || kc->dim() != 4 || !kc->is_contiguous() || !vc->is_contiguous() ||
      kc->sizes() != vc->sizes() || kc->size(2) != Hk || kc->size(3) != D)
    Py_RETURN_NONE;
  typedef int (*Fn)(c_vp, int64_t, c_vp, int64_t, c_vp, int64_t, c_vp, c_vp, float, c_vp, int64_t,
                    int64_t, int, c_vp, int64_t, int64_t, const int64_t*, int, c_vp, int64_t, int64_t,
                    int64_t, int64_t, void*, int64_t, void*, void*, int64_t, int64_t, c_vp, c_vp, void*);
  return made<Fn>(args[0], q.p, q.ld, k.p, k.ld, v.p, v.ld, qw, kw, (float)eps, cs->data_ptr(),
                  cs->size(0), cs->size(1), (int)inter, pos.p, pos.ld, A, (const int64_t*)sections,
                  (int)order, slots, T, Hq, Hk, D, o.p, o.ld, kc->data_ptr(), vc->data_ptr(), kc->size(0),
                  kc->size(1), ks, vs, PyLong_AsVoidPtr(args[19]));
}

// token_logprobs(fn, logits, tokens, scale, k, logprobs, ranks, entropy, lse, top_logprobs, top_ids,
// workspace, device, stream)
PyObject* token_logprobs(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (!counted(nargs, 14)) return nullptr;
  PyObject* dev = args[12];
  const double scale = PyFloat_AsDouble(args[3]);
  const long long k = PyLong_AsLongLong(args[4]);
  if (PyErr_Occurred()) return nullptr;
  Rows x;
  int type = 0;
  if (!rows_of(args[1], at::kBFloat16, dev, &x)) {
    type = 1;
    if (!rows_of(args[1], at::kFloat, dev, &x)) Py_RETURN_NONE;
  }
  const int64_t T = x.rows;
  void *tokens, *lp, *ranks, *ent, *lse, *top, *ids, *ws;
  size_t ws_bytes;
  if (!vector_of(args[2], at::kLong, dev, T, &tokens) || !vector_of(args[5], at::kFloat, dev, T, &lp) ||
      !vector_of(args[6], at::kInt, dev, T, &ranks) || !vector_of(args[7], at::kFloat, dev, T, &ent) ||
      !vector_of(args[8], at::kFloat, dev, T, &lse) ||
      !whole_of(args[9], at::kFloat, dev, T, k, &top) || !whole_of(args[10], at::kInt, dev, T, k, &ids) ||
      !workspace_of(args[11], dev, &ws, &ws_bytes))
    Py_RETURN_NONE;
  typedef int (*Fn)(c_vp, int, int64_t, c_vp, float, int64_t, int64_t, int64_t, void*, void*, void*,
                    void*, void*, void*, void*, size_t, void*);
  return made<Fn>(args[0], x.p, type, x.ld, tokens, (float)scale, T, x.cols, (int64_t)k, lp, ranks, ent,
                  lse, top, ids, ws, ws_bytes, PyLong_AsVoidPtr(args[13]));
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
    {"int4_linear", (PyCFunction)(void (*)(void))guarded<int4_linear>, METH_FASTCALL, nullptr},
    {"add_rms_norm", (PyCFunction)(void (*)(void))guarded<add_rms_norm>, METH_FASTCALL, nullptr},
    {"qk_norm_mrope_cache", (PyCFunction)(void (*)(void))guarded<qk_norm_mrope_cache>, METH_FASTCALL,
     nullptr},
    {"token_logprobs", (PyCFunction)(void (*)(void))guarded<token_logprobs>, METH_FASTCALL, nullptr},
    {"caches", (PyCFunction)(void (*)(void))guarded<caches>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args(void) { return PyModule_Create(&module); }
