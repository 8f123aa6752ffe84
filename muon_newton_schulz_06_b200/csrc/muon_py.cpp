// Argument marshalling of the 8-bit operators for the Python binding: tensors, Fp8Matrix and
// Fp8Product objects into the C structs of muon.h, and the call.  The same checks and
// messages as the rest of the binding; no arithmetic.  A small call is bound by the host (a
// product of 64 x 512 x 512 runs 5 us on the GPU, and building its structs through ctypes
// took as long), so these calls do not go through ctypes.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <vector>

#include "muon.h"

namespace {

// Set once by setup(): the types and functions that the binding hands over.
PyObject *g_tensor, *g_bf16, *g_f32, *g_matrix, *g_product, *g_stream;
PyObject *s_is_cuda, *s_shape, *s_stride, *s_data_ptr, *s_dtype, *s_addr, *s_device, *s_value;
PyObject *s_a, *s_b, *s_out, *s_trans_a, *s_trans_b, *s_add, *s_epilogue, *s_saved;
PyObject* g_epilogues;

decltype(&muon_fp8_quantize) f_quantize;
decltype(&muon_fp8_dequantize) f_dequantize;
decltype(&muon_fp8_act_backward) f_act_backward;
decltype(&muon_fp8_matmul) f_matmul;

// Owned reference, released at the end of the scope.
struct Ref {
  PyObject* p;
  explicit Ref(PyObject* q) : p(q) {}
  Ref(const Ref&) = delete;
  ~Ref() { Py_XDECREF(p); }
  explicit operator bool() const { return p != nullptr; }
};

bool is_instance(PyObject* o, PyObject* type) {
  return PyObject_TypeCheck(o, reinterpret_cast<PyTypeObject*>(type)) != 0;
}

// A bf16 / float32 CUDA tensor with consecutive columns.
bool dense(PyObject* t, const char* name, muon_dense* d) {
  if (!is_instance(t, g_tensor)) {
    PyErr_Format(PyExc_TypeError, "%s must be a CUDA tensor", name);
    return false;
  }
  Ref cuda(PyObject_GetAttr(t, s_is_cuda));
  if (!cuda) return false;
  if (cuda.p != Py_True) {
    PyErr_Format(PyExc_TypeError, "%s must be a CUDA tensor", name);
    return false;
  }
  Ref shape(PyObject_GetAttr(t, s_shape));
  if (!shape) return false;
  if (!PyTuple_Check(shape.p) || PyTuple_GET_SIZE(shape.p) != 2) {
    PyErr_Format(PyExc_ValueError, "%s must be a 2-D tensor", name);
    return false;
  }
  Ref stride(PyObject_CallMethodNoArgs(t, s_stride));
  if (!stride) return false;
  d->rows = PyLong_AsLongLong(PyTuple_GET_ITEM(shape.p, 0));
  d->cols = PyLong_AsLongLong(PyTuple_GET_ITEM(shape.p, 1));
  const int64_t ld = PyLong_AsLongLong(PyTuple_GET_ITEM(stride.p, 0));
  const int64_t step = PyLong_AsLongLong(PyTuple_GET_ITEM(stride.p, 1));
  if (PyErr_Occurred()) return false;
  if (step != 1 && d->cols > 1 && d->rows > 0) {
    PyErr_Format(PyExc_ValueError, "%s must have consecutive columns", name);
    return false;
  }
  d->ld = d->rows > 1 ? ld : d->cols;
  Ref dtype(PyObject_GetAttr(t, s_dtype));
  if (!dtype) return false;
  if (dtype.p == g_bf16) {
    d->dtype = MUON_BF16;
  } else if (dtype.p == g_f32) {
    d->dtype = MUON_F32;
  } else {
    PyErr_Format(PyExc_TypeError, "unsupported dtype %S; use float32 or bfloat16", dtype.p);
    return false;
  }
  Ref ptr(PyObject_CallMethodNoArgs(t, s_data_ptr));
  if (!ptr) return false;
  d->data = PyLong_AsVoidPtr(ptr.p);
  return !PyErr_Occurred();
}

// The struct inside an Fp8Matrix.
bool fp8(PyObject* m, const char* name, muon_fp8_matrix* out) {
  if (!is_instance(m, g_matrix)) {
    PyErr_Format(PyExc_TypeError, "%s must be an Fp8Matrix", name);
    return false;
  }
  Ref addr(PyObject_GetAttr(m, s_addr));
  if (!addr) return false;
  const void* p = PyLong_AsVoidPtr(addr.p);
  if (p == nullptr) return false;
  *out = *static_cast<const muon_fp8_matrix*>(p);
  return true;
}

bool handle_of(PyObject* h, muon_handle_t* out) {
  *out = nullptr;
  if (h == Py_None) return true;
  Ref v(PyObject_GetAttr(h, s_value));  // a ctypes.c_void_p
  if (!v) return false;
  if (v.p != Py_None) *out = static_cast<muon_handle_t>(PyLong_AsVoidPtr(v.p));
  return !PyErr_Occurred();
}

// The stream to use: the caller's, or the current one of `of`'s device.
bool stream_of(PyObject* stream, PyObject* of, void** out) {
  Ref device(PyObject_GetAttr(of, s_device));
  if (!device) return false;
  PyObject* args[2] = {stream, device.p};
  Ref s(PyObject_Vectorcall(g_stream, args, 2, nullptr));
  if (!s) return false;
  *out = PyLong_AsVoidPtr(s.p);
  return !PyErr_Occurred();
}

// A sequence as a list or tuple.
struct Items {
  Ref seq;
  Py_ssize_t n;
  explicit Items(PyObject* o) : seq(PySequence_Fast(o, "expected a sequence")), n(seq ? PySequence_Fast_GET_SIZE(seq.p) : -1) {}
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq.p, i); }
};

bool same_length(const Items& a, const Items& b, const char* names) {
  if (a.n < 0 || b.n < 0) return false;
  if (a.n != b.n) {
    PyErr_Format(PyExc_ValueError, "%s must have the same length", names);
    return false;
  }
  return true;
}

// quantize(handle, xs, outs, activation, stream) -> status
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 5) return PyErr_Format(PyExc_TypeError, "quantize takes 5 arguments");
  Items xs(a[1]), outs(a[2]);
  if (!same_length(xs, outs, "xs and outs")) return nullptr;
  if (xs.n == 0) return PyLong_FromLong(MUON_OK);
  std::vector<muon_dense> x((size_t)xs.n);
  std::vector<muon_fp8_matrix> o((size_t)xs.n);
  for (Py_ssize_t i = 0; i < xs.n; ++i)
    if (!dense(xs[i], "x", &x[(size_t)i]) || !fp8(outs[i], "out", &o[(size_t)i])) return nullptr;
  muon_handle_t h;
  void* st;
  const long act = PyLong_AsLong(a[3]);
  if (PyErr_Occurred() || !handle_of(a[0], &h) || !stream_of(a[4], outs[0], &st)) return nullptr;
  muon_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f_quantize(h, x.data(), o.data(), (int)xs.n, (muon_activation)act, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(s);
}

// dequantize(handle, xs, outs, stream) -> status
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 4) return PyErr_Format(PyExc_TypeError, "dequantize takes 4 arguments");
  Items xs(a[1]), outs(a[2]);
  if (!same_length(xs, outs, "xs and outs")) return nullptr;
  if (xs.n == 0) return PyLong_FromLong(MUON_OK);
  std::vector<muon_fp8_matrix> x((size_t)xs.n);
  std::vector<muon_dense> o((size_t)xs.n);
  for (Py_ssize_t i = 0; i < xs.n; ++i)
    if (!fp8(xs[i], "x", &x[(size_t)i]) || !dense(outs[i], "out", &o[(size_t)i])) return nullptr;
  muon_handle_t h;
  void* st;
  if (!handle_of(a[0], &h) || !stream_of(a[3], xs[0], &st)) return nullptr;
  muon_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f_dequantize(h, x.data(), o.data(), (int)xs.n, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(s);
}

// act_backward(handle, dys, saved, dus, activation, stream) -> status
PyObject* act_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 6) return PyErr_Format(PyExc_TypeError, "act_backward takes 6 arguments");
  Items dys(a[1]), saved(a[2]), dus(a[3]);
  if (!same_length(dys, saved, "dys, saved and dus") || !same_length(dys, dus, "dys, saved and dus")) return nullptr;
  const Py_ssize_t n = dys.n;
  if (n == 0) return PyLong_FromLong(MUON_OK);
  std::vector<muon_dense> dy((size_t)n), du((size_t)n);
  std::vector<muon_fp8_matrix> sv((size_t)n), du8((size_t)n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (!dense(dys[i], "dy", &dy[(size_t)i]) || !fp8(saved[i], "saved", &sv[(size_t)i])) return nullptr;
    if (is_instance(dus[i], g_matrix) ? !fp8(dus[i], "du", &du8[(size_t)i]) : !dense(dus[i], "du", &du[(size_t)i]))
      return nullptr;
  }
  muon_handle_t h;
  void* st;
  const long act = PyLong_AsLong(a[4]);
  if (PyErr_Occurred() || !handle_of(a[0], &h) || !stream_of(a[5], saved[0], &st)) return nullptr;
  muon_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f_act_backward(h, dy.data(), sv.data(), du.data(), du8.data(), (int)n, (muon_activation)act, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(s);
}

bool truth(PyObject* p, PyObject* name, int* out) {
  Ref v(PyObject_GetAttr(p, name));
  if (!v) return false;
  const int t = PyObject_IsTrue(v.p);
  if (t < 0) return false;
  *out = t;
  return true;
}

bool product(PyObject* p, muon_fp8_product* q, PyObject** first) {
  if (!is_instance(p, g_product)) {
    PyErr_SetString(PyExc_TypeError, "products must be Fp8Product objects");
    return false;
  }
  Ref a(PyObject_GetAttr(p, s_a)), b(PyObject_GetAttr(p, s_b)), out(PyObject_GetAttr(p, s_out));
  Ref add(PyObject_GetAttr(p, s_add)), epi(PyObject_GetAttr(p, s_epilogue)), saved(PyObject_GetAttr(p, s_saved));
  if (!a || !b || !out || !add || !epi || !saved) return false;
  if (!fp8(a.p, "a", &q->a) || !fp8(b.p, "b", &q->b)) return false;
  *first = a.p;  // kept alive by the product
  if (!truth(p, s_trans_a, &q->trans_a) || !truth(p, s_trans_b, &q->trans_b)) return false;
  if (is_instance(out.p, g_matrix) ? !fp8(out.p, "out", &q->d8) : !dense(out.p, "out", &q->d)) return false;
  if (add.p != Py_None && !dense(add.p, "add", &q->c)) return false;
  // a tensor without entries has no address, which would say that there is no addend: any other one
  // leaves its shape to the call's checks, which touch no memory of such a matrix
  if (add.p != Py_None && q->c.data == nullptr) q->c.data = reinterpret_cast<void*>(static_cast<uintptr_t>(256));
  PyObject* code = PyDict_GetItemWithError(g_epilogues, epi.p);  // borrowed
  if (code == nullptr) {
    if (!PyErr_Occurred()) {
      Ref names(PySequence_List(g_epilogues));
      if (names && PyList_Sort(names.p) == 0)
        PyErr_Format(PyExc_ValueError, "unknown epilogue %R; use one of %R", epi.p, names.p);
    }
    return false;
  }
  q->epilogue = (muon_fp8_epilogue)PyLong_AsLong(code);
  if ((saved.p != Py_None) != (q->epilogue == MUON_EPI_RELU2_BACKWARD)) {
    PyErr_SetString(PyExc_ValueError, "saved belongs to the relu2_backward epilogue, which needs it");
    return false;
  }
  return saved.p == Py_None || fp8(saved.p, "saved", &q->saved);
}

// matmul(handle, products, stream) -> status
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 3) return PyErr_Format(PyExc_TypeError, "matmul takes 3 arguments");
  Items ps(a[1]);
  if (ps.n < 0) return nullptr;
  if (ps.n == 0) return PyLong_FromLong(MUON_OK);
  std::vector<muon_fp8_product> q((size_t)ps.n);
  PyObject* first = nullptr;
  for (Py_ssize_t i = 0; i < ps.n; ++i) {
    PyObject* m = nullptr;
    if (!product(ps[i], &q[(size_t)i], &m)) return nullptr;
    if (i == 0) first = m;
  }
  muon_handle_t h;
  void* st;
  if (!handle_of(a[0], &h) || !stream_of(a[2], first, &st)) return nullptr;
  muon_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f_matmul(h, q.data(), (int)ps.n, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(s);
}

// setup(torch.Tensor, torch.bfloat16, torch.float32, Fp8Matrix, Fp8Product, stream function,
//       {epilogue name: code}, (addresses of the four functions))
PyObject* setup(PyObject*, PyObject* args) {
  PyObject *t, *bf16, *f32, *m, *p, *st, *epi;
  unsigned long long q, d, ab, mm;
  if (!PyArg_ParseTuple(args, "OOOOOOO(KKKK)", &t, &bf16, &f32, &m, &p, &st, &epi, &q, &d, &ab, &mm)) return nullptr;
  PyObject** slots[] = {&g_tensor, &g_bf16, &g_f32, &g_matrix, &g_product, &g_stream, &g_epilogues};
  PyObject* values[] = {t, bf16, f32, m, p, st, epi};
  for (int i = 0; i < 7; ++i) {
    Py_INCREF(values[i]);
    Py_XDECREF(*slots[i]);
    *slots[i] = values[i];
  }
  f_quantize = reinterpret_cast<decltype(f_quantize)>((uintptr_t)q);
  f_dequantize = reinterpret_cast<decltype(f_dequantize)>((uintptr_t)d);
  f_act_backward = reinterpret_cast<decltype(f_act_backward)>((uintptr_t)ab);
  f_matmul = reinterpret_cast<decltype(f_matmul)>((uintptr_t)mm);
  Py_RETURN_NONE;
}

// A C++ exception (out of memory) must not cross into the interpreter.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (...) {
    return PyErr_NoMemory();
  }
}

PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, nullptr},
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<quantize>)), METH_FASTCALL, nullptr},
    {"dequantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<dequantize>)), METH_FASTCALL, nullptr},
    {"act_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<act_backward>)), METH_FASTCALL,
     nullptr},
    {"matmul", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<matmul>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_muon_py", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__muon_py(void) {
  const struct {
    PyObject** slot;
    const char* name;
  } names[] = {{&s_is_cuda, "is_cuda"}, {&s_shape, "shape"},     {&s_stride, "stride"},   {&s_data_ptr, "data_ptr"},
               {&s_dtype, "dtype"},     {&s_addr, "_addr"},      {&s_device, "device"},   {&s_value, "value"},
               {&s_a, "a"},             {&s_b, "b"},             {&s_out, "out"},         {&s_trans_a, "trans_a"},
               {&s_trans_b, "trans_b"}, {&s_add, "add"},         {&s_epilogue, "epilogue"}, {&s_saved, "saved"}};
  for (const auto& n : names)
    if ((*n.slot = PyUnicode_InternFromString(n.name)) == nullptr) return nullptr;
  return PyModule_Create(&module);
}
