// The small-call path of the Python binding: checks, output allocation and the
// C call of the MX FP4 and query/key functions without Python in between.
//
// Every function returns None for arguments that it does not take as they are
// (another type or layout, an empty size, a status other than Q4_OK); the
// Python function of the same name then goes through its own checks and says
// what is wrong.  The library's entry points come from the binding (bind), so
// that both call the same library.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/headeronly/version.h>

#include <cstdint>

#include "q4.h"

namespace {

decltype(&q4_mx_quantize_rows) quantize_rows_c;
decltype(&q4_mx_dequantize_rows) dequantize_rows_c;
decltype(&q4_linear_w4a4_mx) w4a4_c;
decltype(&q4_w4a4_mx_dynamic_workspace) w4a4_workspace_c;
decltype(&q4_linear_w4a4_mx_dynamic) w4a4_dynamic_c;
decltype(&q4_linear_w4a16_mx) w4a16_c;
decltype(&q4_qk_norm_rope) qk_c;
PyObject *raw_stream;   // device index -> handle of its current stream

PyObject *none() { Py_RETURN_NONE; }

// A dense GPU tensor of dim dimensions, none of them empty, or null.
const at::Tensor *dense(PyObject *o, int64_t dim) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor &t = THPVariable_Unpack(o);
  return t.defined() && t.is_cuda() && t.dim() == dim && t.numel() > 0 && t.is_contiguous() ? &t : nullptr;
}

bool typed(const at::Tensor *t, at::ScalarType a) { return t && t->scalar_type() == a; }
bool floats(const at::Tensor *t) { return typed(t, at::kFloat) || typed(t, at::kBFloat16); }
q4_dtype dt(const at::Tensor &t) { return t.scalar_type() == at::kBFloat16 ? Q4_DT_BF16 : Q4_DT_F32; }

// Codes and scales that belong together; their blocks a row, or 0.
int64_t blocks(const at::Tensor *c, const at::Tensor *s) {
  if (!typed(c, at::kByte) || !typed(s, at::kByte) || c->get_device() != s->get_device()) return 0;
  return c->size(0) == s->size(0) && c->size(1) == 16 * s->size(1) ? s->size(1) : 0;
}

at::Tensor like(const at::Tensor &t, at::IntArrayRef size, at::ScalarType type) {
  return at::empty(size, at::TensorOptions().dtype(type).device(t.device()));
}

// False (with a Python error) if the stream cannot be had.
bool stream_of(const at::Tensor &t, void **st) {
  PyObject *i = PyLong_FromLong(t.get_device());
  PyObject *h = i ? PyObject_CallOneArg(raw_stream, i) : nullptr;
  Py_XDECREF(i);
  if (!h) return false;
  *st = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  return !PyErr_Occurred();
}

PyObject *result(q4_status st, const at::Tensor &y) { return st == Q4_OK ? THPVariable_Wrap(y) : none(); }

bool want_bf16(PyObject *o) { return PyObject_IsTrue(o) == 1; }

// quantize_rows(x) -> (codes, scales)
PyObject *quantize_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor *x = n == 1 ? dense(a[0], 2) : nullptr;
  if (!floats(x)) return none();
  const int64_t M = x->size(0), K = x->size(1), B = (K + 31) / 32;
  void *st;
  if (!stream_of(*x, &st)) return nullptr;
  const at::Tensor c = like(*x, {M, 16 * B}, at::kByte), s = like(*x, {M, B}, at::kByte);
  if (quantize_rows_c(x->const_data_ptr(), dt(*x), M, K, c.mutable_data_ptr<uint8_t>(), s.mutable_data_ptr<uint8_t>(),
                      st) != Q4_OK)
    return none();
  return Py_BuildValue("(NN)", THPVariable_Wrap(c), THPVariable_Wrap(s));
  END_HANDLE_TH_ERRORS
}

// dequantize_rows(codes, scales, K, bf16) -> y
PyObject *dequantize_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4 || !PyLong_Check(a[2])) return none();
  const at::Tensor *c = dense(a[0], 2), *s = dense(a[1], 2);
  const int64_t B = blocks(c, s), K = PyLong_AsLongLong(a[2]);
  if (PyErr_Occurred()) return nullptr;
  if (B == 0 || K <= 0 || (K - 1) / 32 + 1 != B) return none();
  void *st;
  if (!stream_of(*c, &st)) return nullptr;
  const bool bf16 = want_bf16(a[3]);
  const at::Tensor y = like(*c, {c->size(0), K}, bf16 ? at::kBFloat16 : at::kFloat);
  return result(dequantize_rows_c(c->const_data_ptr<uint8_t>(), s->const_data_ptr<uint8_t>(), c->size(0), K,
                                  y.mutable_data_ptr(), dt(y), st),
                y);
  END_HANDLE_TH_ERRORS
}

// w4a4(xq, sx, wq, sw, bf16) -> y
PyObject *w4a4(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5) return none();
  const at::Tensor *xq = dense(a[0], 2), *sx = dense(a[1], 2), *wq = dense(a[2], 2), *sw = dense(a[3], 2);
  const int64_t B = blocks(xq, sx);
  if (B == 0 || blocks(wq, sw) != B || xq->get_device() != wq->get_device()) return none();
  void *st;
  if (!stream_of(*xq, &st)) return nullptr;
  const int64_t M = xq->size(0), N = wq->size(0);
  const at::Tensor y = like(*xq, {M, N}, want_bf16(a[4]) ? at::kBFloat16 : at::kFloat);
  return result(w4a4_c(xq->const_data_ptr<uint8_t>(), sx->const_data_ptr<uint8_t>(), wq->const_data_ptr<uint8_t>(),
                       sw->const_data_ptr<uint8_t>(), y.mutable_data_ptr(), dt(y), M, N, 32 * B, st),
                y);
  END_HANDLE_TH_ERRORS
}

// x [M, K] against weights of as many blocks, on one device
bool fits(const at::Tensor *x, const at::Tensor *wq, const at::Tensor *sw) {
  return x && blocks(wq, sw) == (x->size(1) + 31) / 32 && x->get_device() == wq->get_device();
}

// w4a4_dynamic(x, wq, sw, bf16) -> y
PyObject *w4a4_dynamic(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) return none();
  const at::Tensor *x = dense(a[0], 2), *wq = dense(a[1], 2), *sw = dense(a[2], 2);
  if (!floats(x) || !fits(x, wq, sw)) return none();
  void *st;
  if (!stream_of(*x, &st)) return nullptr;
  const int64_t M = x->size(0), K = x->size(1), N = wq->size(0), need = w4a4_workspace_c(M, K);
  const at::Tensor y = like(*x, {M, N}, want_bf16(a[3]) ? at::kBFloat16 : at::kFloat), ws = like(*x, {need}, at::kByte);
  return result(w4a4_dynamic_c(x->const_data_ptr(), dt(*x), wq->const_data_ptr<uint8_t>(),
                               sw->const_data_ptr<uint8_t>(), y.mutable_data_ptr(), dt(y), M, N, K,
                               ws.mutable_data_ptr(), need, st),
                y);
  END_HANDLE_TH_ERRORS
}

// w4a16(x, wq, sw, bf16) -> y
PyObject *w4a16(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) return none();
  const at::Tensor *x = dense(a[0], 2), *wq = dense(a[1], 2), *sw = dense(a[2], 2);
  if (!typed(x, at::kBFloat16) || !fits(x, wq, sw)) return none();
  void *st;
  if (!stream_of(*x, &st)) return nullptr;
  const int64_t M = x->size(0), N = wq->size(0);
  const at::Tensor y = like(*x, {M, N}, want_bf16(a[3]) ? at::kBFloat16 : at::kFloat);
  return result(w4a16_c(static_cast<const uint16_t *>(x->const_data_ptr()), wq->const_data_ptr<uint8_t>(),
                        sw->const_data_ptr<uint8_t>(), y.mutable_data_ptr(), dt(y), M, N, x->size(1), st),
                y);
  END_HANDLE_TH_ERRORS
}

// Heads [T, H, D] with the D numbers of a head side by side.
const at::Tensor *heads(PyObject *o) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor &t = THPVariable_Unpack(o);
  return t.defined() && t.is_cuda() && floats(&t) && t.dim() == 3 && t.numel() > 0 && t.stride(2) == 1 ? &t : nullptr;
}

// qk_norm_rope(q, k, q_gain, k_gain, positions, cos_sin, eps, pairs, type 0/1 or -1 for q's) -> (q_out, k_out);
// keys and both gains given
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) return none();
  const at::Tensor *q = heads(a[0]), *k = heads(a[1]);
  const at::Tensor *gq = dense(a[2], 1), *gk = dense(a[3], 1), *pos = dense(a[4], 1), *cs = dense(a[5], 2);
  if (!q || !k || !floats(gq) || !typed(gk, gq->scalar_type()) || !typed(pos, at::kLong) || !typed(cs, at::kFloat))
    return none();
  const int64_t T = q->size(0), Hq = q->size(1), Hk = k->size(1), D = q->size(2), dev = q->get_device();
  if (k->size(0) != T || k->size(2) != D || k->scalar_type() != q->scalar_type() || gq->size(0) != D ||
      gk->size(0) != D || pos->size(0) != T)
    return none();
  for (const at::Tensor *t : {k, gq, gk, pos, cs})
    if (t->get_device() != dev) return none();
  const double eps = PyFloat_AsDouble(a[6]);
  const long pairs = PyLong_AsLong(a[7]), type = PyLong_AsLong(a[8]);
  void *st;
  if (PyErr_Occurred() || !stream_of(*q, &st)) return nullptr;
  const at::ScalarType out = type < 0 ? q->scalar_type() : type == 1 ? at::kBFloat16 : at::kFloat;
  const at::Tensor qo = like(*q, {T, Hq, D}, out), ko = like(*q, {T, Hk, D}, out);
  if (qk_c(q->const_data_ptr(), q->stride(0), q->stride(1), k->const_data_ptr(), k->stride(0), k->stride(1), dt(*q),
           gq->const_data_ptr(), gk->const_data_ptr(), dt(*gq), pos->const_data_ptr<int64_t>(),
           cs->const_data_ptr<float>(), qo.mutable_data_ptr(), ko.mutable_data_ptr(), dt(qo), T, Hq, Hk, D, cs->size(1),
           cs->size(0), static_cast<float>(eps), static_cast<q4_rope_pairs>(pairs), st) != Q4_OK)
    return none();
  return Py_BuildValue("(NN)", THPVariable_Wrap(qo), THPVariable_Wrap(ko));
  END_HANDLE_TH_ERRORS
}

// bind(raw_stream, {name: address}): the library's entry points
PyObject *bind(PyObject *, PyObject *args) {
  PyObject *f, *d;
  if (!PyArg_ParseTuple(args, "OO!", &f, &PyDict_Type, &d)) return nullptr;
  bool ok = true;
  auto get = [&](const char *name) -> void * {
    PyObject *o = PyDict_GetItemString(d, name);
    void *p = o ? PyLong_AsVoidPtr(o) : nullptr;
    ok = ok && p;
    return p;
  };
  quantize_rows_c = reinterpret_cast<decltype(quantize_rows_c)>(get("q4_mx_quantize_rows"));
  dequantize_rows_c = reinterpret_cast<decltype(dequantize_rows_c)>(get("q4_mx_dequantize_rows"));
  w4a4_c = reinterpret_cast<decltype(w4a4_c)>(get("q4_linear_w4a4_mx"));
  w4a4_workspace_c = reinterpret_cast<decltype(w4a4_workspace_c)>(get("q4_w4a4_mx_dynamic_workspace"));
  w4a4_dynamic_c = reinterpret_cast<decltype(w4a4_dynamic_c)>(get("q4_linear_w4a4_mx_dynamic"));
  w4a16_c = reinterpret_cast<decltype(w4a16_c)>(get("q4_linear_w4a16_mx"));
  qk_c = reinterpret_cast<decltype(qk_c)>(get("q4_qk_norm_rope"));
  if (!ok) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point is missing");
    return nullptr;
  }
  Py_INCREF(f);
  Py_XSETREF(raw_stream, f);
  return none();
}

#define Q4_FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr}, Q4_FAST(quantize_rows), Q4_FAST(dequantize_rows),
                         Q4_FAST(w4a4), Q4_FAST(w4a4_dynamic), Q4_FAST(w4a16), Q4_FAST(qk_norm_rope),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "q4_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch and Python whose headers this was compiled with; the
// binding does not call a module that was built for others.
PyMODINIT_FUNC PyInit_q4_torch() {
  PyObject *m = PyModule_Create(&module);
  PyObject *v = m ? PyUnicode_FromFormat("torch %d.%d.%d, Python %d.%d", TORCH_VERSION_MAJOR, TORCH_VERSION_MINOR,
                                         TORCH_VERSION_PATCH, PY_MAJOR_VERSION, PY_MINOR_VERSION)
                  : nullptr;
  const bool ok = v && PyObject_SetAttrString(m, "built_for", v) == 0;
  Py_XDECREF(v);
  if (!ok) Py_CLEAR(m);
  return m;
}
