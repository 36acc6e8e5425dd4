// The small-call path of the Python binding: checks, output allocation and the
// C call of the MX FP4, query/key, row norm, cache and attention functions
// without Python in between.
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

#include <cmath>
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
decltype(&q8_rmsnorm_rows) rmsnorm_c;
decltype(&q8_kv_append) append_c;
decltype(&q8_kv_read) read_c;
decltype(&q8_attention_workspace) attention_workspace_c;
decltype(&q8_attention) attention_c;
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

// rmsnorm_rows(x, gain or None, residual or None, eps, total or None) -> (codes, scales, total or None)
PyObject *rmsnorm_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor *x = n == 5 ? dense(a[0], 2) : nullptr;
  if (!floats(x)) return none();
  const at::Tensor *g = nullptr, *r = nullptr;
  const int64_t M = x->size(0), K = x->size(1), dev = x->get_device();
  if (a[1] != Py_None && (!floats(g = dense(a[1], 1)) || g->size(0) != K || g->get_device() != dev)) return none();
  auto fits_x = [&](const at::Tensor *t) {
    return typed(t, x->scalar_type()) && t->size(0) == M && t->size(1) == K && t->get_device() == dev;
  };
  if (a[2] != Py_None && !fits_x(r = dense(a[2], 2))) return none();
  if (a[4] != Py_None && (!r || !fits_x(dense(a[4], 2)))) return none();
  const double eps = PyFloat_AsDouble(a[3]);
  void *st;
  if (PyErr_Occurred() || !stream_of(*x, &st)) return nullptr;
  const at::Tensor q = like(*x, {M, K}, at::kChar), s = like(*x, {M}, at::kFloat);
  at::Tensor sum;
  if (a[4] != Py_None) sum = THPVariable_Unpack(a[4]);
  else if (r) sum = like(*x, {M, K}, x->scalar_type());
  if (rmsnorm_c(x->const_data_ptr(), r ? r->const_data_ptr() : nullptr, dt(*x), g ? g->const_data_ptr() : nullptr,
                g ? dt(*g) : Q4_DT_F32, static_cast<float>(eps), M, K, r ? sum.mutable_data_ptr() : nullptr,
                q.mutable_data_ptr<int8_t>(), s.mutable_data_ptr<float>(), st) != Q4_OK)
    return none();
  return Py_BuildValue("(NNN)", THPVariable_Wrap(q), THPVariable_Wrap(s), r ? THPVariable_Wrap(sum) : none());
  END_HANDLE_TH_ERRORS
}

// A cache (a tuple of four tensors) with a call's pages, starts and lengths; false for what is not taken.
bool cache_of(PyObject *o, PyObject *pages, PyObject *starts, PyObject *lengths, q8_kv_cache *c, const int32_t **st,
              const int32_t **len, const at::Tensor **first) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) return false;
  const at::Tensor *k = dense(PyTuple_GET_ITEM(o, 0), 6), *v = dense(PyTuple_GET_ITEM(o, 1), 5);
  const at::Tensor *ks = dense(PyTuple_GET_ITEM(o, 2), 3), *vs = dense(PyTuple_GET_ITEM(o, 3), 3);
  const at::Tensor *p = dense(pages, 2), *s = dense(starts, 1), *l = dense(lengths, 1);
  if (!typed(k, at::kChar) || !typed(v, at::kChar) || !typed(ks, at::kByte) || !typed(vs, at::kByte) ||
      !typed(p, at::kInt) || !typed(s, at::kInt) || !typed(l, at::kInt))
    return false;
  const int64_t P = k->size(0), H = k->size(1), B = k->size(2), C = k->size(3), N = l->size(0);
  if (k->size(4) != 16 || k->size(5) != 16 || v->size(0) != P || v->size(1) != H || v->size(2) != B ||
      v->size(3) != 16 * C || v->size(4) != 16 || p->size(0) != N || s->size(0) != N + 1)
    return false;
  for (const at::Tensor *t : {ks, vs})
    if (t->size(0) != P || t->size(1) != H || t->size(2) != B) return false;
  for (const at::Tensor *t : {v, ks, vs, p, s, l})
    if (t->get_device() != k->get_device()) return false;
  *c = {k->mutable_data_ptr<int8_t>(), v->mutable_data_ptr<int8_t>(), ks->mutable_data_ptr<uint8_t>(),
        vs->mutable_data_ptr<uint8_t>(), p->const_data_ptr<int32_t>(), P, 16 * B, H, 16 * C, N, p->size(1)};
  *st = s->const_data_ptr<int32_t>();
  *len = l->const_data_ptr<int32_t>();
  *first = k;
  return true;
}

bool heads_of(const at::Tensor *t, int64_t T, int64_t D, int64_t dev) {
  return t && t->size(0) == T && t->size(2) == D && t->get_device() == dev;
}

// kv_append(cache, pages, starts, lengths, k, v, q, cos_sin, k_gain, q_gain, eps, pairs, type 0/1 or -1 for q's,
// q_out) -> (queries or None,); the last eight may be None but pairs and type
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  q8_kv_cache c;
  const int32_t *starts, *lengths;
  const at::Tensor *pool;
  if (n != 14 || !cache_of(a[0], a[1], a[2], a[3], &c, &starts, &lengths, &pool)) return none();
  const at::Tensor *k = heads(a[4]), *v = heads(a[5]), *q = nullptr, *cs = nullptr, *gk = nullptr, *gq = nullptr;
  if (!k) return none();
  const int64_t T = k->size(0), dev = pool->get_device();
  if (!heads_of(k, T, c.D, dev) || !heads_of(v, T, c.D, dev) || k->size(1) != c.heads || v->size(1) != c.heads ||
      v->scalar_type() != k->scalar_type())
    return none();
  if (a[6] != Py_None && (!heads_of(q = heads(a[6]), T, c.D, dev) || q->scalar_type() != k->scalar_type())) return none();
  if (a[7] != Py_None && (!typed(cs = dense(a[7], 2), at::kFloat) || cs->get_device() != dev)) return none();
  if (a[8] != Py_None && (!floats(gk = dense(a[8], 1)) || gk->size(0) != c.D || gk->get_device() != dev)) return none();
  if (a[9] != Py_None && (!floats(gq = dense(a[9], 1)) || gq->size(0) != c.D || gq->get_device() != dev)) return none();
  if (gk && gq && gk->scalar_type() != gq->scalar_type()) return none();
  const bool norm = a[10] != Py_None;
  if (!norm && (gk || gq)) return none();
  const double eps = norm ? PyFloat_AsDouble(a[10]) : 0.0;
  const long pairs = PyLong_AsLong(a[11]), type = PyLong_AsLong(a[12]);
  void *st;
  if (PyErr_Occurred() || !stream_of(*pool, &st)) return nullptr;
  at::Tensor out;
  const at::Tensor *to = nullptr;
  if (q) {
    const at::ScalarType want = type < 0 ? q->scalar_type() : type == 1 ? at::kBFloat16 : at::kFloat;
    if (a[13] != Py_None) {
      to = dense(a[13], 3);
      if (!typed(to, want) || !heads_of(to, T, c.D, dev) || to->size(1) != q->size(1)) return none();
    } else {
      out = like(*q, {T, q->size(1), c.D}, want);
      to = &out;
    }
  } else if (a[13] != Py_None) {
    return none();
  }
  const at::Tensor *g = gk ? gk : gq;
  if (append_c(&c, starts, lengths, T, k->const_data_ptr(), k->stride(0), k->stride(1), v->const_data_ptr(), v->stride(0),
               v->stride(1), q ? q->const_data_ptr() : nullptr, q ? q->stride(0) : 0, q ? q->stride(1) : 0,
               q ? q->size(1) : 0, dt(*k), cs ? cs->const_data_ptr<float>() : nullptr, cs ? cs->size(0) : 0,
               cs ? cs->size(1) : 0, static_cast<q4_rope_pairs>(pairs), norm, gk ? gk->const_data_ptr() : nullptr,
               gq ? gq->const_data_ptr() : nullptr, g ? dt(*g) : Q4_DT_F32, static_cast<float>(eps),
               to ? to->mutable_data_ptr() : nullptr, to ? dt(*to) : Q4_DT_F32, st) != Q4_OK)
    return none();
  return Py_BuildValue("(N)", to ? THPVariable_Wrap(*to) : none());
  END_HANDLE_TH_ERRORS
}

// kv_read(cache, pages, starts, lengths, T, bf16) -> (k, v)
PyObject *kv_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  q8_kv_cache c;
  const int32_t *starts, *lengths;
  const at::Tensor *pool;
  if (n != 6 || !PyLong_Check(a[4]) || !cache_of(a[0], a[1], a[2], a[3], &c, &starts, &lengths, &pool)) return none();
  const int64_t T = PyLong_AsLongLong(a[4]);
  const bool bf16 = want_bf16(a[5]);
  if (PyErr_Occurred()) return nullptr;
  if (T <= 0) return none();
  void *st;
  if (!stream_of(*pool, &st)) return nullptr;
  const at::ScalarType want = bf16 ? at::kBFloat16 : at::kFloat;
  const at::Tensor k = like(*pool, {T, c.heads, c.D}, want), v = like(*pool, {T, c.heads, c.D}, want);
  if (read_c(&c, starts, lengths, T, k.mutable_data_ptr(), v.mutable_data_ptr(), dt(k), st) != Q4_OK) return none();
  return Py_BuildValue("(NN)", THPVariable_Wrap(k), THPVariable_Wrap(v));
  END_HANDLE_TH_ERRORS
}

// attention(q, cache, pages, starts, lengths, scale or None, window, sinks, max_len or None, type 0/1 or -1 for q's, ws,
// y) -> y
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  q8_kv_cache c;
  const int32_t *starts, *lengths;
  const at::Tensor *pool;
  if (n != 12 || a[10] != Py_None || !cache_of(a[1], a[2], a[3], a[4], &c, &starts, &lengths, &pool)) return none();
  const at::Tensor *q = heads(a[0]);
  const int64_t dev = pool->get_device();
  if (!q || !heads_of(q, q->size(0), c.D, dev)) return none();
  const int64_t T = q->size(0), Hq = q->size(1);
  const double scale = a[5] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.D)) : PyFloat_AsDouble(a[5]);
  const int64_t window = PyLong_AsLongLong(a[6]), sinks = PyLong_AsLongLong(a[7]);
  const int64_t max_len = a[8] == Py_None ? c.page * c.table : PyLong_AsLongLong(a[8]);
  const long type = PyLong_AsLong(a[9]);
  void *st;
  if (PyErr_Occurred() || !stream_of(*pool, &st)) return nullptr;
  const at::ScalarType want = type < 0 ? q->scalar_type() : type == 1 ? at::kBFloat16 : at::kFloat;
  at::Tensor out, ws;
  const at::Tensor *y = &out;
  if (a[11] != Py_None) {
    y = dense(a[11], 3);
    if (!typed(y, want) || !heads_of(y, T, c.D, dev) || y->size(1) != Hq) return none();
  } else {
    out = like(*q, {T, Hq, c.D}, want);
  }
  const size_t need = attention_workspace_c(T, c.sequences, Hq, c.heads, c.D, max_len, window, sinks);
  if (need) ws = like(*q, {static_cast<int64_t>(need)}, at::kByte);
  return result(attention_c(q->const_data_ptr(), q->stride(0), q->stride(1), dt(*q), &c, starts, lengths, T, Hq, max_len,
                            static_cast<float>(scale), window, sinks, y->mutable_data_ptr(), dt(*y),
                            need ? ws.mutable_data_ptr() : nullptr, need, st),
                *y);
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
  rmsnorm_c = reinterpret_cast<decltype(rmsnorm_c)>(get("q8_rmsnorm_rows"));
  append_c = reinterpret_cast<decltype(append_c)>(get("q8_kv_append"));
  read_c = reinterpret_cast<decltype(read_c)>(get("q8_kv_read"));
  attention_workspace_c = reinterpret_cast<decltype(attention_workspace_c)>(get("q8_attention_workspace"));
  attention_c = reinterpret_cast<decltype(attention_c)>(get("q8_attention"));
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
                         Q4_FAST(rmsnorm_rows), Q4_FAST(kv_append), Q4_FAST(kv_read), Q4_FAST(attention),
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
