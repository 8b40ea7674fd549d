/*
 * Argument marshalling of the serving calls for kvc.py, against the CPython C
 * API: tensors are checked (type, elements, contiguity, device) and passed as
 * device pointers, host arrays through the buffer protocol.  These calls run
 * once per token and layer, where a call's checks cost more than its kernels:
 * a decoding step's attention takes 5 us here and 9 through ctypes, of which 2 to
 * 4 are the launches.
 *
 * Nothing of torch is linked: a tensor is whatever has dtype, numel(),
 * is_contiguous(), get_device() and data_ptr().  The library's functions come in
 * as addresses (init), so that whichever build kvc.py has loaded is called.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <stdint.h>

#include "../../include/kvc.h"

static PyObject *s_dtype, *s_numel, *s_contiguous, *s_device, *s_ptr, *s_shape, *s_stride, *s_stream;
static PyObject *bf16, *i32, *u8, *f32;                       /* torch dtypes */
static PyObject *cur_dev, *raw_stream, *refuse, *tokens_arg, *host_array, *kvc_error; /* kvc.py's functions and error */

static __typeof__(&kvc_last_error) p_last_error;
static __typeof__(&kvc_qk_norm_rope) p_rope;
static __typeof__(&kvc_gather_q4) p_gather;
static __typeof__(&kvc_append_q4) p_append;
static __typeof__(&kvc_read_q4) p_read;
static __typeof__(&kvc_attention_q4) p_attention;

/* ---------------------------------------------------------------- arguments */
static int as_int(PyObject* o, int* out) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  if (v < INT_MIN || v > INT_MAX) {
    PyErr_SetString(PyExc_OverflowError, "an integer argument does not fit 32 bits");
    return -1;
  }
  *out = (int)v;
  return 0;
}
static int as_i64(PyObject* o, int64_t* out) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  *out = v;
  return 0;
}
/* Products of sizes: the largest int64 where they do not fit. */
static int64_t times(int64_t a, int64_t b) {
  int64_t r;
  return __builtin_mul_overflow(a, b, &r) ? INT64_MAX : r;
}
static int call_i64(PyObject* t, PyObject* name, int64_t* out) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (!r) return -1;
  const int rc = as_i64(r, out);
  Py_DECREF(r);
  return rc;
}
/* None, a raw pointer, or a contiguous tensor of dtype and at least n elements on dev. */
static int as_tensor(PyObject* t, PyObject* dtype, int64_t n, const char* name, int64_t dev, void** out) {
  int64_t v;
  *out = NULL;
  if (t == Py_None) return 0;
  if (PyLong_Check(t)) {
    *out = PyLong_AsVoidPtr(t);
    return PyErr_Occurred() ? -1 : 0;
  }
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return -1;
  int ok = d == dtype;
  Py_DECREF(d);
  if (ok) {
    if (call_i64(t, s_numel, &v)) return -1;
    ok = v >= n;
  }
  if (ok) {
    PyObject* c = PyObject_CallMethodNoArgs(t, s_contiguous);
    if (!c) return -1;
    ok = c == Py_True;
    Py_DECREF(c);
  }
  if (ok) {
    if (call_i64(t, s_device, &v)) return -1;
    ok = v == dev;
  }
  if (!ok) {
    PyObject* r = PyObject_CallFunction(refuse, "OOLs", t, dtype, (long long)n, name);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s was refused", name);
    return -1;
  }
  if (call_i64(t, s_ptr, &v)) return -1;
  *out = (void*)(uintptr_t)v;
  return 0;
}
/* A strided projection [B, T, n] whose tokens lie ld elements apart.  The usual
 * three dimensions are checked here, other forms and refusals in kvc.py. */
static int as_tokens(PyObject* t, int64_t B, int64_t T, int64_t n, int64_t ld, const char* name, int64_t dev,
                     void** out) {
  int64_t v;
  *out = NULL;
  if (t == Py_None) return 0;
  if (PyLong_Check(t)) {
    *out = PyLong_AsVoidPtr(t);
    return PyErr_Occurred() ? -1 : 0;
  }
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return -1;
  int ok = d == bf16;
  Py_DECREF(d);
  if (ok) {
    if (call_i64(t, s_device, &v)) return -1;
    ok = v == dev;
  }
  if (ok) {
    PyObject* sh = PyObject_GetAttr(t, s_shape);
    if (!sh) return -1;
    PyObject* st = PyObject_CallMethodNoArgs(t, s_stride);
    if (!st) {
      Py_DECREF(sh);
      return -1;
    }
    ok = PyTuple_Check(sh) && PyTuple_Check(st) && PyTuple_GET_SIZE(sh) == 3 && PyTuple_GET_SIZE(st) == 3;
    int64_t x[3] = {0, 0, 0}, y[3] = {0, 0, 0};
    for (int i = 0; ok && i < 3; ++i)
      if (as_i64(PyTuple_GET_ITEM(sh, i), &x[i]) || as_i64(PyTuple_GET_ITEM(st, i), &y[i])) ok = -1;
    Py_DECREF(sh);
    Py_DECREF(st);
    if (ok < 0) return -1;
    ok = ok && x[0] == B && x[1] == T && x[2] == n && y[2] == 1 && (T == 1 || y[1] == ld) &&
         (B == 1 || y[0] == times(T, ld));
  }
  if (!ok) {
    PyObject* r = PyObject_CallFunction(tokens_arg, "OLLLLsL", t, (long long)B, (long long)T, (long long)n,
                                        (long long)ld, name, (long long)dev);
    if (!r) return -1;
    const int rc = as_i64(r, &v);
    Py_DECREF(r);
    if (rc) return -1;
  } else if (call_i64(t, s_ptr, &v)) {
    return -1;
  }
  *out = (void*)(uintptr_t)v;
  return 0;
}
/* A host array of n integers of `size` bytes; others are converted by kvc.py. */
typedef struct {
  Py_buffer view;
  PyObject* keep;
  const void* p;
} Host;
static int take_buffer(PyObject* o, int size, Py_ssize_t n, Host* h) {
  if (!PyObject_CheckBuffer(o) || PyObject_GetBuffer(o, &h->view, PyBUF_FORMAT | PyBUF_ND)) {
    PyErr_Clear();
    return 0;
  }
  const char* f = h->view.format ? h->view.format : "B";
  while (*f == '<' || *f == '=' || *f == '@') ++f;
  const int whole = f[0] && !f[1] && strchr("iqlhn", f[0]) != NULL;
  if (whole && h->view.itemsize == size && h->view.len >= n * size) {
    h->p = h->view.buf;
    return 1;
  }
  PyBuffer_Release(&h->view);
  h->view.obj = NULL;
  return 0;
}
static int as_host(PyObject* o, int size, int64_t n, const char* name, Host* h) {
  h->view.obj = NULL;
  h->keep = NULL;
  h->p = NULL;
  if (o == Py_None) return 0;
  if (n < 0) n = 0;
  if (take_buffer(o, size, (Py_ssize_t)n, h)) return 0;
  h->keep = PyObject_CallFunction(host_array, "OiLs", o, size, (long long)n, name);
  if (!h->keep) return -1;
  if (take_buffer(h->keep, size, (Py_ssize_t)n, h)) return 0;
  PyErr_Format(PyExc_TypeError, "%s is no array of integers", name);
  return -1;
}
static void drop(Host* h) {
  if (h->view.obj) PyBuffer_Release(&h->view);
  Py_CLEAR(h->keep);
}
static int as_device(int64_t* dev) {
  PyObject* r = PyObject_CallNoArgs(cur_dev);
  if (!r) return -1;
  const int rc = as_i64(r, dev);
  Py_DECREF(r);
  return rc;
}
static int as_stream(PyObject* o, int64_t dev, kvc_stream_t* out) {
  PyObject* r;
  if (o == Py_None) {
    PyObject* d = PyLong_FromLongLong(dev);
    if (!d) return -1;
    r = PyObject_CallOneArg(raw_stream, d);
    Py_DECREF(d);
  } else if (PyLong_Check(o)) {
    r = Py_NewRef(o);
  } else {
    r = PyObject_GetAttr(o, s_stream);
  }
  if (!r) return -1;
  *out = (kvc_stream_t)PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return PyErr_Occurred() ? -1 : 0;
}
static PyObject* done(int rc) {
  if (rc == KVC_OK) Py_RETURN_NONE;
  PyObject* e = PyObject_CallFunction(kvc_error, "is", rc, p_last_error());
  if (e) {
    PyErr_SetObject(kvc_error, e);
    Py_DECREF(e);
  }
  return NULL;
}
static int want(Py_ssize_t got, Py_ssize_t n, const char* name) {
  if (got == n) return 0;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, n, got);
  return -1;
}
#define RUN(rc, call)        \
  Py_BEGIN_ALLOW_THREADS;    \
  rc = (call);               \
  Py_END_ALLOW_THREADS

/* -------------------------------------------------------------------- calls */
/* (q, k, v, B, T, H_q, H_kv, D, q_ld, k_ld, v_ld, R, interleaved, q_weight, k_weight, eps, inv_freq, pos, S, row0,
 *  q_out, k_act, v_act, stream) */
static PyObject* qk_norm_rope(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  int B, T, H_q, H_kv, D, R, inter, S, row0, rc;
  int64_t ld[3], dev;
  void *q, *k, *v, *qw, *kw, *inv, *pos, *qo, *ka, *va;
  kvc_stream_t st;
  if (want(n_args, 24, "qk_norm_rope") || as_int(a[3], &B) || as_int(a[4], &T) || as_int(a[5], &H_q) ||
      as_int(a[6], &H_kv) || as_int(a[7], &D) || as_i64(a[8], &ld[0]) || as_i64(a[9], &ld[1]) ||
      as_i64(a[10], &ld[2]) || as_int(a[11], &R) || as_int(a[12], &inter) || as_int(a[18], &S) ||
      as_int(a[19], &row0) || as_device(&dev))
    return NULL;
  const double eps = PyFloat_AsDouble(a[15]);
  if (eps == -1.0 && PyErr_Occurred()) return NULL;
  const int64_t kv = times(times(B, H_kv), times(S, D));
  if (as_tokens(a[0], B, T, times(H_q, D), ld[0], "q", dev, &q) ||
      as_tokens(a[1], B, T, times(H_kv, D), ld[1], "k", dev, &k) ||
      as_tokens(a[2], B, T, times(H_kv, D), ld[2], "v", dev, &v) || as_tensor(a[13], bf16, D, "q_weight", dev, &qw) ||
      as_tensor(a[14], bf16, D, "k_weight", dev, &kw) || as_tensor(a[16], f32, R / 2, "inv_freq", dev, &inv) ||
      as_tensor(a[17], i32, times(B, T), "pos", dev, &pos) ||
      as_tensor(a[20], bf16, times(times(B, H_q), times(T, D)), "q_out", dev, &qo) ||
      as_tensor(a[21], bf16, kv, "k_act", dev, &ka) || as_tensor(a[22], bf16, kv, "v_act", dev, &va) ||
      as_stream(a[23], dev, &st))
    return NULL;
  RUN(rc, p_rope(q, k, v, B, T, H_q, H_kv, D, ld[0], ld[1], ld[2], R, inter, qw, kw, (float)eps, inv, pos, S, row0, qo,
                 ka, va, st));
  return done(rc);
}

/* Rows of all batch elements of a 4-bit cache, and its bytes. */
static int64_t cache_rows(int B, int H_kv, const Host* slot) {
  return slot->p && H_kv >= 0 ? times(B, ((const int64_t*)slot->p)[H_kv]) : 0;
}
static int64_t cache_bytes(int64_t rows, int D) {
  const int64_t x = times(times(rows, D), 9);
  return x == INT64_MAX ? x : x / 8;
}

/* (k, v, idx, B, H_kv, S, D, K_l, slot_off, cache, pos, stream) */
static PyObject* gather_q4(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  int B, H, S, D, rc;
  int64_t dev;
  void *k, *v, *idx, *cache, *pos;
  kvc_stream_t st;
  Host kl = {0}, slot = {0};
  PyObject* r = NULL;
  if (want(n_args, 12, "gather_q4") || as_int(a[3], &B) || as_int(a[4], &H) || as_int(a[5], &S) ||
      as_int(a[6], &D) || as_device(&dev))
    return NULL;
  if (as_host(a[7], 4, H, "K_l", &kl) || as_host(a[8], 8, (int64_t)H + 1, "slot_off", &slot)) goto out;
  const int64_t rows = cache_rows(B, H, &slot), kv = times(times(B, H), times(S, D));
  if (as_tensor(a[0], bf16, kv, "k", dev, &k) || as_tensor(a[1], bf16, kv, "v", dev, &v) ||
      as_tensor(a[2], i32, rows, "idx", dev, &idx) || as_tensor(a[9], u8, cache_bytes(rows, D), "cache", dev, &cache) ||
      as_tensor(a[10], i32, rows, "pos", dev, &pos) || as_stream(a[11], dev, &st))
    goto out;
  RUN(rc, p_gather(k, v, idx, B, H, S, D, kl.p, slot.p, cache, pos, st));
  r = done(rc);
out:
  drop(&kl);
  drop(&slot);
  return r;
}

/* (k, v, pos_new, B, H_kv, T, D, slot_off, rows, cache, pos, stream) */
static PyObject* append_q4(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  int B, H, T, D, rc;
  int64_t dev;
  void *k, *v, *pn, *rows, *cache, *pos;
  kvc_stream_t st;
  Host slot = {0};
  PyObject* r = NULL;
  if (want(n_args, 12, "append_q4") || as_int(a[3], &B) || as_int(a[4], &H) || as_int(a[5], &T) ||
      as_int(a[6], &D) || as_device(&dev))
    return NULL;
  if (as_host(a[7], 8, (int64_t)H + 1, "slot_off", &slot)) goto out;
  const int64_t n = cache_rows(B, H, &slot), kv = times(times(B, H), times(T, D));
  if (as_tensor(a[0], bf16, kv, "k", dev, &k) || as_tensor(a[1], bf16, kv, "v", dev, &v) ||
      as_tensor(a[2], i32, times(B, T), "pos_new", dev, &pn) || as_tensor(a[8], i32, times(B, H), "rows", dev, &rows) ||
      as_tensor(a[9], u8, cache_bytes(n, D), "cache", dev, &cache) || as_tensor(a[10], i32, n, "pos", dev, &pos) ||
      as_stream(a[11], dev, &st))
    goto out;
  RUN(rc, p_append(k, v, pn, B, H, T, D, slot.p, rows, cache, pos, st));
  r = done(rc);
out:
  drop(&slot);
  return r;
}

/* (cache, B, H_kv, D, slot_off, first, n_rows, out_off, k_out, v_out, stream) */
static PyObject* read_q4(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  int B, H, D, rc;
  int64_t dev, t = 0;
  void *cache, *first, *ko, *vo;
  kvc_stream_t st;
  Host slot = {0}, nr = {0}, off = {0};
  PyObject* r = NULL;
  if (want(n_args, 11, "read_q4") || as_int(a[1], &B) || as_int(a[2], &H) || as_int(a[3], &D) || as_device(&dev))
    return NULL;
  if (as_host(a[4], 8, (int64_t)H + 1, "slot_off", &slot) || as_host(a[6], 4, H, "n_rows", &nr) ||
      as_host(a[7], 8, (int64_t)H + 1, "out_off", &off))
    goto out;
  if (off.p) t = H >= 0 ? ((const int64_t*)off.p)[H] : 0;
  else if (nr.p)
    for (int h = 0; h < H; ++h) t += ((const int32_t*)nr.p)[h];
  t = times(times(B, t), D);
  if (as_tensor(a[0], u8, cache_bytes(cache_rows(B, H, &slot), D), "cache", dev, &cache) ||
      as_tensor(a[5], i32, times(B, H), "first", dev, &first) || as_tensor(a[8], bf16, t, "k_out", dev, &ko) ||
      as_tensor(a[9], bf16, t, "v_out", dev, &vo) || as_stream(a[10], dev, &st))
    goto out;
  RUN(rc, p_read(cache, B, H, D, slot.p, first, nr.p, off.p, ko, vo, st));
  r = done(rc);
out:
  drop(&slot);
  drop(&nr);
  drop(&off);
  return r;
}

/* (q, cache, pos, rows, extra, q_pos, B, T, H_q, H_kv, D, slot_off, out, lse, ws, ws_bytes, stream) */
static PyObject* attention_q4(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  int extra, B, T, H_q, H, D, rc;
  int64_t dev, ws_bytes = 0;
  void *q, *cache, *pos, *rows, *qp, *out, *lse, *ws;
  kvc_stream_t st;
  Host slot = {0};
  PyObject* r = NULL;
  if (want(n_args, 17, "attention_q4") || as_int(a[4], &extra) || as_int(a[6], &B) || as_int(a[7], &T) ||
      as_int(a[8], &H_q) || as_int(a[9], &H) || as_int(a[10], &D) || as_device(&dev))
    return NULL;
  if (as_host(a[11], 8, (int64_t)H + 1, "slot_off", &slot)) goto out;
  const int64_t n = cache_rows(B, H, &slot), nq = times(times(B, H_q), T);
  if (as_tensor(a[0], bf16, times(nq, D), "q", dev, &q) ||
      as_tensor(a[1], u8, cache_bytes(n, D), "cache", dev, &cache) || as_tensor(a[2], i32, n, "pos", dev, &pos) ||
      as_tensor(a[3], i32, times(B, H), "rows", dev, &rows) || as_tensor(a[5], i32, times(B, T), "q_pos", dev, &qp) ||
      as_tensor(a[12], bf16, times(nq, D), "out", dev, &out) || as_tensor(a[13], f32, nq, "lse", dev, &lse) ||
      (a[15] != Py_None ? as_i64(a[15], &ws_bytes) : call_i64(a[14], s_numel, &ws_bytes)) ||
      as_tensor(a[14], u8, ws_bytes, "ws", dev, &ws) || as_stream(a[16], dev, &st))
    goto out;
  RUN(rc, p_attention(q, cache, pos, rows, extra, qp, B, T, H_q, H, D, slot.p, out, lse, ws,
                      ws_bytes < 0 ? 0 : (size_t)ws_bytes, st));
  r = done(rc);
out:
  drop(&slot);
  return r;
}

/* (library: six addresses; dtypes: bf16, int32, uint8, float32; kvc.py's functions and error class) */
static PyObject* init(PyObject* self, PyObject* args) {
  (void)self;
  unsigned long long f[6];
  PyObject* o[10];
  if (!PyArg_ParseTuple(args, "(KKKKKK)(OOOO)(OOOOOO)", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &o[0], &o[1], &o[2],
                        &o[3], &o[4], &o[5], &o[6], &o[7], &o[8], &o[9]))
    return NULL;
  p_last_error = (__typeof__(p_last_error))(uintptr_t)f[0];
  p_rope = (__typeof__(p_rope))(uintptr_t)f[1];
  p_gather = (__typeof__(p_gather))(uintptr_t)f[2];
  p_append = (__typeof__(p_append))(uintptr_t)f[3];
  p_read = (__typeof__(p_read))(uintptr_t)f[4];
  p_attention = (__typeof__(p_attention))(uintptr_t)f[5];
  PyObject** to[10] = {&bf16, &i32, &u8, &f32, &cur_dev, &raw_stream, &refuse, &tokens_arg, &host_array, &kvc_error};
  for (int i = 0; i < 10; ++i) {
    Py_INCREF(o[i]);
    Py_XSETREF(*to[i], o[i]);
  }
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, NULL},
    {"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, NULL},
    {"gather_q4", (PyCFunction)(void (*)(void))gather_q4, METH_FASTCALL, NULL},
    {"append_q4", (PyCFunction)(void (*)(void))append_q4, METH_FASTCALL, NULL},
    {"read_q4", (PyCFunction)(void (*)(void))read_q4, METH_FASTCALL, NULL},
    {"attention_q4", (PyCFunction)(void (*)(void))attention_q4, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_numel = PyUnicode_InternFromString("numel");
  s_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_device = PyUnicode_InternFromString("get_device");
  s_ptr = PyUnicode_InternFromString("data_ptr");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_stream = PyUnicode_InternFromString("cuda_stream");
  if (!s_dtype || !s_numel || !s_contiguous || !s_device || !s_ptr || !s_shape || !s_stride || !s_stream) return NULL;
  return PyModule_Create(&module);
}
