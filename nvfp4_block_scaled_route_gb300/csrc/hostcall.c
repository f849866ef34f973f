/* Argument checks and calls of the attention and serving operators for binding.py.
 *
 * A call of few tokens takes the GPU some 5 us, and the same calls by way of ctypes took
 * the host 8 to 10: 0.4 us for each tensor that is checked in Python, 1.5 to 2.5 for the
 * conversion of 20 to 30 arguments.  Here the checks read the same attributes of the same
 * objects, and the C entry points are called with their types known. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "nvfp4moe.h"

/* ---- checks ---- */
static PyObject *s_dtype, *s_shape, *s_is_cuda, *s_is_contiguous, *s_data_ptr, *s_stride, *s_numel;

static int is_true(PyObject* t, PyObject* name, int call) {
  PyObject* v = call ? PyObject_CallMethodNoArgs(t, name) : PyObject_GetAttr(t, name);
  if (v == NULL) return -1;
  const int yes = v == Py_True ? 1 : (v == Py_False ? 0 : PyObject_IsTrue(v));
  Py_DECREF(v);
  return yes;
}

static int has_dtype(PyObject* t, PyObject* dtype) {
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (d == NULL) return -1;
  Py_DECREF(d);
  return d == dtype;
}

/* Whether t is a CUDA tensor, its memory dense (of fewer than two elements: or not). */
static int is_dense(PyObject* t, long long n) {
  const int ok = is_true(t, s_is_cuda, 0);
  return ok > 0 && n > 1 ? is_true(t, s_is_contiguous, 1) : ok;
}

/* Length of the vector t of this type, -1 if it is none, -2 with an exception. */
static long long length_of(PyObject* t, PyObject* dtype) {
  const int ok = has_dtype(t, dtype);
  if (ok <= 0) return ok < 0 ? -2 : -1;
  PyObject* shape = PyObject_GetAttr(t, s_shape);
  if (shape == NULL) return -2;
  long long n = -1;
  if (PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == 1) {
    n = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0));
    if (n == -1 && PyErr_Occurred()) n = -2;
  }
  Py_DECREF(shape);
  return n;
}

/* vector(t, n, dtype, what): address of the dense CUDA tensor [n], None for None. */
static PyObject* vector(PyObject* self, PyObject* const* args, Py_ssize_t count) {
  (void)self;
  if (count != 4) return PyErr_Format(PyExc_TypeError, "vector takes 4 arguments");
  PyObject* t = args[0];
  if (t == Py_None) Py_RETURN_NONE;
  const long long n = PyLong_AsLongLong(args[1]);
  if (n == -1 && PyErr_Occurred()) return NULL;
  const long long have = length_of(t, args[2]);
  if (have == -2) return NULL;
  if (have != n || n < 0)
    return PyErr_Format(PyExc_ValueError, "%U must be %S [%lld]", args[3], args[2], n);
  const int ok = is_dense(t, n);
  if (ok < 0) return NULL;
  if (!ok) return PyErr_Format(PyExc_ValueError, "%U must be a dense CUDA tensor", args[3]);
  return PyObject_CallMethodNoArgs(t, s_data_ptr);
}

/* run(t, dtype, what): (address, length) of a dense CUDA tensor of one axis. */
static PyObject* run(PyObject* self, PyObject* const* args, Py_ssize_t count) {
  (void)self;
  if (count != 3) return PyErr_Format(PyExc_TypeError, "run takes 3 arguments");
  PyObject* t = args[0];
  const long long n = length_of(t, args[1]);
  if (n == -2) return NULL;
  if (n < 0) return PyErr_Format(PyExc_ValueError, "%U must be %S of one axis", args[2], args[1]);
  const int ok = is_dense(t, n);
  if (ok < 0) return NULL;
  if (!ok) return PyErr_Format(PyExc_ValueError, "%U must be a dense CUDA tensor", args[2]);
  PyObject* p = PyObject_CallMethodNoArgs(t, s_data_ptr);
  PyObject* out = p != NULL ? Py_BuildValue("(NL)", p, n) : NULL;
  return out;
}

/* dense(t): (address, number of elements) of a dense CUDA tensor. */
static PyObject* dense(PyObject* self, PyObject* t) {
  (void)self;
  int ok = is_true(t, s_is_cuda, 0);
  if (ok == 0) PyErr_SetString(PyExc_ValueError, "expected a CUDA tensor");
  if (ok <= 0) return NULL;
  ok = is_true(t, s_is_contiguous, 1);
  if (ok == 0)
    PyErr_SetString(PyExc_ValueError,
                    "expected a contiguous tensor (the library reads dense row-major memory)");
  if (ok <= 0) return NULL;
  PyObject* n = PyObject_CallMethodNoArgs(t, s_numel);
  PyObject* p = n != NULL ? PyObject_CallMethodNoArgs(t, s_data_ptr) : NULL;
  if (p == NULL) {
    Py_XDECREF(n);
    return NULL;
  }
  return Py_BuildValue("(NN)", p, n);
}

/* rows(t, dtype, what): (address, token stride, head stride) of head rows [T, heads, D]. */
static PyObject* rows(PyObject* self, PyObject* const* args, Py_ssize_t count) {
  (void)self;
  if (count != 3) return PyErr_Format(PyExc_TypeError, "rows takes 3 arguments");
  PyObject* t = args[0];
  PyObject* s = PyObject_CallMethodNoArgs(t, s_stride);
  if (s == NULL) return NULL;
  int ok = PyTuple_Check(s) && PyTuple_GET_SIZE(s) == 3 ? has_dtype(t, args[1]) : 0;
  if (ok > 0) ok = is_true(t, s_is_cuda, 0);
  PyObject* out = NULL;
  if (ok == 0) {
    PyErr_Format(PyExc_ValueError, "%U must be a bf16 CUDA tensor [tokens, heads, head_dim]", args[2]);
  } else if (ok > 0) {
    const long long last = PyLong_AsLongLong(PyTuple_GET_ITEM(s, 2));
    if (last != 1) {
      if (!PyErr_Occurred())
        PyErr_Format(PyExc_ValueError, "%U: head_dim must be contiguous", args[2]);
    } else {
      PyObject* p = PyObject_CallMethodNoArgs(t, s_data_ptr);
      if (p != NULL) {
        out = PyTuple_Pack(3, p, PyTuple_GET_ITEM(s, 0), PyTuple_GET_ITEM(s, 1));
        Py_DECREF(p);
      }
    }
  }
  Py_DECREF(s);
  return out;
}

/* ---- calls ---- */
/* The next argument as an address (an int, or None), an integer, a float or the memory of
 * a ctypes structure, which stays alive until done(). */
typedef struct {
  PyObject* const* at;
  Py_buffer held[2];
  int holds, bad;
} Args;

static void* ptr(Args* a) {
  PyObject* o = *a->at++;
  if (o == Py_None || a->bad) return NULL;
  void* p = PyLong_AsVoidPtr(o);
  if (p == NULL && PyErr_Occurred()) a->bad = 1;
  return p;
}
static long long integer(Args* a) {
  PyObject* o = *a->at++;
  if (a->bad) return 0;
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) a->bad = 1;
  return v;
}
static int int32(Args* a) { return (int)integer(a); }   /* (as ctypes: the low bits) */
static float real(Args* a) {
  PyObject* o = *a->at++;
  if (a->bad) return 0.0f;
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) a->bad = 1;
  return (float)v;
}
static void* structure(Args* a) {
  PyObject* o = *a->at++;
  if (a->bad) return NULL;
  Py_buffer* view = &a->held[a->holds];
  if (PyObject_GetBuffer(o, view, PyBUF_SIMPLE) != 0) {
    a->bad = 1;
    return NULL;
  }
  ++a->holds;
  return view->buf;
}
static PyObject* done(Args* a, int status) {
  while (a->holds > 0) PyBuffer_Release(&a->held[--a->holds]);
  return a->bad ? NULL : PyLong_FromLong(status);
}

static __typeof__(&attn_qk_norm_rope) f_qk_norm_rope;
static __typeof__(&attn_kv_append) f_kv_append;
static __typeof__(&attn_paged_forward) f_paged_forward;
static __typeof__(&attn_plan_pages) f_plan_pages;
static __typeof__(&draft_verify) f_draft_verify;

/* Arguments are read in order (each into a variable: C leaves the order of a call's open);
 * the call itself runs without the interpreter's lock, as ctypes has it. */
#define BEGIN(name, n)                                                                    \
  static PyObject* call_##name(PyObject* self, PyObject* const* args, Py_ssize_t count) { \
    (void)self;                                                                           \
    if (count != (n) || f_##name == NULL)                                                 \
      return PyErr_Format(PyExc_TypeError, #name " takes %d arguments, once bound", (n)); \
    Args a = {args, {{0}}, 0, 0};                                                         \
    int status = 0;
#define CALL(...)            \
  if (!a.bad) {              \
    Py_BEGIN_ALLOW_THREADS   \
    status = __VA_ARGS__;    \
    Py_END_ALLOW_THREADS     \
  }                          \
  return done(&a, status);   \
  }

BEGIN(qk_norm_rope, 27)
  void* q = ptr(&a); const int64_t qt = integer(&a), qh = integer(&a); const int hq = int32(&a);
  void* k = ptr(&a); const int64_t kt = integer(&a), kh = integer(&a); const int hk = int32(&a);
  const int64_t T = integer(&a); const int D = int32(&a); void* pos = ptr(&a); void* rope = ptr(&a);
  const int64_t npos = integer(&a); const int rot = int32(&a), pairs = int32(&a);
  void* wq = ptr(&a); void* wk = ptr(&a); const float eps = real(&a);
  void* qo = ptr(&a); const int64_t qot = integer(&a), qoh = integer(&a);
  void* ko = ptr(&a); const int64_t kot = integer(&a), koh = integer(&a);
  void* ws = ptr(&a); const size_t n = (size_t)integer(&a); void* stream = ptr(&a);
CALL(f_qk_norm_rope(q, qt, qh, hq, k, kt, kh, hk, T, D, pos, rope, npos, rot, pairs, wq, wk, eps, qo,
                    qot, qoh, ko, kot, koh, ws, n, stream))

BEGIN(kv_append, 25)
  void* cache = structure(&a); void* batch = structure(&a);
  void* k = ptr(&a); const int64_t kt = integer(&a), kh = integer(&a);
  void* v = ptr(&a); const int64_t vt = integer(&a), vh = integer(&a);
  void* q = ptr(&a); const int64_t qt = integer(&a), qh = integer(&a); const int hq = int32(&a);
  void* qo = ptr(&a); const int64_t qot = integer(&a), qoh = integer(&a);
  void* rope = ptr(&a); const int64_t npos = integer(&a); const int rot = int32(&a), pairs = int32(&a);
  void* wq = ptr(&a); void* wk = ptr(&a); const float eps = real(&a);
  void* ws = ptr(&a); const size_t n = (size_t)integer(&a); void* stream = ptr(&a);
CALL(f_kv_append(cache, batch, k, kt, kh, v, vt, vh, q, qt, qh, hq, qo, qot, qoh, rope, npos, rot, pairs,
                 wq, wk, eps, ws, n, stream))

BEGIN(paged_forward, 15)
  void* q = ptr(&a); const int64_t qt = integer(&a), qh = integer(&a); const int hq = int32(&a);
  void* cache = structure(&a); void* batch = structure(&a);
  const float scale = real(&a); const int window = int32(&a);
  void* out = ptr(&a); const int64_t ot = integer(&a), oh = integer(&a); void* lse = ptr(&a);
  void* ws = ptr(&a); const size_t n = (size_t)integer(&a); void* stream = ptr(&a);
CALL(f_paged_forward(q, qt, qh, hq, cache, batch, scale, window, out, ot, oh, lse, ws, n, stream))

BEGIN(plan_pages, 19)
  void* ring = ptr(&a); const int64_t size = integer(&a); void* state = ptr(&a); void* state_out = ptr(&a);
  const int batch = int32(&a), page = int32(&a); const int64_t most = integer(&a);
  void* before = ptr(&a); void* cached = ptr(&a); void* fresh = ptr(&a); void* kv_len = ptr(&a);
  void* q_start = ptr(&a); void* table = ptr(&a); void* positions = ptr(&a); void* slots = ptr(&a);
  const int64_t count_rows = integer(&a);
  void* ws = ptr(&a); const size_t n = (size_t)integer(&a); void* stream = ptr(&a);
CALL(f_plan_pages(ring, size, state, state_out, batch, page, most, before, cached, fresh, kv_len, q_start,
                  table, positions, slots, count_rows, ws, n, stream))

BEGIN(draft_verify, 19)
  void* target = ptr(&a); const int64_t ts = integer(&a); void* draft = ptr(&a); const int64_t ds = integer(&a);
  const int dtype = int32(&a); const int64_t count_rows = integer(&a), vocab = integer(&a);
  void* tokens = ptr(&a); const int batch = int32(&a); void* q_start = ptr(&a); void* kv_len = ptr(&a);
  void* accept_u = ptr(&a); void* sample_u = ptr(&a); void* accepted = ptr(&a); void* next = ptr(&a);
  void* cached = ptr(&a);
  void* ws = ptr(&a); const size_t n = (size_t)integer(&a); void* stream = ptr(&a);
CALL(f_draft_verify(target, ts, draft, ds, dtype, count_rows, vocab, tokens, batch, q_start, kv_len, accept_u,
                    sample_u, accepted, next, cached, ws, n, stream))

/* bind(qk_norm_rope, kv_append, paged_forward, plan_pages, draft_verify): addresses of the
 * library's entry points. */
static PyObject* bind(PyObject* self, PyObject* const* args, Py_ssize_t count) {
  (void)self;
  if (count != 5) return PyErr_Format(PyExc_TypeError, "bind takes 5 addresses");
  Args a = {args, {{0}}, 0, 0};
  void* p[5];
  for (int i = 0; i < 5; ++i) p[i] = ptr(&a);
  if (a.bad) return NULL;
  f_qk_norm_rope = (__typeof__(f_qk_norm_rope))p[0];
  f_kv_append = (__typeof__(f_kv_append))p[1];
  f_paged_forward = (__typeof__(f_paged_forward))p[2];
  f_plan_pages = (__typeof__(f_plan_pages))p[3];
  f_draft_verify = (__typeof__(f_draft_verify))p[4];
  Py_RETURN_NONE;
}

#define METHOD(name, fn) {name, (PyCFunction)(void (*)(void))fn, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD("vector", vector),
                                METHOD("run", run),
                                {"dense", dense, METH_O, NULL},
                                METHOD("rows", rows),
                                METHOD("bind", bind),
                                METHOD("attn_qk_norm_rope", call_qk_norm_rope),
                                METHOD("attn_kv_append", call_kv_append),
                                METHOD("attn_paged_forward", call_paged_forward),
                                METHOD("attn_plan_pages", call_plan_pages),
                                METHOD("draft_verify", call_draft_verify),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hostcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__hostcall(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_is_cuda = PyUnicode_InternFromString("is_cuda");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_stride = PyUnicode_InternFromString("stride");
  s_numel = PyUnicode_InternFromString("numel");
  if (!s_dtype || !s_shape || !s_is_cuda || !s_is_contiguous || !s_data_ptr || !s_stride || !s_numel)
    return NULL;
  return PyModule_Create(&module);
}
