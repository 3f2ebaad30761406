/* _fdcall — the entry points of the 4-bit cache and of the page bookkeeping for
 * Python, where a call's time on the host counts: a launch itself takes about 2 us,
 * and ctypes' conversions of 16 arguments took another 3.8 us (1.1 us here).
 * A tensor is anything with a data_ptr() method, an int is a device address, None is
 * NULL.  The library is the one that the package has loaded: bind() takes its
 * functions' addresses. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "fd.h"

static struct {
  fd_status (*append)(const fd_problem*, int, const void*, int64_t, const void*, int64_t,
                      const int64_t*, void*, void*, void*, fd_stream_t);
  fd_status (*expand)(const fd_problem*, const void*, const void*, const void*, const int32_t*,
                      const int32_t*, void*, void*, fd_stream_t);
  fd_status (*decode)(const fd_problem*, const void*, const void*, const void*, const void*,
                      const int32_t*, const int32_t*, float, int, void*, float*, void*, size_t,
                      fd_stream_t);
  fd_status (*alloc)(int, int, int, int, int, const int32_t*, const int32_t*, const int32_t*,
                     const int32_t*, int32_t*, int32_t*, int32_t*, int64_t*, int32_t*, int32_t*,
                     fd_stream_t);
  fd_status (*release)(int, int, int, int, const int32_t*, const uint8_t*, const int32_t*,
                       int32_t*, const int32_t*, int32_t*, int32_t*, fd_stream_t);
} g_fd;

static PyObject* g_data_ptr;   /* "data_ptr" */

/* One call's arguments, taken from left to right; `failed` once a conversion set a
 * Python error. */
typedef struct {
  PyObject* const* args;
  int failed;
  Py_buffer problem;           /* obj is NULL until taken */
} call;

static PyObject* next_arg(call* c) { return *c->args++; }

static int64_t take_int64(call* c) {
  PyObject* x = next_arg(c);
  if (c->failed) return 0;
  const long long v = PyLong_AsLongLong(x);
  if (v == -1 && PyErr_Occurred()) c->failed = 1;
  return v;
}

static int take_int(call* c) {
  const int64_t v = take_int64(c);
  if (!c->failed && (v < INT32_MIN || v > INT32_MAX)) {
    PyErr_SetString(PyExc_OverflowError, "an argument does not fit a C int");
    c->failed = 1;
  }
  return (int)v;
}

static float take_float(call* c) {
  PyObject* x = next_arg(c);
  if (c->failed) return 0.f;
  const double v = PyFloat_AsDouble(x);
  if (v == -1.0 && PyErr_Occurred()) c->failed = 1;
  return (float)v;
}

static void* take_ptr(call* c) {
  PyObject* x = next_arg(c);
  if (c->failed || x == Py_None) return NULL;
  PyObject* address = PyLong_Check(x) ? Py_NewRef(x) : PyObject_CallMethodNoArgs(x, g_data_ptr);
  void* p = address ? PyLong_AsVoidPtr(address) : NULL;
  Py_XDECREF(address);
  if (!p && PyErr_Occurred()) c->failed = 1;
  return p;
}

static const fd_problem* take_problem(call* c) {
  PyObject* x = next_arg(c);
  if (c->failed) return NULL;
  if (PyObject_GetBuffer(x, &c->problem, PyBUF_SIMPLE) != 0) {
    c->failed = 1;
    return NULL;
  }
  if (c->problem.len != (Py_ssize_t)sizeof(fd_problem)) {
    PyErr_SetString(PyExc_TypeError, "problem: expected an fd_problem");
    c->failed = 1;
  }
  return (const fd_problem*)c->problem.buf;
}

static int begin(call* c, PyObject* const* args, Py_ssize_t n, Py_ssize_t want, int bound) {
  c->args = args;
  c->failed = 0;
  c->problem.obj = NULL;
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, want);
    return 0;
  }
  if (!bound) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not loaded");
    return 0;
  }
  return 1;
}

/* Runs `expr` without the interpreter's lock, unless an argument failed. */
#define FINISH(expr)                                   \
  do {                                                 \
    fd_status status = FD_OK;                          \
    if (!c.failed) {                                   \
      Py_BEGIN_ALLOW_THREADS                           \
      status = (expr);                                 \
      Py_END_ALLOW_THREADS                             \
    }                                                  \
    if (c.problem.obj) PyBuffer_Release(&c.problem);   \
    return c.failed ? NULL : PyLong_FromLong(status);  \
  } while (0)

static PyObject* append_int4(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  (void)self;
  call c;
  if (!begin(&c, args, n, 11, g_fd.append != NULL)) return NULL;
  const fd_problem* p = take_problem(&c);
  const int tokens = take_int(&c);
  const void* k = take_ptr(&c);
  const int64_t k_stride = take_int64(&c);
  const void* v = take_ptr(&c);
  const int64_t v_stride = take_int64(&c);
  const int64_t* slots = take_ptr(&c);
  void* k4 = take_ptr(&c);
  void* v4 = take_ptr(&c);
  void* params = take_ptr(&c);
  fd_stream_t s = take_ptr(&c);
  FINISH(g_fd.append(p, tokens, k, k_stride, v, v_stride, slots, k4, v4, params, s));
}

static PyObject* expand_int4(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  (void)self;
  call c;
  if (!begin(&c, args, n, 9, g_fd.expand != NULL)) return NULL;
  const fd_problem* p = take_problem(&c);
  const void* k4 = take_ptr(&c);
  const void* v4 = take_ptr(&c);
  const void* params = take_ptr(&c);
  const int32_t* seqlens = take_ptr(&c);
  const int32_t* table = take_ptr(&c);
  void* k = take_ptr(&c);
  void* v = take_ptr(&c);
  fd_stream_t s = take_ptr(&c);
  FINISH(g_fd.expand(p, k4, v4, params, seqlens, table, k, v, s));
}

static PyObject* decode_int4(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  (void)self;
  call c;
  if (!begin(&c, args, n, 14, g_fd.decode != NULL)) return NULL;
  const fd_problem* p = take_problem(&c);
  const void* q = take_ptr(&c);
  const void* k4 = take_ptr(&c);
  const void* v4 = take_ptr(&c);
  const void* params = take_ptr(&c);
  const int32_t* seqlens = take_ptr(&c);
  const int32_t* table = take_ptr(&c);
  const float scale = take_float(&c);
  const int splits = take_int(&c);
  void* out = take_ptr(&c);
  float* lse = take_ptr(&c);
  void* workspace = take_ptr(&c);
  const int64_t bytes = take_int64(&c);
  fd_stream_t s = take_ptr(&c);
  FINISH(g_fd.decode(p, q, k4, v4, params, seqlens, table, scale, splits, out, lse, workspace,
                     bytes > 0 ? (size_t)bytes : 0, s));
}

static PyObject* alloc_pages(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  (void)self;
  call c;
  if (!begin(&c, args, n, 16, g_fd.alloc != NULL)) return NULL;
  const int B = take_int(&c), block = take_int(&c), most = take_int(&c), tokens = take_int(&c);
  const int pages = take_int(&c);
  const int32_t* seqlens = take_ptr(&c);
  const int32_t* new_lens = take_ptr(&c);
  const int32_t* free_pages = take_ptr(&c);
  const int32_t* free_count = take_ptr(&c);
  int32_t* table = take_ptr(&c);
  int32_t* seqlens_out = take_ptr(&c);
  int32_t* cu_new = take_ptr(&c);
  int64_t* slots = take_ptr(&c);
  int32_t* positions = take_ptr(&c);
  int32_t* count_out = take_ptr(&c);
  fd_stream_t s = take_ptr(&c);
  FINISH(g_fd.alloc(B, block, most, tokens, pages, seqlens, new_lens, free_pages, free_count,
                    table, seqlens_out, cu_new, slots, positions, count_out, s));
}

static PyObject* release_pages(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  (void)self;
  call c;
  if (!begin(&c, args, n, 12, g_fd.release != NULL)) return NULL;
  const int B = take_int(&c), block = take_int(&c), most = take_int(&c), pages = take_int(&c);
  const int32_t* seqlens = take_ptr(&c);
  const uint8_t* done = take_ptr(&c);
  const int32_t* table = take_ptr(&c);
  int32_t* free_pages = take_ptr(&c);
  const int32_t* free_count = take_ptr(&c);
  int32_t* seqlens_out = take_ptr(&c);
  int32_t* count_out = take_ptr(&c);
  fd_stream_t s = take_ptr(&c);
  FINISH(g_fd.release(B, block, most, pages, seqlens, done, table, free_pages, free_count,
                      seqlens_out, count_out, s));
}

static PyObject* bind(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  (void)self;
  call c;
  if (!begin(&c, args, n, 5, 1)) return NULL;
  void* f[5];
  for (int i = 0; i < 5; ++i) f[i] = take_ptr(&c);
  if (c.failed) return NULL;
  *(void**)&g_fd.append = f[0];
  *(void**)&g_fd.expand = f[1];
  *(void**)&g_fd.decode = f[2];
  *(void**)&g_fd.alloc = f[3];
  *(void**)&g_fd.release = f[4];
  Py_RETURN_NONE;
}

#define METHOD(name, doc) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, doc}
static PyMethodDef methods[] = {
    METHOD(append_int4, "fd_append_int4"),
    METHOD(expand_int4, "fd_expand_int4"),
    METHOD(decode_int4, "fd_decode_int4"),
    METHOD(alloc_pages, "fd_alloc_pages"),
    METHOD(release_pages, "fd_release_pages"),
    METHOD(bind, "Addresses of the five functions, in this order."),
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fdcall", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fdcall(void) {
  if (!g_data_ptr) g_data_ptr = PyUnicode_InternFromString("data_ptr");
  return g_data_ptr ? PyModule_Create(&module) : NULL;
}
