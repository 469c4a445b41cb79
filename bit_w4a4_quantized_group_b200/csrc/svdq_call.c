/* CPython extension that calls the hot entry points of libsvdq with positional integers, floats and
 * None (a null pointer).  ctypes takes 1.5 us to convert the 14 arguments of such a call, about the
 * time of the launch behind it; this takes a tenth of that.  The functions' addresses are handed over
 * by the ctypes binding, so that it works on whichever library file that has loaded; nothing is
 * checked here that the library checks itself. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>
#include <string.h>

#include "svdq.h"

typedef svdq_status (*fn_quantize)(svdq_format, int64_t, int64_t, int, const void*, const float*, float, const void*,
                                   void*, void*, void*, void*);
typedef svdq_status (*fn_gemm)(svdq_format, int64_t, int64_t, int64_t, int, const void*, const void*, float,
                               const void*, const void*, float, const void*, const void*, const void*, void*, void*);
typedef svdq_status (*fn_rmsnorm)(svdq_format, int64_t, int64_t, const void*, int64_t, const void*, int64_t,
                                  const float*, float, void*, int64_t, void*, void*, void*);
typedef svdq_status (*fn_glu)(svdq_format, svdq_activation, int64_t, int64_t, const void*, int64_t, const void*,
                              int64_t, const float*, void*, void*, void*);

static fn_quantize quantize_fn;
static fn_gemm gemm_fn;
static fn_rmsnorm rmsnorm_fn;
static fn_glu glu_fn;

static int64_t as_int(PyObject* o) { return (int64_t)PyLong_AsLongLong(o); }
/* What ctypes takes for a pointer besides an address and None: a c_void_p, or an object that names one,
 * such as a torch.cuda.Stream. */
static void* as_ptr_of_object(PyObject* o, int nested);
static void* as_ptr(PyObject* o) {
  if (o == Py_None) return NULL;
  if (PyLong_Check(o)) return PyLong_AsVoidPtr(o);
  return as_ptr_of_object(o, 0);
}
static void* as_ptr_of_object(PyObject* o, int nested) {
  if (PyErr_Occurred()) return NULL; /* an earlier argument's */
  const char* dot = strrchr(Py_TYPE(o)->tp_name, '.');
  const int is_pointer = strcmp(dot ? dot + 1 : Py_TYPE(o)->tp_name, "c_void_p") == 0;
  PyObject* v = is_pointer || !nested ? PyObject_GetAttrString(o, is_pointer ? "value" : "_as_parameter_") : NULL;
  void* p = NULL;
  if (v && (v == Py_None || PyLong_Check(v))) {
    p = v == Py_None ? NULL : PyLong_AsVoidPtr(v);
  } else if (v && !nested) {
    p = as_ptr_of_object(v, 1);
  } else {
    PyErr_SetString(PyExc_TypeError, "expected an address, a c_void_p or None");
  }
  Py_XDECREF(v);
  return p;
}
static float as_float(PyObject* o) { return (float)PyFloat_AsDouble(o); }

static int wrong_count(const char* name, Py_ssize_t n, Py_ssize_t want, const void* fn) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, n);
    return 1;
  }
  if (!fn) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
    return 1;
  }
  return 0;
}

/* The call itself, without the interpreter lock: a launch waits when the device's queue is full. */
#define CALL(expr)                          \
  do {                                      \
    svdq_status st;                         \
    if (PyErr_Occurred()) return NULL;      \
    Py_BEGIN_ALLOW_THREADS st = (expr);     \
    Py_END_ALLOW_THREADS                    \
    return PyLong_FromLong((long)st);       \
  } while (0)

static PyObject* call_quantize(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (wrong_count("svdq_quantize_act_lowrank_down", n, 12, (const void*)quantize_fn)) return NULL;
  const svdq_format fmt = (svdq_format)as_int(a[0]);
  const int64_t M = as_int(a[1]), K = as_int(a[2]);
  const int rank = (int)as_int(a[3]);
  const void *X = as_ptr(a[4]), *lam = as_ptr(a[5]), *L1 = as_ptr(a[7]);
  const float g = as_float(a[6]);
  void *codes = as_ptr(a[8]), *scales = as_ptr(a[9]), *Z = as_ptr(a[10]), *stream = as_ptr(a[11]);
  CALL(quantize_fn(fmt, M, K, rank, X, (const float*)lam, g, L1, codes, scales, Z, stream));
}

static PyObject* call_gemm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (wrong_count("svdq_w4a4_gemm_lowrank_up", n, 16, (const void*)gemm_fn)) return NULL;
  const svdq_format fmt = (svdq_format)as_int(a[0]);
  const int64_t M = as_int(a[1]), N = as_int(a[2]), K = as_int(a[3]);
  const int rank = (int)as_int(a[4]);
  const void *ac = as_ptr(a[5]), *as = as_ptr(a[6]), *wc = as_ptr(a[8]), *ws = as_ptr(a[9]);
  const float ga = as_float(a[7]), gw = as_float(a[10]);
  const void *Z = as_ptr(a[11]), *L2 = as_ptr(a[12]), *bias = as_ptr(a[13]);
  void *Y = as_ptr(a[14]), *stream = as_ptr(a[15]);
  CALL(gemm_fn(fmt, M, N, K, rank, ac, as, ga, wc, ws, gw, Z, L2, bias, Y, stream));
}

static PyObject* call_rmsnorm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (wrong_count("svdq_rmsnorm_quantize_act", n, 14, (const void*)rmsnorm_fn)) return NULL;
  const svdq_format fmt = (svdq_format)as_int(a[0]);
  const int64_t M = as_int(a[1]), K = as_int(a[2]), ldx = as_int(a[4]), ldr = as_int(a[6]), ldh = as_int(a[10]);
  const void *X = as_ptr(a[3]), *R = as_ptr(a[5]), *gamma = as_ptr(a[7]);
  const float eps = as_float(a[8]);
  void *H = as_ptr(a[9]), *codes = as_ptr(a[11]), *scales = as_ptr(a[12]), *stream = as_ptr(a[13]);
  CALL(rmsnorm_fn(fmt, M, K, X, ldx, R, ldr, (const float*)gamma, eps, H, ldh, codes, scales, stream));
}

static PyObject* call_glu(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (wrong_count("svdq_glu_quantize_act", n, 12, (const void*)glu_fn)) return NULL;
  const svdq_format fmt = (svdq_format)as_int(a[0]);
  const svdq_activation act = (svdq_activation)as_int(a[1]);
  const int64_t M = as_int(a[2]), K = as_int(a[3]), ldg = as_int(a[5]), ldu = as_int(a[7]);
  const void *gate = as_ptr(a[4]), *up = as_ptr(a[6]), *lam = as_ptr(a[8]);
  void *codes = as_ptr(a[9]), *scales = as_ptr(a[10]), *stream = as_ptr(a[11]);
  CALL(glu_fn(fmt, act, M, K, gate, ldg, up, ldu, (const float*)lam, codes, scales, stream));
}

/* bind(quantize, gemm, rmsnorm, glu): the addresses of the four functions. */
static PyObject* call_bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
    return NULL;
  }
  void *q = as_ptr(a[0]), *g = as_ptr(a[1]), *r = as_ptr(a[2]), *l = as_ptr(a[3]);
  if (PyErr_Occurred()) return NULL;
  quantize_fn = (fn_quantize)q;
  gemm_fn = (fn_gemm)g;
  rmsnorm_fn = (fn_rmsnorm)r;
  glu_fn = (fn_glu)l;
  Py_RETURN_NONE;
}

#define METHOD(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD("svdq_quantize_act_lowrank_down", call_quantize),
                                METHOD("svdq_w4a4_gemm_lowrank_up", call_gemm),
                                METHOD("svdq_rmsnorm_quantize_act", call_rmsnorm),
                                METHOD("svdq_glu_quantize_act", call_glu),
                                METHOD("bind", call_bind),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "svdq_call", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_svdq_call(void) { return PyModule_Create(&module); }
