/* Calls of the library's short entry points without ctypes: the same functions
 * with the same arguments in the same order, each an int, a float or None (a
 * null pointer).  Marshalling fifteen arguments through ctypes takes about
 * 1.5 us, nearly as long as the launch itself.
 *
 * As ctypes does, a wrapper lets other Python threads run during the call: a
 * launch can wait for room in the device's queue, or for a host callback that
 * needs the interpreter.
 *
 * bind(name, address) gives a function its address in the loaded libtqmoe.so;
 * the module links to nothing but Python. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <string.h>

#include "tqmoe.h"

#define MAX_ARGS 32

/* The arguments as integers (pointers too), the one 'f' among them apart.
 * p: pointer or None, i: int, l: int64 or size, f: float.  Returns 0 with a
 * Python error set. */
static int take(const char* sig, const void* fn, PyObject* const* a, Py_ssize_t n, long long* v, float* f) {
  if (!fn) {
    PyErr_SetString(PyExc_RuntimeError, "the function is not bound to the library");
    return 0;
  }
  if (n != (Py_ssize_t)strlen(sig)) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", (Py_ssize_t)strlen(sig), n);
    return 0;
  }
  for (Py_ssize_t k = 0; k < n; ++k) {
    switch (sig[k]) {
      case 'f': *f = (float)PyFloat_AsDouble(a[k]); break;
      case 'p': v[k] = a[k] == Py_None ? 0 : (long long)(intptr_t)PyLong_AsVoidPtr(a[k]); break;
      default:
        v[k] = PyLong_AsLongLong(a[k]);
        if (sig[k] == 'i' && (v[k] < INT32_MIN || v[k] > INT32_MAX)) {
          if (!PyErr_Occurred()) PyErr_SetString(PyExc_OverflowError, "argument out of the range of int");
        }
    }
    if (PyErr_Occurred()) return 0;
  }
  return 1;
}

#define PTR(k) ((void*)(intptr_t)v[k])
#define INT(k) ((int)v[k])
#define STREAM(k) ((tq_stream_t)(intptr_t)v[k])

/* A wrapper of `name`: its arguments by `sig`, then the call as written. */
#define WRAPPER(name, sig, ...)                                                        \
  static __typeof__(&name) fn_##name;                                                  \
  static PyObject* call_##name(PyObject* self, PyObject* const* a, Py_ssize_t n) {     \
    long long v[MAX_ARGS];                                                             \
    float f = 0.f;                                                                     \
    int rc;                                                                            \
    (void)self;                                                                        \
    (void)f;                                                                           \
    if (!take(sig, (const void*)fn_##name, a, n, v, &f)) return NULL;                  \
    Py_BEGIN_ALLOW_THREADS                                                             \
    rc = fn_##name(__VA_ARGS__);                                                       \
    Py_END_ALLOW_THREADS                                                               \
    return PyLong_FromLong(rc);                                                        \
  }

WRAPPER(tq_router_scored, "pilpliiiiiifppp", PTR(0), INT(1), v[2], PTR(3), v[4], INT(5), INT(6), INT(7), INT(8), INT(9),
        INT(10), f, PTR(12), PTR(13), STREAM(14))
WRAPPER(tq_router_scored_backward, "pilpppliiiifpp", PTR(0), INT(1), v[2], PTR(3), PTR(4), PTR(5), v[6], INT(7), INT(8),
        INT(9), INT(10), f, PTR(12), STREAM(13))
WRAPPER(tq_fp4_quantize, "pilliipppp", PTR(0), INT(1), v[2], v[3], INT(4), INT(5), PTR(6), PTR(7), PTR(8), STREAM(9))
WRAPPER(tq_fp4_dequantize, "ppliippip", PTR(0), PTR(1), v[2], INT(3), INT(4), PTR(5), PTR(6), INT(7), STREAM(8))
WRAPPER(tq_fp4_linear, "pilppippliiplpip", PTR(0), INT(1), v[2], PTR(3), PTR(4), INT(5), PTR(6), PTR(7), v[8], INT(9),
        INT(10), PTR(11), (size_t)v[12], PTR(13), INT(14), STREAM(15))
WRAPPER(tq_fp4_moe_forward, "pilppippppliiiiplpip", PTR(0), INT(1), v[2], PTR(3), PTR(4), INT(5), PTR(6), PTR(7),
        PTR(8), PTR(9), v[10], INT(11), INT(12), INT(13), INT(14), PTR(15), (size_t)v[16], PTR(17), INT(18), STREAM(19))
WRAPPER(tq_fp4_moe_mlp_forward, "pilppppppippppliiiiplpip", PTR(0), INT(1), v[2], PTR(3), PTR(4), PTR(5), PTR(6),
        PTR(7), PTR(8), INT(9), PTR(10), PTR(11), PTR(12), PTR(13), v[14], INT(15), INT(16), INT(17), INT(18), PTR(19),
        (size_t)v[20], PTR(21), INT(22), STREAM(23))

WRAPPER(tq_rms_norm, "pilplpiflipppppp", PTR(0), INT(1), v[2], PTR(3), v[4], PTR(5), INT(6), f, v[8], INT(9), PTR(10),
        PTR(11), PTR(12), PTR(13), PTR(14), STREAM(15))
WRAPPER(tq_rms_norm_backward, "plpilpipplliplppp", PTR(0), v[1], PTR(2), INT(3), v[4], PTR(5), INT(6), PTR(7), PTR(8),
        v[9], v[10], INT(11), PTR(12), (size_t)v[13], PTR(14), PTR(15), STREAM(16))
WRAPPER(tq_fp8_quantize, "pililiippp", PTR(0), INT(1), v[2], INT(3), v[4], INT(5), INT(6), PTR(7), PTR(8), STREAM(9))
WRAPPER(tq_fp8_dequantize, "ppiliipip", PTR(0), PTR(1), INT(2), v[3], INT(4), INT(5), PTR(6), INT(7), STREAM(8))
WRAPPER(tq_fp8_linear, "ppppliiplpip", PTR(0), PTR(1), PTR(2), PTR(3), v[4], INT(5), INT(6), PTR(7), (size_t)v[8],
        PTR(9), INT(10), STREAM(11))
WRAPPER(tq_fp8_moe_forward, "ppppppliiiiplpip", PTR(0), PTR(1), PTR(2), PTR(3), PTR(4), PTR(5), v[6], INT(7),
        INT(8), INT(9), INT(10), PTR(11), (size_t)v[12], PTR(13), INT(14), STREAM(15))
WRAPPER(tq_fp8_moe_mlp_forward, "ppppppppliiiiplpip", PTR(0), PTR(1), PTR(2), PTR(3), PTR(4), PTR(5), PTR(6),
        PTR(7), v[8], INT(9), INT(10), INT(11), INT(12), PTR(13), (size_t)v[14], PTR(15), INT(16), STREAM(17))
WRAPPER(tq_swiglu_linear, "pilpliiplppp", PTR(0), INT(1), v[2], PTR(3), v[4], INT(5), INT(6), PTR(7), (size_t)v[8],
        PTR(9), PTR(10), STREAM(11))
WRAPPER(tq_swiglu_linear_backward, "pilpppliiplppp", PTR(0), INT(1), v[2], PTR(3), PTR(4), PTR(5), v[6], INT(7),
        INT(8), PTR(9), (size_t)v[10], PTR(11), PTR(12), STREAM(13))

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))call_##name, METH_FASTCALL, NULL}
#define BIND(name)                                         \
  if (!strcmp(which, #name)) {                             \
    fn_##name = (__typeof__(&name))(intptr_t)address;      \
    Py_RETURN_NONE;                                        \
  }

static PyObject* bind(PyObject* self, PyObject* args) {
  const char* which;
  unsigned long long address;
  (void)self;
  if (!PyArg_ParseTuple(args, "sK", &which, &address)) return NULL;
  BIND(tq_router_scored)
  BIND(tq_router_scored_backward)
  BIND(tq_fp4_quantize)
  BIND(tq_fp4_dequantize)
  BIND(tq_fp4_linear)
  BIND(tq_fp4_moe_forward)
  BIND(tq_fp4_moe_mlp_forward)
  BIND(tq_rms_norm)
  BIND(tq_rms_norm_backward)
  BIND(tq_fp8_quantize)
  BIND(tq_fp8_dequantize)
  BIND(tq_fp8_linear)
  BIND(tq_fp8_moe_forward)
  BIND(tq_fp8_moe_mlp_forward)
  BIND(tq_swiglu_linear)
  BIND(tq_swiglu_linear_backward)
  PyErr_Format(PyExc_KeyError, "no wrapper of %s", which);
  return NULL;
}

static PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, NULL},
                                METHOD(tq_router_scored),
                                METHOD(tq_router_scored_backward),
                                METHOD(tq_fp4_quantize),
                                METHOD(tq_fp4_dequantize),
                                METHOD(tq_fp4_linear),
                                METHOD(tq_fp4_moe_forward),
                                METHOD(tq_fp4_moe_mlp_forward),
                                METHOD(tq_rms_norm),
                                METHOD(tq_rms_norm_backward),
                                METHOD(tq_fp8_quantize),
                                METHOD(tq_fp8_dequantize),
                                METHOD(tq_fp8_linear),
                                METHOD(tq_fp8_moe_forward),
                                METHOD(tq_fp8_moe_mlp_forward),
                                METHOD(tq_swiglu_linear),
                                METHOD(tq_swiglu_linear_backward),
                                {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tqcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__tqcall(void) { return PyModule_Create(&module); }
