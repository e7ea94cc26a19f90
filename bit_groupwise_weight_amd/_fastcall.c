/* Argument marshalling for eager calls of the library from Python.
 *
 * A CPython extension with two functions for lowbit_linear:
 *   bind(fn, act, packed, scales, zeros, bias, bits, group, N, K) -> capsule
 *       keeps the arguments of one layer that do not change between calls,
 *       and fn, the address of lowbit_linear in the loaded library;
 *   call(capsule, x, y, M, workspace, workspace_bytes, stream) -> status
 *       calls fn with them and the per-call arguments (device pointers and
 *       the stream handle as Python ints, 0 for NULL).
 * and one for each entry point of the 8-bit path, around the experts and of
 * the adapters, named as it, which takes the entry point's address in the
 * loaded library and then its arguments.
 * It does no arithmetic of the layer and holds no state beyond the capsule:
 * every argument is passed on unchanged and the library validates them.
 * (ctypes builds and converts fifteen argument objects per call; this takes
 * seven ints through the vectorcall protocol.)
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stddef.h>
#include <stdint.h>

#include "lowbit.h"

typedef __typeof__(lowbit_linear)* linear_fn;   /* the declared signature */

typedef struct {
  linear_fn fn;
  lowbit_dtype act;
  int bits, group;
  const uint8_t* packed;
  const void *scales, *zeros, *bias;
  int64_t N, K;
} bound_layer;

static const char kCapsule[] = "lowbit.bound_layer";

static void free_bound(PyObject* cap) {
  void* p = PyCapsule_GetPointer(cap, kCapsule);
  PyMem_Free(p);
}

static void* as_ptr(PyObject* o) {
  if (o == Py_None) return NULL;
  return PyLong_AsVoidPtr(o);
}

static PyObject* bind(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  (void)self;
  if (nargs != 10) {
    PyErr_SetString(PyExc_TypeError, "bind takes 10 arguments");
    return NULL;
  }
  bound_layer* b = (bound_layer*)PyMem_Malloc(sizeof(bound_layer));
  if (!b) return PyErr_NoMemory();
  b->fn = (linear_fn)as_ptr(args[0]);
  b->act = (lowbit_dtype)PyLong_AsLong(args[1]);
  b->packed = (const uint8_t*)as_ptr(args[2]);
  b->scales = as_ptr(args[3]);
  b->zeros = as_ptr(args[4]);
  b->bias = as_ptr(args[5]);
  b->bits = (int)PyLong_AsLong(args[6]);
  b->group = (int)PyLong_AsLong(args[7]);
  b->N = PyLong_AsLongLong(args[8]);
  b->K = PyLong_AsLongLong(args[9]);
  if (PyErr_Occurred() || !b->fn) {
    PyMem_Free(b);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null function address");
    return NULL;
  }
  PyObject* cap = PyCapsule_New(b, kCapsule, free_bound);
  if (!cap) PyMem_Free(b);
  return cap;
}

static PyObject* call(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  (void)self;
  if (nargs != 7) {
    PyErr_SetString(PyExc_TypeError, "call takes 7 arguments");
    return NULL;
  }
  const bound_layer* b = (const bound_layer*)PyCapsule_GetPointer(args[0], kCapsule);
  if (!b) return NULL;
  void* x = as_ptr(args[1]);
  void* y = as_ptr(args[2]);
  const int64_t M = PyLong_AsLongLong(args[3]);
  void* ws = as_ptr(args[4]);
  const size_t ws_bytes = (size_t)PyLong_AsSize_t(args[5]);
  void* stream = as_ptr(args[6]);
  if (PyErr_Occurred()) return NULL;
  const lowbit_status st = b->fn(x, b->act, b->packed, b->scales, b->zeros, b->bias, y, b->bits, b->group,
                       M, b->N, b->K, ws, ws_bytes, stream);
  return PyLong_FromLong((long)st);
}

/* The 8-bit path: args[0] is the entry point's address, the rest its arguments
 * (pointers and the stream as ints or None). */
#define PTR(i) as_ptr(args[i])
#define I64(i) ((int64_t)PyLong_AsLongLong(args[i]))
#define INT(i) ((int)PyLong_AsLong(args[i]))
#define ENTRY(name, count, ...)                                                         \
  static PyObject* py_##name(PyObject* self, PyObject* const* args, Py_ssize_t nargs) { \
    (void)self;                                                                         \
    if (nargs != (count) + 1) {                                                         \
      PyErr_SetString(PyExc_TypeError, #name " takes an address and " #count " arguments"); \
      return NULL;                                                                      \
    }                                                                                   \
    __typeof__(name)* fn = (__typeof__(name)*)as_ptr(args[0]);                          \
    if (!fn) {                                                                          \
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null function address"); \
      return NULL;                                                                      \
    }                                                                                   \
    __VA_ARGS__                                                                         \
    if (PyErr_Occurred()) return NULL;                                                  \
    return PyLong_FromLong((long)CALL);                                                 \
  }

/* (arguments are converted before the call, so that a bad one is a Python error) */
#define CALL fn(a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13)
ENTRY(lowbit_add_rmsnorm_q8, 13, const void* a1 = PTR(1); const void* a2 = PTR(2); const void* a3 = PTR(3);
      float a4 = (float)PyFloat_AsDouble(args[4]); lowbit_dtype a5 = (lowbit_dtype)INT(5); int64_t a6 = I64(6);
      int64_t a7 = I64(7); lowbit_q8_format a8 = (lowbit_q8_format)INT(8); void* a9 = PTR(9);
      float* a10 = (float*)PTR(10); void* a11 = PTR(11); void* a12 = PTR(12); void* a13 = PTR(13);)
#undef CALL
#define CALL fn(a1, a2, a3, a4, a5, a6, a7)
ENTRY(lowbit_quantize_act_f8, 7, const void* a1 = PTR(1); lowbit_dtype a2 = (lowbit_dtype)INT(2);
      int64_t a3 = I64(3); int64_t a4 = I64(4); uint8_t* a5 = (uint8_t*)PTR(5); float* a6 = (float*)PTR(6);
      void* a7 = PTR(7);)
#undef CALL
#define CALL fn(a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13)
ENTRY(lowbit_linear_f8, 13, const uint8_t* a1 = (const uint8_t*)PTR(1); const float* a2 = (const float*)PTR(2);
      const uint8_t* a3 = (const uint8_t*)PTR(3); const float* a4 = (const float*)PTR(4); const void* a5 = PTR(5);
      void* a6 = PTR(6); lowbit_dtype a7 = (lowbit_dtype)INT(7); int64_t a8 = I64(8); int64_t a9 = I64(9);
      int64_t a10 = I64(10); void* a11 = PTR(11); size_t a12 = (size_t)I64(12); void* a13 = PTR(13);)
#undef CALL
#define CALL fn(a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, a15, a16, a17)
ENTRY(lowbit_linear_f8_grouped, 17, const uint8_t* a1 = (const uint8_t*)PTR(1);
      const float* a2 = (const float*)PTR(2); const int32_t* a3 = (const int32_t*)PTR(3);
      const int32_t* a4 = (const int32_t*)PTR(4); const uint8_t* a5 = (const uint8_t*)PTR(5);
      const float* a6 = (const float*)PTR(6); const void* a7 = PTR(7); void* a8 = PTR(8);
      lowbit_dtype a9 = (lowbit_dtype)INT(9); int64_t a10 = I64(10); int64_t a11 = I64(11); int64_t a12 = I64(12);
      int64_t a13 = I64(13); int64_t a14 = I64(14); void* a15 = PTR(15); size_t a16 = (size_t)I64(16);
      void* a17 = PTR(17);)
#undef CALL
#define CALL fn(a1, a2, a3, a4, a5, a6)
ENTRY(lowbit_linear_f8_workspace_bytes, 6, int64_t a1 = I64(1); int64_t a2 = I64(2); int64_t a3 = I64(3);
      int64_t a4 = I64(4); int64_t a5 = I64(5); lowbit_dtype a6 = (lowbit_dtype)INT(6);)
#undef CALL

#define CALL fn(a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, a15)
ENTRY(lowbit_moe_route, 15, const void* a1 = PTR(1); lowbit_dtype a2 = (lowbit_dtype)INT(2);
      const float* a3 = (const float*)PTR(3); int64_t a4 = I64(4); int64_t a5 = I64(5); int64_t a6 = I64(6);
      lowbit_route_score a7 = (lowbit_route_score)INT(7); int64_t a8 = I64(8); int64_t a9 = I64(9);
      int a10 = INT(10); int a11 = INT(11); float a12 = (float)PyFloat_AsDouble(args[12]);
      int32_t* a13 = (int32_t*)PTR(13); float* a14 = (float*)PTR(14); void* a15 = PTR(15);)
#undef CALL
#define CALL fn(a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11)
ENTRY(lowbit_group_rows, 11, const void* a1 = PTR(1); int a2 = INT(2); int64_t a3 = I64(3); int64_t a4 = I64(4);
      int64_t a5 = I64(5); int32_t* a6 = (int32_t*)PTR(6); int32_t* a7 = (int32_t*)PTR(7);
      int32_t* a8 = (int32_t*)PTR(8); void* a9 = PTR(9); size_t a10 = (size_t)I64(10); void* a11 = PTR(11);)
#undef CALL
#define CALL fn(a1, a2, a3)
ENTRY(lowbit_group_rows_workspace_bytes, 3, int64_t a1 = I64(1); int64_t a2 = I64(2); int64_t a3 = I64(3);)
#undef CALL
#define CALL fn(a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11)
ENTRY(lowbit_moe_combine, 11, const void* a1 = PTR(1); const int32_t* a2 = (const int32_t*)PTR(2);
      const float* a3 = (const float*)PTR(3); const void* a4 = PTR(4); void* a5 = PTR(5);
      lowbit_dtype a6 = (lowbit_dtype)INT(6); int64_t a7 = I64(7); int64_t a8 = I64(8); int64_t a9 = I64(9);
      int64_t a10 = I64(10); void* a11 = PTR(11);)
#undef CALL
#define CALL fn(a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, a15, a16, a17, a18)
ENTRY(lowbit_lora, 18, const void* a1 = PTR(1); const void* a2 = PTR(2); const void* a3 = PTR(3);
      const float* a4 = (const float*)PTR(4); const int32_t* a5 = (const int32_t*)PTR(5);
      const int32_t* a6 = (const int32_t*)PTR(6); const void* a7 = PTR(7); void* a8 = PTR(8);
      lowbit_dtype a9 = (lowbit_dtype)INT(9); int64_t a10 = I64(10); int64_t a11 = I64(11); int64_t a12 = I64(12);
      int64_t a13 = I64(13); int64_t a14 = I64(14); int64_t a15 = I64(15); void* a16 = PTR(16);
      size_t a17 = (size_t)I64(17); void* a18 = PTR(18);)
#undef CALL
#define CALL fn(a1, a2, a3, a4, a5, a6)
ENTRY(lowbit_lora_workspace_bytes, 6, int64_t a1 = I64(1); int64_t a2 = I64(2); int64_t a3 = I64(3);
      int64_t a4 = I64(4); int64_t a5 = I64(5); lowbit_dtype a6 = (lowbit_dtype)INT(6);)
#undef CALL

#define METHOD(name) \
  {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, "call " #name " at the address given first"}
static PyMethodDef kMethods[] = {
    METHOD(lowbit_add_rmsnorm_q8), METHOD(lowbit_quantize_act_f8), METHOD(lowbit_linear_f8),
    METHOD(lowbit_linear_f8_grouped), METHOD(lowbit_linear_f8_workspace_bytes), METHOD(lowbit_moe_route),
    METHOD(lowbit_group_rows), METHOD(lowbit_group_rows_workspace_bytes), METHOD(lowbit_moe_combine), METHOD(lowbit_lora), METHOD(lowbit_lora_workspace_bytes),
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, "bind one layer's fixed arguments"},
    {"call", (PyCFunction)(void (*)(void))call, METH_FASTCALL, "call lowbit_linear for a bound layer"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_lowbit_fastcall",
                                     "argument marshalling for eager calls of the library", -1,
                                     kMethods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__lowbit_fastcall(void) { return PyModule_Create(&kModule); }
