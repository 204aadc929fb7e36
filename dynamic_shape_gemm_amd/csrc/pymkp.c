/* Argument marshalling for the GEMM, vocabulary-loss and 8-bit entry points of
 * libmkp.so, as a CPython extension: integers in (and floats, for the losses),
 * the C ABI's status code out.  It exists because a
 * ctypes call converts each of its 10-14 arguments through Python objects,
 * which for the smallest GEMMs costs as much host time as the launch itself.
 * Every argument is a Python int (device addresses included); the stream is
 * the raw stream handle (void *, 0 for the null stream).  Nothing here
 * computes: each function converts its arguments and calls the entry point
 * of the same name.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

#include "mkp.h"

static int get_i64(PyObject* o, int64_t* v) {
    long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) return -1;
    *v = (int64_t)x;
    return 0;
}

static int get_ptr(PyObject* o, void** p) {
    void* x = PyLong_AsVoidPtr(o);
    if (x == NULL && PyErr_Occurred()) return -1;
    *p = x;
    return 0;
}

static int check_nargs(Py_ssize_t n, Py_ssize_t want, const char* name) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", name, want, n);
        return -1;
    }
    return 0;
}

/* (M, N, K, A, lda, B, ldb, C, ldc, stream) */
typedef int (*gemm_fn)(int64_t, int64_t, int64_t, const void*, int64_t, const void*, int64_t, float*, int64_t,
                       void*);
/* (batch, M, N, K, A, lda, sA, B, ldb, sB, C, ldc, sC, stream) */
typedef int (*batched_fn)(int64_t, int64_t, int64_t, int64_t, const void*, int64_t, int64_t, const void*, int64_t,
                          int64_t, float*, int64_t, int64_t, void*);

static PyObject* call_gemm(gemm_fn fn, const char* name, PyObject* const* a, Py_ssize_t n) {
    if (check_nargs(n, 10, name)) return NULL;
    int64_t M, N, K, lda, ldb, ldc;
    void *A, *B, *C, *st;
    if (get_i64(a[0], &M) || get_i64(a[1], &N) || get_i64(a[2], &K) || get_ptr(a[3], &A) || get_i64(a[4], &lda) ||
        get_ptr(a[5], &B) || get_i64(a[6], &ldb) || get_ptr(a[7], &C) || get_i64(a[8], &ldc) || get_ptr(a[9], &st))
        return NULL;
    return PyLong_FromLong(fn(M, N, K, A, lda, B, ldb, (float*)C, ldc, st));
}

static PyObject* call_batched(batched_fn fn, const char* name, PyObject* const* a, Py_ssize_t n) {
    if (check_nargs(n, 14, name)) return NULL;
    int64_t bt, M, N, K, lda, sA, ldb, sB, ldc, sC;
    void *A, *B, *C, *st;
    if (get_i64(a[0], &bt) || get_i64(a[1], &M) || get_i64(a[2], &N) || get_i64(a[3], &K) || get_ptr(a[4], &A) ||
        get_i64(a[5], &lda) || get_i64(a[6], &sA) || get_ptr(a[7], &B) || get_i64(a[8], &ldb) ||
        get_i64(a[9], &sB) || get_ptr(a[10], &C) || get_i64(a[11], &ldc) || get_i64(a[12], &sC) ||
        get_ptr(a[13], &st))
        return NULL;
    return PyLong_FromLong(fn(bt, M, N, K, A, lda, sA, B, ldb, sB, (float*)C, ldc, sC, st));
}

static PyObject* py_gemm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    return call_gemm(mkp_gemm, "gemm", a, n);
}
static PyObject* py_gemm_bt(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    return call_gemm(mkp_gemm_bt, "gemm_bt", a, n);
}
static PyObject* py_gemm_batched(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    return call_batched(mkp_gemm_batched, "gemm_batched", a, n);
}
static PyObject* py_gemm_batched_bt(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    return call_batched(mkp_gemm_batched_bt, "gemm_batched_bt", a, n);
}

/* The vocabulary losses' and 8-bit calls' arguments, by kind: i an integer, p an address, f a
 * float, in the order of the C ABI. */
typedef union {
    int64_t i;
    void* p;
    float f;
} arg_t;

static int get_args(const char* kinds, PyObject* const* a, Py_ssize_t n, arg_t* v, const char* name) {
    Py_ssize_t want = (Py_ssize_t)strlen(kinds);
    if (check_nargs(n, want, name)) return -1;
    for (Py_ssize_t k = 0; k < want; ++k) {
        if (kinds[k] == 'i') {
            if (get_i64(a[k], &v[k].i)) return -1;
        } else if (kinds[k] == 'p') {
            if (get_ptr(a[k], &v[k].p)) return -1;
        } else {
            double d = PyFloat_AsDouble(a[k]);
            if (d == -1.0 && PyErr_Occurred()) return -1;
            v[k].f = (float)d;
        }
    }
    return 0;
}

static PyObject* py_linear_xent(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    arg_t v[18];
    if (get_args("iiipipippffffpppip", a, n, v, "linear_xent")) return NULL;
    return PyLong_FromLong(mkp_linear_xent(v[0].i, v[1].i, v[2].i, v[3].p, v[4].i, v[5].p, v[6].i, v[7].p, v[8].p, v[9].f,
                                           v[10].f, v[11].f, v[12].f, v[13].p, v[14].p, v[15].p, v[16].i, v[17].p));
}
static PyObject* py_linear_xent_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    arg_t v[24];
    if (get_args("iiipipippffffpppipipipip", a, n, v, "linear_xent_backward")) return NULL;
    return PyLong_FromLong(mkp_linear_xent_backward(
        v[0].i, v[1].i, v[2].i, v[3].p, v[4].i, v[5].p, v[6].i, v[7].p, v[8].p, v[9].f, v[10].f, v[11].f, v[12].f, v[13].p,
        v[14].p, v[15].p, v[16].i, v[17].p, v[18].i, v[19].p, (int)v[20].i, v[21].p, v[22].i, v[23].p));
}
static PyObject* py_linear_distill(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    arg_t v[22];
    if (get_args("iiipipipipipipfffpppip", a, n, v, "linear_distill")) return NULL;
    return PyLong_FromLong(mkp_linear_distill(v[0].i, v[1].i, v[2].i, v[3].p, v[4].i, v[5].p, v[6].i, v[7].p, v[8].i, v[9].p,
                                              v[10].i, v[11].p, v[12].i, v[13].p, v[14].f, v[15].f, v[16].f, v[17].p,
                                              v[18].p, v[19].p, v[20].i, v[21].p));
}
static PyObject* py_linear_distill_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    arg_t v[28];
    if (get_args("iiipipipipipipfffpppipipipip", a, n, v, "linear_distill_backward")) return NULL;
    return PyLong_FromLong(mkp_linear_distill_backward(
        v[0].i, v[1].i, v[2].i, v[3].p, v[4].i, v[5].p, v[6].i, v[7].p, v[8].i, v[9].p, v[10].i, v[11].p, v[12].i, v[13].p,
        v[14].f, v[15].f, v[16].f, v[17].p, v[18].p, v[19].p, v[20].i, v[21].p, v[22].i, v[23].p, (int)v[24].i, v[25].p,
        v[26].i, v[27].p));
}

static PyObject* py_quantize_rows(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    arg_t v[11];
    if (get_args("iipiiipipip", a, n, v, "quantize_rows")) return NULL;
    return PyLong_FromLong(
        mkp_quantize_rows(v[0].i, v[1].i, v[2].p, v[3].i, (int)v[4].i, v[5].i, v[6].p, v[7].i, v[8].p, v[9].i, v[10].p));
}
static PyObject* py_dequantize_rows(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    arg_t v[11];
    if (get_args("iipipiipiip", a, n, v, "dequantize_rows")) return NULL;
    return PyLong_FromLong(
        mkp_dequantize_rows(v[0].i, v[1].i, v[2].p, v[3].i, v[4].p, v[5].i, v[6].i, v[7].p, v[8].i, (int)v[9].i, v[10].p));
}
static PyObject* py_linear_i8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    arg_t v[18];
    if (get_args("iiipiippippipiipip", a, n, v, "linear_i8")) return NULL;
    return PyLong_FromLong(mkp_linear_i8(v[0].i, v[1].i, v[2].i, v[3].p, v[4].i, (int)v[5].i, v[6].p, v[7].p, v[8].i, v[9].p,
                                         v[10].p, (int)v[11].i, v[12].p, v[13].i, (int)v[14].i, v[15].p, v[16].i, v[17].p));
}
static PyObject* py_linear_q8_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    arg_t v[24];
    if (get_args("iiipiipippipiiipipiippip", a, n, v, "linear_q8_backward")) return NULL;
    return PyLong_FromLong(mkp_linear_q8_backward(
        v[0].i, v[1].i, v[2].i, v[3].p, v[4].i, (int)v[5].i, v[6].p, v[7].i, v[8].p, v[9].p, v[10].i, v[11].p, v[12].i, v[13].i,
        (int)v[14].i, v[15].p, v[16].i, v[17].p, v[18].i, (int)v[19].i, v[20].p, v[21].p, v[22].i, v[23].p));
}

static PyMethodDef methods[] = {
    {"gemm", (PyCFunction)(void (*)(void))py_gemm, METH_FASTCALL, "mkp_gemm"},
    {"gemm_bt", (PyCFunction)(void (*)(void))py_gemm_bt, METH_FASTCALL, "mkp_gemm_bt"},
    {"gemm_batched", (PyCFunction)(void (*)(void))py_gemm_batched, METH_FASTCALL, "mkp_gemm_batched"},
    {"gemm_batched_bt", (PyCFunction)(void (*)(void))py_gemm_batched_bt, METH_FASTCALL, "mkp_gemm_batched_bt"},
    {"linear_xent", (PyCFunction)(void (*)(void))py_linear_xent, METH_FASTCALL, "mkp_linear_xent"},
    {"linear_xent_backward", (PyCFunction)(void (*)(void))py_linear_xent_backward, METH_FASTCALL,
     "mkp_linear_xent_backward"},
    {"linear_distill", (PyCFunction)(void (*)(void))py_linear_distill, METH_FASTCALL, "mkp_linear_distill"},
    {"linear_distill_backward", (PyCFunction)(void (*)(void))py_linear_distill_backward, METH_FASTCALL,
     "mkp_linear_distill_backward"},
    {"quantize_rows", (PyCFunction)(void (*)(void))py_quantize_rows, METH_FASTCALL, "mkp_quantize_rows"},
    {"dequantize_rows", (PyCFunction)(void (*)(void))py_dequantize_rows, METH_FASTCALL, "mkp_dequantize_rows"},
    {"linear_i8", (PyCFunction)(void (*)(void))py_linear_i8, METH_FASTCALL, "mkp_linear_i8"},
    {"linear_q8_backward", (PyCFunction)(void (*)(void))py_linear_q8_backward, METH_FASTCALL, "mkp_linear_q8_backward"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mkpfast", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__mkpfast(void) { return PyModule_Create(&module); }
