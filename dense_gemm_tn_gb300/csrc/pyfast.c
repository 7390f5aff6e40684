/* CPython-API binding of the C ABI's compute calls (include/tn_gemm.h).
 *
 * Argument marshalling only, with the C ABI's names and argument order: sizes
 * and leading dimensions are Python ints, pointers are ints (device or host
 * addresses) or None for NULL, scales are floats, and each call returns the
 * C ABI's gemm_status_t as an int.  Every call goes straight to the C ABI
 * function of libdense_gemm_tn.so.
 *
 * Why it exists: a ctypes call with ten arguments costs about 1.5 us of host
 * time on the GPU machine's cores, as much as a whole small GEMM on the GPU; a
 * METH_FASTCALL function converts the same arguments in a fraction of that.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <string.h>

#include "tn_gemm.h"

/* Reads args[i] as a 64-bit int; returns 0 and sets an exception on failure. */
static int arg_i64(PyObject *const *args, Py_ssize_t i, int64_t *out)
{
    long long v = PyLong_AsLongLong(args[i]);
    if (v == -1 && PyErr_Occurred()) return 0;
    *out = (int64_t)v;
    return 1;
}

static int arg_int(PyObject *const *args, Py_ssize_t i, int *out)
{
    long v = PyLong_AsLong(args[i]);
    if (v == -1 && PyErr_Occurred()) return 0;
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "argument does not fit a C int");
        return 0;
    }
    *out = (int)v;
    return 1;
}

/* A pointer: None -> NULL, else a non-negative int address. */
static int arg_ptr(PyObject *const *args, Py_ssize_t i, void **out)
{
    if (args[i] == Py_None) {
        *out = NULL;
        return 1;
    }
    void *p = PyLong_AsVoidPtr(args[i]);
    if (p == NULL && PyErr_Occurred()) return 0;
    *out = p;
    return 1;
}

static int arg_float(PyObject *const *args, Py_ssize_t i, float *out)
{
    double v = PyFloat_AsDouble(args[i]);
    if (v == -1.0 && PyErr_Occurred()) return 0;
    *out = (float)v;
    return 1;
}

static int check_nargs(const char *name, Py_ssize_t nargs, Py_ssize_t want)
{
    if (nargs == want) return 1;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", name, want, nargs);
    return 0;
}

/* The ten-argument form shared by gemm_f16_tn and gemm_f16_tn_noalloc:
 * (M, N, K, A, lda, B, ldb, C, ldc, stream). */
typedef gemm_status_t (*f16_fn)(int64_t, int64_t, int64_t, const void *, int64_t, const void *, int64_t, void *,
                                int64_t, void *);

static PyObject *call_f16(const char *name, f16_fn fn, PyObject *const *args, Py_ssize_t nargs)
{
    int64_t M, N, K, lda, ldb, ldc;
    void *A, *B, *C, *stream;
    if (!check_nargs(name, nargs, 10) || !arg_i64(args, 0, &M) || !arg_i64(args, 1, &N) || !arg_i64(args, 2, &K) ||
        !arg_ptr(args, 3, &A) || !arg_i64(args, 4, &lda) || !arg_ptr(args, 5, &B) || !arg_i64(args, 6, &ldb) ||
        !arg_ptr(args, 7, &C) || !arg_i64(args, 8, &ldc) || !arg_ptr(args, 9, &stream))
        return NULL;
    return PyLong_FromLong((long)fn(M, N, K, A, lda, B, ldb, C, ldc, stream));
}

static PyObject *py_gemm_f16_tn(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    return call_f16("gemm_f16_tn", gemm_f16_tn, args, nargs);
}

static PyObject *py_gemm_f16_tn_noalloc(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    return call_f16("gemm_f16_tn_noalloc", gemm_f16_tn_noalloc, args, nargs);
}

/* (M, N, K, A, lda, B, ldb, C, ldc, scale_a, scale_b, stream) */
static PyObject *py_gemm_f8e4m3_tn(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    int64_t M, N, K, lda, ldb, ldc;
    void *A, *B, *C, *stream;
    float sa, sb;
    if (!check_nargs("gemm_f8e4m3_tn", nargs, 12) || !arg_i64(args, 0, &M) || !arg_i64(args, 1, &N) ||
        !arg_i64(args, 2, &K) || !arg_ptr(args, 3, &A) || !arg_i64(args, 4, &lda) || !arg_ptr(args, 5, &B) ||
        !arg_i64(args, 6, &ldb) || !arg_ptr(args, 7, &C) || !arg_i64(args, 8, &ldc) || !arg_float(args, 9, &sa) ||
        !arg_float(args, 10, &sb) || !arg_ptr(args, 11, &stream))
        return NULL;
    return PyLong_FromLong((long)gemm_f8e4m3_tn(M, N, K, A, lda, B, ldb, C, ldc, sa, sb, stream));
}

/* (M, N, K, A, lda, B, ldb, C, ldc, scale_a_ptr, scale_b_ptr, stream) */
static PyObject *py_gemm_f8e4m3_tn_dscale(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    int64_t M, N, K, lda, ldb, ldc;
    void *A, *B, *C, *sa, *sb, *stream;
    if (!check_nargs("gemm_f8e4m3_tn_dscale", nargs, 12) || !arg_i64(args, 0, &M) || !arg_i64(args, 1, &N) ||
        !arg_i64(args, 2, &K) || !arg_ptr(args, 3, &A) || !arg_i64(args, 4, &lda) || !arg_ptr(args, 5, &B) ||
        !arg_i64(args, 6, &ldb) || !arg_ptr(args, 7, &C) || !arg_i64(args, 8, &ldc) || !arg_ptr(args, 9, &sa) ||
        !arg_ptr(args, 10, &sb) || !arg_ptr(args, 11, &stream))
        return NULL;
    return PyLong_FromLong(
        (long)gemm_f8e4m3_tn_dscale(M, N, K, A, lda, B, ldb, C, ldc, (const float *)sa, (const float *)sb, stream));
}

/* (M, N, K, A, lda, B, ldb, C, ldc, scale, row_max, row_sum, stream) */
static PyObject *py_gemm_f16_tn_softmax_stats(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    int64_t M, N, K, lda, ldb, ldc;
    void *A, *B, *C, *mx, *sm, *stream;
    float scale;
    if (!check_nargs("gemm_f16_tn_softmax_stats", nargs, 13) || !arg_i64(args, 0, &M) || !arg_i64(args, 1, &N) ||
        !arg_i64(args, 2, &K) || !arg_ptr(args, 3, &A) || !arg_i64(args, 4, &lda) || !arg_ptr(args, 5, &B) ||
        !arg_i64(args, 6, &ldb) || !arg_ptr(args, 7, &C) || !arg_i64(args, 8, &ldc) ||
        !arg_float(args, 9, &scale) || !arg_ptr(args, 10, &mx) || !arg_ptr(args, 11, &sm) ||
        !arg_ptr(args, 12, &stream))
        return NULL;
    return PyLong_FromLong((long)gemm_f16_tn_softmax_stats(M, N, K, A, lda, B, ldb, C, ldc, scale, (float *)mx,
                                                           (float *)sm, stream));
}

/* (x, dtype, rows, cols, ldx, q, ldq, scale_out, stream) */
static PyObject *py_gemm_quantize_e4m3(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    void *x, *q, *scale, *stream;
    int dtype;
    int64_t rows, cols, ldx, ldq;
    if (!check_nargs("gemm_quantize_e4m3", nargs, 9) || !arg_ptr(args, 0, &x) || !arg_int(args, 1, &dtype) ||
        !arg_i64(args, 2, &rows) || !arg_i64(args, 3, &cols) || !arg_i64(args, 4, &ldx) || !arg_ptr(args, 5, &q) ||
        !arg_i64(args, 6, &ldq) || !arg_ptr(args, 7, &scale) || !arg_ptr(args, 8, &stream))
        return NULL;
    return PyLong_FromLong(
        (long)gemm_quantize_e4m3(x, dtype, rows, cols, ldx, q, ldq, (float *)scale, stream));
}

/* The calls with many arguments: `form` has one letter per argument, 'i' a C
 * int, 'l' a 64-bit int, 'p' a pointer; the values are left in v[]. */
typedef union {
    int i;
    int64_t l;
    void *p;
} arg_value;

static int read_args(const char *name, const char *form, PyObject *const *args, Py_ssize_t nargs, arg_value *v)
{
    const Py_ssize_t want = (Py_ssize_t)strlen(form);
    if (!check_nargs(name, nargs, want)) return 0;
    for (Py_ssize_t k = 0; k < want; ++k) {
        const int ok = form[k] == 'i' ? arg_int(args, k, &v[k].i)
                       : form[k] == 'l' ? arg_i64(args, k, &v[k].l) : arg_ptr(args, k, &v[k].p);
        if (!ok) return 0;
    }
    return 1;
}

/* (op, E, M, K, T, X, ldx, stride_x, Y, ldy) -> bytes */
static PyObject *py_gemm_grouped_workspace(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[10];
    if (!read_args("gemm_grouped_workspace", "illllpllpl", args, nargs, v)) return NULL;
    return PyLong_FromLongLong(gemm_grouped_workspace(v[0].i, v[1].l, v[2].l, v[3].l, v[4].l, v[5].p, v[6].l, v[7].l,
                                                      v[8].p, v[9].l));
}

/* (type, E, M, K, T, A, lda, stride_a, B, ldb, offsets, C, ldc, workspace, workspace_bytes, stream) */
static PyObject *py_gemm_tn_grouped(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[16];
    if (!read_args("gemm_tn_grouped", "illllpllplpplplp", args, nargs, v)) return NULL;
    return PyLong_FromLong((long)gemm_tn_grouped(v[0].i, v[1].l, v[2].l, v[3].l, v[4].l, v[5].p, v[6].l, v[7].l, v[8].p,
                                                 v[9].l, (const int32_t *)v[10].p, v[11].p, v[12].l, v[13].p, v[14].l,
                                                 v[15].p));
}

/* (type, E, M, K, T, A, lda, stride_a, dC, lddc, offsets, dB, lddb, workspace, workspace_bytes, stream) */
static PyObject *py_gemm_tn_grouped_grad_b(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[16];
    if (!read_args("gemm_tn_grouped_grad_b", "illllpllplpplplp", args, nargs, v)) return NULL;
    return PyLong_FromLong((long)gemm_tn_grouped_grad_b(v[0].i, v[1].l, v[2].l, v[3].l, v[4].l, v[5].p, v[6].l, v[7].l,
                                                        v[8].p, v[9].l, (const int32_t *)v[10].p, v[11].p, v[12].l,
                                                        v[13].p, v[14].l, v[15].p));
}

/* (type, E, M, K, T, dC, lddc, B, ldb, offsets, dA, ldda, stride_da, workspace, workspace_bytes, stream) */
static PyObject *py_gemm_tn_grouped_grad_a(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[16];
    if (!read_args("gemm_tn_grouped_grad_a", "illllplplppllplp", args, nargs, v)) return NULL;
    return PyLong_FromLong((long)gemm_tn_grouped_grad_a(v[0].i, v[1].l, v[2].l, v[3].l, v[4].l, v[5].p, v[6].l, v[7].p,
                                                        v[8].l, (const int32_t *)v[9].p, v[10].p, v[11].l, v[12].l,
                                                        v[13].p, v[14].l, v[15].p));
}

/* (out_type, M, N, K, A, lda, scale_a, B, ldb, scale_b, C, ldc, workspace, workspace_bytes, stream) */
static PyObject *py_gemm_i8_tn(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[15];
    if (!read_args("gemm_i8_tn", "illlplpplpplplp", args, nargs, v)) return NULL;
    return PyLong_FromLong((long)gemm_i8_tn(v[0].i, v[1].l, v[2].l, v[3].l, (const int8_t *)v[4].p, v[5].l,
                                            (const float *)v[6].p, (const int8_t *)v[7].p, v[8].l,
                                            (const float *)v[9].p, v[10].p, v[11].l, v[12].p, v[13].l, v[14].p));
}

/* (out_type, E, M, K, T, A, lda, stride_a, scale_a, B, ldb, scale_b, offsets, C, ldc, workspace, workspace_bytes, stream) */
static PyObject *py_gemm_i8_tn_grouped(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[18];
    if (!read_args("gemm_i8_tn_grouped", "illllpllpplppplplp", args, nargs, v)) return NULL;
    return PyLong_FromLong((long)gemm_i8_tn_grouped(
        v[0].i, v[1].l, v[2].l, v[3].l, v[4].l, (const int8_t *)v[5].p, v[6].l, v[7].l, (const float *)v[8].p,
        (const int8_t *)v[9].p, v[10].l, (const float *)v[11].p, (const int32_t *)v[12].p, v[13].p, v[14].l, v[15].p,
        v[16].l, v[17].p));
}

/* (x, x_type, rows, cols, ldx, q, ldq, scale, stream) */
static PyObject *py_gemm_quantize_i8_rows(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[9];
    if (!read_args("gemm_quantize_i8_rows", "pilllplpp", args, nargs, v)) return NULL;
    return PyLong_FromLong((long)gemm_quantize_i8_rows(v[0].p, v[1].i, v[2].l, v[3].l, v[4].l, (int8_t *)v[5].p, v[6].l,
                                                       (float *)v[7].p, v[8].p));
}

/* (grad, dense, E, M, K, T, A, lda, stride_a, B, ldb) -> bytes */
static PyObject *py_gemm_gated_workspace(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[11];
    if (!read_args("gemm_gated_workspace", "iillllpllpl", args, nargs, v)) return NULL;
    return PyLong_FromLongLong(gemm_gated_workspace(v[0].i, v[1].i, v[2].l, v[3].l, v[4].l, v[5].l, v[6].p, v[7].l, v[8].l,
                                                    v[9].p, v[10].l));
}

/* (type, act, E, M, K, T, A, lda, stride_a, B, ldb, offsets, H, ldh, P, ldp, workspace, workspace_bytes, stream) */
static PyObject *py_gemm_tn_gated(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[19];
    if (!read_args("gemm_tn_gated", "iillllpllplpplplplp", args, nargs, v)) return NULL;
    return PyLong_FromLong((long)gemm_tn_gated(v[0].i, v[1].i, v[2].l, v[3].l, v[4].l, v[5].l, v[6].p, v[7].l, v[8].l,
                                               v[9].p, v[10].l, (const int32_t *)v[11].p, v[12].p, v[13].l,
                                               (float *)v[14].p, v[15].l, v[16].p, v[17].l, v[18].p));
}

/* (type, act, E, M, K, T, A, lda, stride_a, B, ldb, offsets, P, ldp, dH, lddh, dA, ldda, stride_da, dB, lddb, workspace,
 * workspace_bytes, stream) */
static PyObject *py_gemm_tn_gated_grad(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[24];
    if (!read_args("gemm_tn_gated_grad", "iillllpllplpplplpllplplp", args, nargs, v)) return NULL;
    return PyLong_FromLong((long)gemm_tn_gated_grad(
        v[0].i, v[1].i, v[2].l, v[3].l, v[4].l, v[5].l, v[6].p, v[7].l, v[8].l, v[9].p, v[10].l, (const int32_t *)v[11].p,
        (const float *)v[12].p, v[13].l, v[14].p, v[15].l, v[16].p, v[17].l, v[18].l, v[19].p, v[20].l, v[21].p, v[22].l,
        v[23].p));
}

/* (grad, M, N, K, A, lda, B, ldb) -> bytes */
static PyObject *py_gemm_cross_entropy_workspace(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[8];
    if (!read_args("gemm_cross_entropy_workspace", "illlplpl", args, nargs, v)) return NULL;
    return PyLong_FromLongLong(gemm_cross_entropy_workspace(v[0].i, v[1].l, v[2].l, v[3].l, v[4].p, v[5].l, v[6].p, v[7].l));
}

/* (type, M, N, K, A, lda, B, ldb, targets, loss, lse, workspace, workspace_bytes, stream) */
static PyObject *py_gemm_tn_cross_entropy(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[14];
    if (!read_args("gemm_tn_cross_entropy", "illlplplpppplp", args, nargs, v)) return NULL;
    return PyLong_FromLong((long)gemm_tn_cross_entropy(v[0].i, v[1].l, v[2].l, v[3].l, v[4].p, v[5].l, v[6].p, v[7].l,
                                                       (const int64_t *)v[8].p, (float *)v[9].p, (float *)v[10].p, v[11].p,
                                                       v[12].l, v[13].p));
}

/* (type, M, N, K, A, lda, B, ldb, targets, lse, dloss, dA, ldda, dB, lddb, workspace, workspace_bytes, stream) */
static PyObject *py_gemm_tn_cross_entropy_grad(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[18];
    if (!read_args("gemm_tn_cross_entropy_grad", "illlplplpppplplplp", args, nargs, v)) return NULL;
    return PyLong_FromLong((long)gemm_tn_cross_entropy_grad(
        v[0].i, v[1].l, v[2].l, v[3].l, v[4].p, v[5].l, v[6].p, v[7].l, (const int64_t *)v[8].p, (const float *)v[9].p,
        (const float *)v[10].p, v[11].p, v[12].l, v[13].p, v[14].l, v[15].p, v[16].l, v[17].p));
}

/* (type, M, N, K, A, lda, scale_a, ld_scale, group, B, ldb, C, ldc, stream) */
static PyObject *py_gemm_w4_tn(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[14];
    if (!read_args("gemm_w4_tn", "illlplpllplplp", args, nargs, v)) return NULL;
    return PyLong_FromLong((long)gemm_w4_tn(v[0].i, v[1].l, v[2].l, v[3].l, v[4].p, v[5].l, v[6].p, v[7].l, v[8].l, v[9].p,
                                            v[10].l, v[11].p, v[12].l, v[13].p));
}

/* (x, x_type, rows, cols, ldx, group, q, ldq, scale_type, scale, ld_scale, stream) */
static PyObject *py_gemm_quantize_w4_rows(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    arg_value v[12];
    if (!read_args("gemm_quantize_w4_rows", "pillllpliplp", args, nargs, v)) return NULL;
    return PyLong_FromLong((long)gemm_quantize_w4_rows(v[0].p, v[1].i, v[2].l, v[3].l, v[4].l, v[5].l, v[6].p, v[7].l,
                                                       v[8].i, v[9].p, v[10].l, v[11].p));
}

static PyMethodDef methods[] = {
    {"gemm_f16_tn", (PyCFunction)(void (*)(void))py_gemm_f16_tn, METH_FASTCALL,
     "gemm_f16_tn(M, N, K, A, lda, B, ldb, C, ldc, stream) -> status"},
    {"gemm_f16_tn_noalloc", (PyCFunction)(void (*)(void))py_gemm_f16_tn_noalloc, METH_FASTCALL,
     "gemm_f16_tn_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream) -> status"},
    {"gemm_f8e4m3_tn", (PyCFunction)(void (*)(void))py_gemm_f8e4m3_tn, METH_FASTCALL,
     "gemm_f8e4m3_tn(M, N, K, A, lda, B, ldb, C, ldc, scale_a, scale_b, stream) -> status"},
    {"gemm_f8e4m3_tn_dscale", (PyCFunction)(void (*)(void))py_gemm_f8e4m3_tn_dscale, METH_FASTCALL,
     "gemm_f8e4m3_tn_dscale(M, N, K, A, lda, B, ldb, C, ldc, scale_a_ptr, scale_b_ptr, stream) -> status"},
    {"gemm_f16_tn_softmax_stats", (PyCFunction)(void (*)(void))py_gemm_f16_tn_softmax_stats, METH_FASTCALL,
     "gemm_f16_tn_softmax_stats(M, N, K, A, lda, B, ldb, C, ldc, scale, row_max, row_sum, stream) -> status"},
    {"gemm_quantize_e4m3", (PyCFunction)(void (*)(void))py_gemm_quantize_e4m3, METH_FASTCALL,
     "gemm_quantize_e4m3(x, dtype, rows, cols, ldx, q, ldq, scale_out, stream) -> status"},
    {"gemm_grouped_workspace", (PyCFunction)(void (*)(void))py_gemm_grouped_workspace, METH_FASTCALL,
     "gemm_grouped_workspace(op, E, M, K, T, X, ldx, stride_x, Y, ldy) -> bytes"},
    {"gemm_tn_grouped", (PyCFunction)(void (*)(void))py_gemm_tn_grouped, METH_FASTCALL,
     "gemm_tn_grouped(type, E, M, K, T, A, lda, stride_a, B, ldb, offsets, C, ldc, workspace, workspace_bytes, stream) "
     "-> status"},
    {"gemm_tn_grouped_grad_b", (PyCFunction)(void (*)(void))py_gemm_tn_grouped_grad_b, METH_FASTCALL,
     "gemm_tn_grouped_grad_b(type, E, M, K, T, A, lda, stride_a, dC, lddc, offsets, dB, lddb, workspace, "
     "workspace_bytes, stream) -> status"},
    {"gemm_tn_grouped_grad_a", (PyCFunction)(void (*)(void))py_gemm_tn_grouped_grad_a, METH_FASTCALL,
     "gemm_tn_grouped_grad_a(type, E, M, K, T, dC, lddc, B, ldb, offsets, dA, ldda, stride_da, workspace, "
     "workspace_bytes, stream) -> status"},
    {"gemm_i8_tn", (PyCFunction)(void (*)(void))py_gemm_i8_tn, METH_FASTCALL,
     "gemm_i8_tn(out_type, M, N, K, A, lda, scale_a, B, ldb, scale_b, C, ldc, workspace, workspace_bytes, stream) -> "
     "status"},
    {"gemm_i8_tn_grouped", (PyCFunction)(void (*)(void))py_gemm_i8_tn_grouped, METH_FASTCALL,
     "gemm_i8_tn_grouped(out_type, E, M, K, T, A, lda, stride_a, scale_a, B, ldb, scale_b, offsets, C, ldc, workspace, "
     "workspace_bytes, stream) -> status"},
    {"gemm_quantize_i8_rows", (PyCFunction)(void (*)(void))py_gemm_quantize_i8_rows, METH_FASTCALL,
     "gemm_quantize_i8_rows(x, x_type, rows, cols, ldx, q, ldq, scale, stream) -> status"},
    {"gemm_gated_workspace", (PyCFunction)(void (*)(void))py_gemm_gated_workspace, METH_FASTCALL,
     "gemm_gated_workspace(grad, dense, E, M, K, T, A, lda, stride_a, B, ldb) -> bytes"},
    {"gemm_tn_gated", (PyCFunction)(void (*)(void))py_gemm_tn_gated, METH_FASTCALL,
     "gemm_tn_gated(type, act, E, M, K, T, A, lda, stride_a, B, ldb, offsets, H, ldh, P, ldp, workspace, workspace_bytes, "
     "stream) -> status"},
    {"gemm_tn_gated_grad", (PyCFunction)(void (*)(void))py_gemm_tn_gated_grad, METH_FASTCALL,
     "gemm_tn_gated_grad(type, act, E, M, K, T, A, lda, stride_a, B, ldb, offsets, P, ldp, dH, lddh, dA, ldda, stride_da, "
     "dB, lddb, workspace, workspace_bytes, stream) -> status"},
    {"gemm_cross_entropy_workspace", (PyCFunction)(void (*)(void))py_gemm_cross_entropy_workspace, METH_FASTCALL,
     "gemm_cross_entropy_workspace(grad, M, N, K, A, lda, B, ldb) -> bytes"},
    {"gemm_tn_cross_entropy", (PyCFunction)(void (*)(void))py_gemm_tn_cross_entropy, METH_FASTCALL,
     "gemm_tn_cross_entropy(type, M, N, K, A, lda, B, ldb, targets, loss, lse, workspace, workspace_bytes, stream) -> "
     "status"},
    {"gemm_tn_cross_entropy_grad", (PyCFunction)(void (*)(void))py_gemm_tn_cross_entropy_grad, METH_FASTCALL,
     "gemm_tn_cross_entropy_grad(type, M, N, K, A, lda, B, ldb, targets, lse, dloss, dA, ldda, dB, lddb, workspace, "
     "workspace_bytes, stream) -> status"},
    {"gemm_w4_tn", (PyCFunction)(void (*)(void))py_gemm_w4_tn, METH_FASTCALL,
     "gemm_w4_tn(type, M, N, K, A, lda, scale_a, ld_scale, group, B, ldb, C, ldc, stream) -> status"},
    {"gemm_quantize_w4_rows", (PyCFunction)(void (*)(void))py_gemm_quantize_w4_rows, METH_FASTCALL,
     "gemm_quantize_w4_rows(x, x_type, rows, cols, ldx, group, q, ldq, scale_type, scale, ld_scale, stream) -> status"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tn_fast",
                                    "CPython-API binding of the dense TN GEMM C ABI's compute calls.", -1, methods};

PyMODINIT_FUNC PyInit__tn_fast(void) { return PyModule_Create(&module); }
