/* py_calls.c -- the Python side of the MXFP4 and 16-bit entry points: arguments from Python objects to
 * the C calls of include/fgemm.h.  (Of a small call's 5 us on the host, ctypes and conversions
 * in Python took 3; here they take under 1.)
 *
 * A matrix may be a CUDA tensor (its data_ptr() is passed) or an address; an unquantised one
 * must have the call's element type.  A call's tensors have to be on the current device, where the
 * library launches.  Nothing of the library is linked: bind() is given the entries' addresses. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <cuda_runtime_api.h>

#include "fgemm.h"

static struct {
    fgemm_status (*quantize)(fgemm_dtype, int, int, const void *, int, void *, int, void *, void *, int, void *, cudaStream_t);
    fgemm_status (*quantize_grad)(fgemm_dtype, int, int, const void *, int, const void *, int, void *, int, void *, void *, int,
                                  void *, float *, void *, size_t, cudaStream_t);
    fgemm_status (*dequantize)(fgemm_dtype, int, int, const void *, int, const void *, void *, int, cudaStream_t);
    fgemm_status (*gemm)(fgemm_dtype, int, int, int, float, const void *, int, const void *, const void *, int, const void *,
                         float, void *, int, const float *, int, cudaStream_t);
    fgemm_status (*linear)(fgemm_dtype, int, int, int, const void *, int, const void *, int, const void *, const float *, int,
                           void *, int, void *, size_t, cudaStream_t);
    fgemm_status (*gemm16)(fgemm_dtype, fgemm_dtype, fgemm_op, fgemm_op, int, int, int, float, const void *, int, const void *, int,
                           const float *, fgemm_activation, void *, int, float, const void *, int, void *, int, void *, size_t,
                           cudaStream_t);
    fgemm_status (*gemm16_grad)(fgemm_dtype, fgemm_dtype, fgemm_op, fgemm_op, int, int, int, float, const void *, int, const void *,
                                int, fgemm_activation, const void *, int, void *, int, float *, void *, size_t, cudaStream_t);
    fgemm_status (*gemm16_grouped)(fgemm_dtype, fgemm_dtype, fgemm_op, int, int, int, int, const int *, float, const void *, int,
                                   const void *, int, long long, const float *, fgemm_activation, void *, int, float, const void *,
                                   int, void *, int, void *, size_t, cudaStream_t);
    fgemm_status (*gemm16_grouped_grad)(fgemm_dtype, fgemm_dtype, fgemm_op, int, int, int, int, const int *, float, const void *,
                                        int, const void *, int, long long, fgemm_activation, const void *, int, void *, int,
                                        float *, void *, size_t, cudaStream_t);
    fgemm_status (*gemm16_weight_grad)(fgemm_dtype, fgemm_dtype, int, int, int, int, const int *, float, const void *, int,
                                       const void *, int, float, void *, int, long long, void *, size_t, cudaStream_t);
    fgemm_status (*act16_grad)(fgemm_dtype, int, int, int, const int *, fgemm_activation, const void *, int, const void *, int,
                               void *, int, float *, void *, size_t, cudaStream_t);
} entry;
enum { ENTRIES = 11 };
static PyObject *type_of;     /* Python: torch dtype -> fgemm_dtype value or -1 */
static PyObject *raw_stream;  /* torch's (device index) -> current stream's handle */
static PyObject *current_device;  /* torch's () -> current device's index */
static int one_device;            /* torch sees one device: its tensors are on the current one, number 0 */
static PyObject *s_is_cuda, *s_dtype, *s_device, *s_data_ptr, *s_get_device, *s_cuda_stream;
/* Types met so far (borrowed for good: torch's dtypes live as long as the process). */
static PyObject *known_type[8];
static long known_value[8];
static int known;

enum { TYPE_I32 = 3 };  /* type_of's value for 32-bit integers, behind those of fgemm_dtype */

static long element_type(PyObject *dtype)
{
    for (int i = 0; i < known; ++i)
        if (known_type[i] == dtype) return known_value[i];
    PyObject *v = PyObject_CallOneArg(type_of, dtype);
    if (!v) return -2;
    const long t = PyLong_AsLong(v);
    Py_DECREF(v);
    if (known < 8 && !PyErr_Occurred()) {
        Py_INCREF(dtype);
        known_type[known] = dtype;
        known_value[known++] = t;
    }
    return t;
}

/* The address of a tensor or number; type: the element type it must have (-1: any).  device: that of
 * the call's tensors, -1 before the first one. */
static int address(PyObject *x, long type, long *device, void **out)
{
    if (x == Py_None) {
        *out = NULL;
        return 1;
    }
    if (PyLong_Check(x)) {
        *out = PyLong_AsVoidPtr(x);
        return *out != NULL || !PyErr_Occurred();
    }
    PyObject *where = one_device ? PyObject_GetAttr(x, s_is_cuda) : PyObject_CallMethodNoArgs(x, s_get_device);
    if (!where) {
        if (PyErr_ExceptionMatches(PyExc_AttributeError))
            PyErr_Format(PyExc_TypeError, "expected a CUDA tensor or a device address, got %R", (PyObject *)Py_TYPE(x));
        return 0;
    }
    const long on = one_device ? (where == Py_True) - 1 : PyLong_AsLong(where);  /* -1: on the host */
    Py_DECREF(where);
    if (on == -1 && PyErr_Occurred()) return 0;
    const int ok = on >= 0;
    if (type >= 0 || !ok) {
        PyObject *dtype = PyObject_GetAttr(x, s_dtype);
        if (!dtype) return 0;
        const long t = type >= 0 ? element_type(dtype) : 0;
        if (t == -2) {
            Py_DECREF(dtype);
            return 0;
        }
        if (!ok || (type >= 0 && t != type)) {
            PyObject *device = PyObject_GetAttr(x, s_device);
            if (device) {
                if (type >= 0)
                    PyErr_Format(PyExc_TypeError, "fgemm type %ld takes a CUDA tensor of that type (got %S on %S)", type, dtype,
                                 device);
                else
                    PyErr_Format(PyExc_TypeError, "expected a CUDA tensor (got %S on %S)", dtype, device);
                Py_DECREF(device);
            }
            Py_DECREF(dtype);
            return 0;
        }
        Py_DECREF(dtype);
    }
    if (*device < 0) {
        *device = on;
    } else if (*device != on) {
        PyErr_Format(PyExc_ValueError, "tensors on several devices (cuda:%ld and cuda:%ld)", *device, on);
        return 0;
    }
    PyObject *ptr = PyObject_CallMethodNoArgs(x, s_data_ptr);
    if (!ptr) return 0;
    *out = PyLong_AsVoidPtr(ptr);
    Py_DECREF(ptr);
    return *out != NULL || !PyErr_Occurred();
}

/* The stream a call runs on: the one given (a handle or an object with cuda_stream), else the
 * current one of its tensors' device, else the default stream.  device: that of the call's tensors (-1:
 * there are none), which has to be the current one. */
static int stream_of(PyObject *s, long device, cudaStream_t *out)
{
    PyObject *v;
    if (device >= 0 && !one_device) {
        v = PyObject_CallNoArgs(current_device);
        if (!v) return 0;
        const long current = PyLong_AsLong(v);
        Py_DECREF(v);
        if (current == -1 && PyErr_Occurred()) return 0;
        if (current != device) {
            PyErr_Format(PyExc_ValueError, "tensors on cuda:%ld, but the current device is cuda:%ld", device, current);
            return 0;
        }
    }
    if (s != Py_None) {
        if (PyLong_Check(s)) {
            Py_INCREF(s);
            v = s;
        } else {
            v = PyObject_GetAttr(s, s_cuda_stream);
        }
    } else if (device < 0) {
        *out = NULL;
        return 1;
    } else {
        PyObject *d = PyLong_FromLong(device);
        if (!d) return 0;
        v = PyObject_CallOneArg(raw_stream, d);
        Py_DECREF(d);
    }
    if (!v) return 0;
    *out = (cudaStream_t)PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return !PyErr_Occurred();
}

static int integer(PyObject *x, int *out)
{
    const long v = PyLong_AsLong(x);
    if (v == -1 && PyErr_Occurred()) return 0;
    if (v < INT_MIN || v > INT_MAX) {
        PyErr_Format(PyExc_OverflowError, "%ld does not fit a C int", v);
        return 0;
    }
    *out = (int)v;
    return 1;
}

static int wide(PyObject *x, long long *out)
{
    *out = PyLong_AsLongLong(x);
    return *out != -1 || !PyErr_Occurred();
}

static int number(PyObject *x, float *out)
{
    const double v = PyFloat_AsDouble(x);
    *out = (float)v;
    return v != -1.0 || !PyErr_Occurred();
}

static int bytes(PyObject *x, size_t *out)
{
    *out = PyLong_AsSize_t(x);
    return *out != (size_t)-1 || !PyErr_Occurred();
}

static int count(const char *name, Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return 1;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", name, want, n);
    return 0;
}

/* The call itself runs without the interpreter's lock: a launch may wait for room in a stream. */
#define RETURN_CALL(call)                \
    do {                                 \
        fgemm_status st;                 \
        Py_BEGIN_ALLOW_THREADS st = call; \
        Py_END_ALLOW_THREADS             \
        return PyLong_FromLong(st);      \
    } while (0)

#define INT(i, v) integer(a[i], &v)
#define MATRIX(i, v) address(a[i], type, &device, (void **)&v)
#define RAW(i, v) address(a[i], -1, &device, (void **)&v)
#define FLOATS(i, v) address(a[i], FGEMM_F32, &device, (void **)&v)
#define OUT(i, v) address(a[i], out_type, &device, (void **)&v)
#define INTS(i, v) address(a[i], TYPE_I32, &device, (void **)&v)

/* (type, M, N, X, ldx, row_codes, ld, row_scales, col_codes, ld, col_scales, stream) */
static PyObject *quantize(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int type, M, N, ldx, ldr, ldc;
    void *x, *rc, *rs, *cc, *cs;
    cudaStream_t stream;
    long device = -1;
    if (!count("mxfp4_quantize", n, 12) || !INT(0, type) || !INT(1, M) || !INT(2, N) || !MATRIX(3, x) || !INT(4, ldx) ||
        !RAW(5, rc) || !INT(6, ldr) || !RAW(7, rs) || !RAW(8, cc) || !INT(9, ldc) || !RAW(10, cs) ||
        !stream_of(a[11], device, &stream))
        return NULL;
    RETURN_CALL(entry.quantize((fgemm_dtype)type, M, N, x, ldx, rc, ldr, rs, cc, ldc, cs, stream));
}

/* (type, M, N, G, ldg, Y, ldy, row_codes, ld, row_scales, col_codes, ld, col_scales, bias_grad, workspace, bytes, stream) */
static PyObject *quantize_grad(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int type, M, N, ldg, ldy, ldr, ldc;
    void *g, *y, *rc, *rs, *cc, *cs, *ws;
    float *bias;
    size_t size;
    cudaStream_t stream;
    long device = -1;
    if (!count("mxfp4_quantize_grad", n, 17) || !INT(0, type) || !INT(1, M) || !INT(2, N) || !MATRIX(3, g) || !INT(4, ldg) ||
        !MATRIX(5, y) || !INT(6, ldy) || !RAW(7, rc) || !INT(8, ldr) || !RAW(9, rs) || !RAW(10, cc) || !INT(11, ldc) ||
        !RAW(12, cs) || !FLOATS(13, bias) || !RAW(14, ws) || !bytes(a[15], &size) ||
        !stream_of(a[16], device, &stream))
        return NULL;
    RETURN_CALL(entry.quantize_grad((fgemm_dtype)type, M, N, g, ldg, y, ldy, rc, ldr, rs, cc, ldc, cs, bias, ws, size, stream));
}

/* (type, M, N, codes, ld, scales, X, ldx, stream) */
static PyObject *dequantize(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int type, M, N, ld, ldx;
    void *codes, *scales, *x;
    cudaStream_t stream;
    long device = -1;
    if (!count("mxfp4_dequantize", n, 9) || !INT(0, type) || !INT(1, M) || !INT(2, N) || !RAW(3, codes) || !INT(4, ld) ||
        !RAW(5, scales) || !MATRIX(6, x) || !INT(7, ldx) || !stream_of(a[8], device, &stream))
        return NULL;
    RETURN_CALL(entry.dequantize((fgemm_dtype)type, M, N, codes, ld, scales, x, ldx, stream));
}

/* (type, M, N, K, alpha, A_codes, ld, A_scales, B_codes, ld, B_scales, beta, C, ldc, bias, relu, stream) */
static PyObject *gemm(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int type, M, N, K, lda, ldb, ldc, relu;
    float alpha, beta;
    void *ac, *as, *bc, *bs, *c;
    float *bias;
    cudaStream_t stream;
    long device = -1;
    if (!count("mxfp4_gemm", n, 17) || !INT(0, type) || !INT(1, M) || !INT(2, N) || !INT(3, K) || !number(a[4], &alpha) ||
        !RAW(5, ac) || !INT(6, lda) || !RAW(7, as) || !RAW(8, bc) || !INT(9, ldb) || !RAW(10, bs) || !number(a[11], &beta) ||
        !MATRIX(12, c) || !INT(13, ldc) || !FLOATS(14, bias) || (relu = PyObject_IsTrue(a[15])) < 0 ||
        !stream_of(a[16], device, &stream))
        return NULL;
    RETURN_CALL(entry.gemm((fgemm_dtype)type, M, N, K, alpha, ac, lda, as, bc, ldb, bs, beta, c, ldc, bias, relu, stream));
}

/* (type, M, N, K, X, ldx, W_codes, ld, W_scales, bias, relu, Y, ldy, workspace, bytes, stream) */
static PyObject *linear(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int type, M, N, K, ldx, ldw, ldy, relu;
    void *x, *wc, *ws, *y, *space;
    float *bias;
    size_t size;
    cudaStream_t stream;
    long device = -1;
    if (!count("mxfp4_linear", n, 16) || !INT(0, type) || !INT(1, M) || !INT(2, N) || !INT(3, K) || !MATRIX(4, x) ||
        !INT(5, ldx) || !RAW(6, wc) || !INT(7, ldw) || !RAW(8, ws) || !FLOATS(9, bias) ||
        (relu = PyObject_IsTrue(a[10])) < 0 || !MATRIX(11, y) || !INT(12, ldy) || !RAW(13, space) || !bytes(a[14], &size) ||
        !stream_of(a[15], device, &stream))
        return NULL;
    RETURN_CALL(entry.linear((fgemm_dtype)type, M, N, K, x, ldx, wc, ldw, ws, bias, relu, y, ldy, space, size, stream));
}

/* (type, out_type, transa, transb, M, N, K, alpha, A, lda, B, ldb, bias, act, Z, ldz, beta, R, ldr, Y, ldy, workspace, bytes, stream) */
static PyObject *gemm16(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int type, out_type, ta, tb, M, N, K, lda, ldb, act, ldz, ldr, ldy;
    float alpha, beta;
    void *A, *B, *Z, *R, *Y, *ws;
    float *bias;
    size_t size;
    cudaStream_t stream;
    long device = -1;
    if (!count("gemm16", n, 24) || !INT(0, type) || !INT(1, out_type) || !INT(2, ta) || !INT(3, tb) || !INT(4, M) || !INT(5, N) ||
        !INT(6, K) || !number(a[7], &alpha) || !MATRIX(8, A) || !INT(9, lda) || !MATRIX(10, B) || !INT(11, ldb) ||
        !FLOATS(12, bias) || !INT(13, act) || !MATRIX(14, Z) || !INT(15, ldz) || !number(a[16], &beta) || !OUT(17, R) ||
        !INT(18, ldr) || !OUT(19, Y) || !INT(20, ldy) || !RAW(21, ws) || !bytes(a[22], &size) || !stream_of(a[23], device, &stream))
        return NULL;
    RETURN_CALL(entry.gemm16((fgemm_dtype)type, (fgemm_dtype)out_type, (fgemm_op)ta, (fgemm_op)tb, M, N, K, alpha, A, lda, B, ldb,
                             bias, (fgemm_activation)act, Z, ldz, beta, R, ldr, Y, ldy, ws, size, stream));
}

/* (type, out_type, transa, transb, M, N, K, alpha, A, lda, B, ldb, act, Z, ldz, Y, ldy, col_sums, workspace, bytes, stream) */
static PyObject *gemm16_grad(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int type, out_type, ta, tb, M, N, K, lda, ldb, act, ldz, ldy;
    float alpha;
    void *A, *B, *Z, *Y, *ws;
    float *sums;
    size_t size;
    cudaStream_t stream;
    long device = -1;
    if (!count("gemm16_grad", n, 21) || !INT(0, type) || !INT(1, out_type) || !INT(2, ta) || !INT(3, tb) || !INT(4, M) ||
        !INT(5, N) || !INT(6, K) || !number(a[7], &alpha) || !MATRIX(8, A) || !INT(9, lda) || !MATRIX(10, B) || !INT(11, ldb) ||
        !INT(12, act) || !MATRIX(13, Z) || !INT(14, ldz) || !OUT(15, Y) || !INT(16, ldy) || !FLOATS(17, sums) || !RAW(18, ws) ||
        !bytes(a[19], &size) || !stream_of(a[20], device, &stream))
        return NULL;
    RETURN_CALL(entry.gemm16_grad((fgemm_dtype)type, (fgemm_dtype)out_type, (fgemm_op)ta, (fgemm_op)tb, M, N, K, alpha, A, lda, B,
                                  ldb, (fgemm_activation)act, Z, ldz, Y, ldy, sums, ws, size, stream));
}

/* (type, out_type, transb, groups, M, N, K, offsets, alpha, A, lda, B, ldb, strideB, bias, act, Z, ldz, beta, R, ldr, Y, ldy, workspace,
 * bytes, stream) */
static PyObject *gemm16_grouped(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int type, out_type, tb, groups, M, N, K, lda, ldb, act, ldz, ldr, ldy;
    float alpha, beta;
    void *A, *B, *Z, *R, *Y, *ws;
    int *offsets;
    long long strideB;
    float *bias;
    size_t size;
    cudaStream_t stream;
    long device = -1;
    if (!count("gemm16_grouped", n, 26) || !INT(0, type) || !INT(1, out_type) || !INT(2, tb) || !INT(3, groups) || !INT(4, M) ||
        !INT(5, N) || !INT(6, K) || !INTS(7, offsets) || !number(a[8], &alpha) || !MATRIX(9, A) || !INT(10, lda) ||
        !MATRIX(11, B) || !INT(12, ldb) || !wide(a[13], &strideB) || !FLOATS(14, bias) || !INT(15, act) || !MATRIX(16, Z) ||
        !INT(17, ldz) || !number(a[18], &beta) || !OUT(19, R) || !INT(20, ldr) || !OUT(21, Y) || !INT(22, ldy) || !RAW(23, ws) ||
        !bytes(a[24], &size) || !stream_of(a[25], device, &stream))
        return NULL;
    RETURN_CALL(entry.gemm16_grouped((fgemm_dtype)type, (fgemm_dtype)out_type, (fgemm_op)tb, groups, M, N, K, offsets, alpha, A, lda,
                                     B, ldb, strideB, bias, (fgemm_activation)act, Z, ldz, beta, R, ldr, Y, ldy, ws, size, stream));
}

/* (type, out_type, transb, groups, M, N, K, offsets, alpha, A, lda, B, ldb, strideB, act, Z, ldz, Y, ldy, col_sums, workspace, bytes,
 * stream) */
static PyObject *gemm16_grouped_grad(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int type, out_type, tb, groups, M, N, K, lda, ldb, act, ldz, ldy;
    float alpha;
    void *A, *B, *Z, *Y, *ws;
    int *offsets;
    long long strideB;
    float *sums;
    size_t size;
    cudaStream_t stream;
    long device = -1;
    if (!count("gemm16_grouped_grad", n, 23) || !INT(0, type) || !INT(1, out_type) || !INT(2, tb) || !INT(3, groups) || !INT(4, M) ||
        !INT(5, N) || !INT(6, K) || !INTS(7, offsets) || !number(a[8], &alpha) || !MATRIX(9, A) || !INT(10, lda) ||
        !MATRIX(11, B) || !INT(12, ldb) || !wide(a[13], &strideB) || !INT(14, act) || !MATRIX(15, Z) || !INT(16, ldz) ||
        !OUT(17, Y) || !INT(18, ldy) || !FLOATS(19, sums) || !RAW(20, ws) || !bytes(a[21], &size) ||
        !stream_of(a[22], device, &stream))
        return NULL;
    RETURN_CALL(entry.gemm16_grouped_grad((fgemm_dtype)type, (fgemm_dtype)out_type, (fgemm_op)tb, groups, M, N, K, offsets, alpha, A,
                                          lda, B, ldb, strideB, (fgemm_activation)act, Z, ldz, Y, ldy, sums, ws, size, stream));
}

/* (type, out_type, groups, M, N, K, offsets, alpha, A, lda, G, ldg, beta, C, ldc, strideC, workspace, bytes, stream) */
static PyObject *gemm16_weight_grad(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int type, out_type, groups, M, N, K, lda, ldg, ldc;
    float alpha, beta;
    void *A, *G, *C, *ws;
    int *offsets;
    long long strideC;
    size_t size;
    cudaStream_t stream;
    long device = -1;
    if (!count("gemm16_weight_grad", n, 19) || !INT(0, type) || !INT(1, out_type) || !INT(2, groups) || !INT(3, M) || !INT(4, N) ||
        !INT(5, K) || !INTS(6, offsets) || !number(a[7], &alpha) || !MATRIX(8, A) || !INT(9, lda) || !MATRIX(10, G) ||
        !INT(11, ldg) || !number(a[12], &beta) || !OUT(13, C) || !INT(14, ldc) || !wide(a[15], &strideC) || !RAW(16, ws) ||
        !bytes(a[17], &size) || !stream_of(a[18], device, &stream))
        return NULL;
    RETURN_CALL(entry.gemm16_weight_grad((fgemm_dtype)type, (fgemm_dtype)out_type, groups, M, N, K, offsets, alpha, A, lda, G, ldg,
                                         beta, C, ldc, strideC, ws, size, stream));
}

/* (type, groups, M, N, offsets, act, G, ldg, Z, ldz, D, ldd, col_sums, workspace, bytes, stream) */
static PyObject *act16_grad(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int type, groups, M, N, act, ldg, ldz, ldd;
    void *G, *Z, *D, *ws;
    int *offsets;
    float *sums;
    size_t size;
    cudaStream_t stream;
    long device = -1;
    if (!count("act16_grad", n, 16) || !INT(0, type) || !INT(1, groups) || !INT(2, M) || !INT(3, N) || !INTS(4, offsets) ||
        !INT(5, act) || !MATRIX(6, G) || !INT(7, ldg) || !MATRIX(8, Z) || !INT(9, ldz) || !MATRIX(10, D) || !INT(11, ldd) ||
        !FLOATS(12, sums) || !RAW(13, ws) || !bytes(a[14], &size) || !stream_of(a[15], device, &stream))
        return NULL;
    RETURN_CALL(entry.act16_grad((fgemm_dtype)type, groups, M, N, offsets, (fgemm_activation)act, G, ldg, Z, ldz, D, ldd, sums, ws,
                                 size, stream));
}

/* (type_of, raw_stream, current_device, one_device, the entries' addresses in their order above) */
static PyObject *bind(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *p[ENTRIES];
    long device = -1;
    if (!count("bind", n, 4 + ENTRIES)) return NULL;
    for (int i = 0; i < ENTRIES; ++i)
        if (!address(a[4 + i], -1, &device, &p[i])) return NULL;
    const int one = PyObject_IsTrue(a[3]);
    if (one < 0) return NULL;
    one_device = one;
    for (int i = 0; i < 3; ++i) Py_INCREF(a[i]);
    Py_XSETREF(type_of, a[0]);
    Py_XSETREF(raw_stream, a[1]);
    Py_XSETREF(current_device, a[2]);
    *(void **)&entry.quantize = p[0];
    *(void **)&entry.quantize_grad = p[1];
    *(void **)&entry.dequantize = p[2];
    *(void **)&entry.gemm = p[3];
    *(void **)&entry.linear = p[4];
    *(void **)&entry.gemm16 = p[5];
    *(void **)&entry.gemm16_grad = p[6];
    *(void **)&entry.gemm16_grouped = p[7];
    *(void **)&entry.gemm16_grouped_grad = p[8];
    *(void **)&entry.gemm16_weight_grad = p[9];
    *(void **)&entry.act16_grad = p[10];
    Py_RETURN_NONE;
}

#define METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(bind), METHOD(quantize), METHOD(quantize_grad), METHOD(dequantize),
                                METHOD(gemm), METHOD(linear), METHOD(gemm16), METHOD(gemm16_grad), METHOD(gemm16_grouped),
                                METHOD(gemm16_grouped_grad), METHOD(gemm16_weight_grad), METHOD(act16_grad),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "MXFP4 and 16-bit calls of libfgemm", -1, methods};

PyMODINIT_FUNC PyInit__calls(void)
{
    s_is_cuda = PyUnicode_InternFromString("is_cuda");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_device = PyUnicode_InternFromString("device");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!s_is_cuda || !s_dtype || !s_device || !s_data_ptr || !s_get_device || !s_cuda_stream) return NULL;
    return PyModule_Create(&module);
}
