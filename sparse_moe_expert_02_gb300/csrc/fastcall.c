/* The small operators' way from Python to libmoe: argument checks and the call
 * in one C function each (module _fastcall).
 *
 * These operators run a few microseconds, and a decode step calls them one
 * after another, so the caller's time counts: reading the tensors and calling
 * through ctypes took 10.7 us for a post-norm with everything (a launch itself
 * is 2 us), here 5.3 us (quantise 5.6 to 3.3, 4-bit product 9.5 to 5.4).
 * Nothing is kept from one call to the next.  The call itself runs without the
 * interpreter lock, as through ctypes: a launch waits while the stream's queue
 * is full, for as long as what is queued takes, and a host function queued
 * there may need the lock.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "moe.h"

static PyObject *s_dtype, *s_is_cuda, *s_shape, *s_stride, *s_data_ptr, *s_is_contiguous, *s_get_device;
static PyObject *t_f32, *t_bf16, *t_u8, *t_i32, *f_device, *f_stream;

static moe_status (*p_norm_pre)(const moe_norm*, const void*, int32_t, int64_t, int32_t, int32_t, void*, int32_t, int64_t, void*);
static moe_status (*p_norm_post)(const moe_post*, const void*, int32_t, int64_t, const void*, int32_t, int64_t, int32_t, int32_t, void*,
                                 int64_t, void*, int32_t, int64_t, void*);
static moe_status (*p_quantize)(const void*, int32_t, int64_t, int64_t, int32_t, uint8_t*, uint8_t*, void*);
static moe_status (*p_dequantize)(const uint8_t*, const uint8_t*, int64_t, int32_t, void*, int32_t, int64_t, void*);
static moe_status (*p_gemm)(const uint8_t*, const uint8_t*, const uint8_t*, const uint8_t*, const int32_t*, int32_t, int32_t, int32_t,
                            int32_t, void*, int32_t, int64_t, uint32_t*, void*);
/* the experts' products: the product and its gradient by the rows (one signature), its gradient by the weights, and so on */
static moe_status (*p_grouped[2])(const void*, int64_t, const void*, int32_t, const int32_t*, int32_t, int32_t, int32_t, int32_t, void*,
                                  int32_t, int64_t, uint32_t*, void*);
static moe_status (*p_dw)(const void*, int64_t, const void*, int64_t, int32_t, const int32_t*, int32_t, int32_t, int32_t, int32_t, void*,
                          int32_t, int32_t, uint32_t*, void*);
static moe_status (*p_swiglu)(const void*, int64_t, const void*, int64_t, int32_t, const float*, int32_t, int32_t, void*, int32_t, int64_t,
                              void*);
static moe_status (*p_swiglu_grad)(const void*, int64_t, const void*, int64_t, const void*, int64_t, int32_t, const float*, int32_t,
                                   int32_t, void*, int64_t, void*, int64_t, float*, void*);
static moe_status (*p_int4_quantize)(const void*, int32_t, int64_t, int64_t, int32_t, int32_t, uint8_t*, void*, int32_t, uint8_t*, void*);
static moe_status (*p_int4_dequantize)(const uint8_t*, const void*, int32_t, const uint8_t*, int32_t, int64_t, int32_t, void*, int32_t,
                                       int64_t, void*);
static moe_status (*p_int4_gemm)(const void*, int32_t, int64_t, const uint8_t*, const void*, int32_t, const uint8_t*, int32_t,
                                 const int32_t*, int32_t, int32_t, int32_t, int32_t, void*, int32_t, int64_t, uint32_t*, void*);

/* A tensor's address, sizes and, if asked for, strides. */
typedef struct {
    void* p;
    int dtype; /* moe_dtype; -1: not fp32 or bf16 */
    PyObject* type;
    int dims;
    int64_t size[8], stride[8];
} Tensor;

static int fail(const char* what, const char* why) {
    PyErr_Format(PyExc_ValueError, "%s: %s", what, why);
    return -1;
}

static int numbers(PyObject* tuple, int64_t* out, int dims) {
    if (!tuple) return -1;
    int ok = PyTuple_Check(tuple) && (dims < 0 ? PyTuple_GET_SIZE(tuple) <= 8 : PyTuple_GET_SIZE(tuple) == dims);
    if (ok) {
        dims = (int)PyTuple_GET_SIZE(tuple);
        for (int i = 0; i < dims; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    }
    Py_DECREF(tuple);
    if (!ok) {
        PyErr_SetString(PyExc_ValueError, "tensors of at most eight dimensions");
        return -1;
    }
    return PyErr_Occurred() ? -1 : dims;
}

static int read_tensor(PyObject* t, const char* what, Tensor* r, int strides) {
    PyObject* o = PyObject_GetAttr(t, s_is_cuda);
    if (!o) return -1;
    const int cuda = o == Py_True;
    Py_DECREF(o);
    if (!cuda) return fail(what, "libmoe takes device tensors");
    o = PyObject_GetAttr(t, s_dtype);
    if (!o) return -1;
    r->type = o; /* the type objects live for good */
    r->dtype = o == t_f32 ? MOE_F32 : o == t_bf16 ? MOE_BF16 : -1;
    Py_DECREF(o);
    if ((r->dims = numbers(PyObject_GetAttr(t, s_shape), r->size, -1)) < 0) return -1;
    if (strides && numbers(PyObject_CallMethodNoArgs(t, s_stride), r->stride, r->dims) < 0) return -1;
    if (!strides) {
        o = PyObject_CallMethodNoArgs(t, s_is_contiguous);
        if (!o) return -1;
        const int whole = o == Py_True;
        Py_DECREF(o);
        if (!whole) return fail(what, "libmoe takes contiguous tensors");
    }
    o = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!o) return -1;
    r->p = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    return PyErr_Occurred() ? -1 : 0;
}

/* [T, D] of fp32 or bf16 with contiguous rows; the row stride in stride[0]. */
static int read_rows(PyObject* t, const char* what, Tensor* r, const Tensor* like) {
    if (read_tensor(t, what, r, 1) < 0) return -1;
    if (r->dtype < 0) return fail(what, "fp32 or bf16");
    if (r->dims != 2 || (r->stride[1] != 1 && r->size[1] > 1)) return fail(what, "a 2-D tensor whose rows are contiguous");
    if (r->size[0] <= 1) r->stride[0] = r->size[1]; /* the stride of a single row says nothing */
    if (like && (r->size[0] != like->size[0] || r->size[1] != like->size[1])) {
        PyErr_Format(PyExc_ValueError, "%s: shape (%lld, %lld), not (%lld, %lld)", what, (long long)like->size[0], (long long)like->size[1],
                     (long long)r->size[0], (long long)r->size[1]);
        return -1;
    }
    if (r->size[0] > INT32_MAX || r->size[1] > INT32_MAX) return fail(what, "at most 2^31 - 1 rows and columns");
    return 0;
}

/* A contiguous vector of n fp32 or bf16. */
static int read_vector(PyObject* t, int64_t n, const char* what, Tensor* r) {
    if (read_tensor(t, what, r, 0) < 0) return -1;
    if (r->dtype < 0 || r->dims != 1 || r->size[0] != n) {
        PyErr_Format(PyExc_ValueError, "%s: a contiguous device tensor [%lld] of fp32 or bf16", what, (long long)n);
        return -1;
    }
    return 0;
}

static int read_norm(moe_norm* m, PyObject* kind, PyObject* eps, PyObject* off, PyObject* w, PyObject* b, int64_t D) {
    Tensor t;
    m->kind = (int32_t)PyLong_AsLong(kind);
    m->eps = (float)PyFloat_AsDouble(eps);
    m->w_offset = (float)PyFloat_AsDouble(off);
    m->p_dtype = MOE_F32;
    m->w = m->b = NULL;
    if (PyErr_Occurred()) return -1;
    if (w != Py_None) {
        if (read_vector(w, D, "norm parameters", &t) < 0) return -1;
        m->w = t.p;
        m->p_dtype = t.dtype;
    }
    if (b != Py_None) {
        if (read_vector(b, D, "norm parameters", &t) < 0) return -1;
        if (m->w && t.dtype != m->p_dtype) return fail("norm parameters", "w and b of one type");
        m->b = t.p;
        m->p_dtype = t.dtype;
    }
    return 0;
}

/* The current torch stream of the current device. */
static int read_stream(void** s) {
    PyObject* d = PyObject_CallNoArgs(f_device);
    if (!d) return -1;
    PyObject* o = PyObject_CallOneArg(f_stream, d);
    Py_DECREF(d);
    if (!o) return -1;
    *s = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    return PyErr_Occurred() ? -1 : 0;
}

static int count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return 0;
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
    return -1;
}

#define CALL(call)                  \
    do {                            \
        moe_status st;              \
        Py_BEGIN_ALLOW_THREADS      \
        st = call;                  \
        Py_END_ALLOW_THREADS        \
        return PyLong_FromLong(st); \
    } while (0)

/* x, w, b, kind, eps, w_offset, out */
static PyObject* norm_pre(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor x, out;
    moe_norm m;
    void* s;
    if (count(n, 7) < 0 || read_rows(a[0], "x", &x, NULL) < 0 || read_rows(a[6], "out", &out, &x) < 0 ||
        read_norm(&m, a[3], a[4], a[5], a[1], a[2], x.size[1]) < 0 || read_stream(&s) < 0)
        return NULL;
    CALL(p_norm_pre(&m, x.p, x.dtype, x.stride[0], (int32_t)x.size[0], (int32_t)x.size[1], out.p, out.dtype, out.stride[0], s));
}

/* y, res, out, next_out | kind, eps, w_offset, w, b | next_kind, next_w, next_b | res_scale, branch_scale |
 * gate_by, gate, gate_sigmoid */
static PyObject* norm_post(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor y, res, out, next = {0}, g;
    moe_post p = {0};
    void* s;
    if (count(n, 17) < 0 || read_rows(a[0], "y", &y, NULL) < 0 || read_rows(a[1], "res", &res, &y) < 0 ||
        read_rows(a[2], "out", &out, &y) < 0)
        return NULL;
    if (out.dtype != res.dtype) {
        fail("out", "the type of res");
        return NULL;
    }
    next.dtype = MOE_BF16;
    if (a[3] != Py_None && read_rows(a[3], "next_out", &next, &y) < 0) return NULL;
    const int64_t T = y.size[0], D = y.size[1];
    if (read_norm(&p.norm, a[4], a[5], a[6], a[7], a[8], D) < 0) return NULL;
    if (a[3] != Py_None && read_norm(&p.next, a[9], a[5], a[6], a[10], a[11], D) < 0) return NULL;
    p.res_scale = (float)PyFloat_AsDouble(a[12]);
    p.branch_scale = (float)PyFloat_AsDouble(a[13]);
    p.gate_by = (int32_t)PyLong_AsLong(a[14]);
    p.gate_sigmoid = PyObject_IsTrue(a[16]);
    if (PyErr_Occurred()) return NULL;
    if (p.gate_by == MOE_GATE_FULL) {
        if (read_rows(a[15], "gate", &g, &y) < 0) return NULL;
        p.ld_gate = g.stride[0];
    } else if (p.gate_by != MOE_GATE_NONE && read_vector(a[15], p.gate_by == MOE_GATE_CHANNEL ? D : T, "gate", &g) < 0) {
        return NULL;
    }
    if (p.gate_by != MOE_GATE_NONE) {
        p.gate = g.p;
        p.gate_dtype = g.dtype;
    }
    if (read_stream(&s) < 0) return NULL;
    CALL(p_norm_post(&p, y.p, y.dtype, y.stride[0], res.p, res.dtype, res.stride[0], (int32_t)T, (int32_t)D, out.p,
                     out.stride[0], next.p, next.dtype, next.stride[0], s));
}

/* Codes and scales that hold `cols` columns; *rows: of all leading dimensions. */
static int read_mx(PyObject* codes, PyObject* scales, PyObject* columns, const char* what, Tensor* q, Tensor* s, int64_t* rows, int64_t* cols) {
    if (read_tensor(codes, what, q, 0) < 0 || read_tensor(scales, what, s, 0) < 0) return -1;
    *cols = PyLong_AsLongLong(columns);
    if (PyErr_Occurred()) return -1;
    const int64_t nb = (*cols + 31) / 32;
    int ok = q->type == t_u8 && s->type == t_u8 && q->dims == s->dims && q->dims >= 1 && q->size[q->dims - 1] == 16 * nb &&
             s->size[s->dims - 1] == nb;
    *rows = 1;
    for (int i = 0; ok && i < q->dims - 1; ++i) {
        ok = q->size[i] == s->size[i];
        *rows *= q->size[i];
    }
    return ok ? 0 : fail(what, "uint8 codes and scales of its columns");
}

static int held(const Tensor* x, int64_t rows, int64_t cols, const char* what) {
    if (x->size[0] == rows && x->size[1] == cols) return 0;
    PyErr_Format(PyExc_ValueError, "%s holds (%lld, %lld), not (%lld, %lld)", what, (long long)rows, (long long)cols, (long long)x->size[0],
                 (long long)x->size[1]);
    return -1;
}

/* x, codes, scales, cols */
static PyObject* mx_quantize(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor x, q, sc;
    int64_t rows, cols;
    void* s;
    if (count(n, 4) < 0 || read_rows(a[0], "x", &x, NULL) < 0 || read_mx(a[1], a[2], a[3], "out", &q, &sc, &rows, &cols) < 0 ||
        held(&x, rows, cols, "out") < 0 || read_stream(&s) < 0)
        return NULL;
    CALL(p_quantize(x.p, x.dtype, x.stride[0], rows, (int32_t)cols, (uint8_t*)q.p, (uint8_t*)sc.p, s));
}

/* codes, scales, cols, out */
static PyObject* mx_dequantize(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor q, sc, out;
    int64_t rows, cols;
    void* s;
    if (count(n, 4) < 0 || read_mx(a[0], a[1], a[2], "q", &q, &sc, &rows, &cols) < 0 || read_rows(a[3], "out", &out, NULL) < 0 ||
        held(&out, rows, cols, "q") < 0 || read_stream(&s) < 0)
        return NULL;
    CALL(p_dequantize((const uint8_t*)q.p, (const uint8_t*)sc.p, rows, (int32_t)cols, out.p, out.dtype, out.stride[0], s));
}

/* a codes, scales, cols | b codes, scales, cols | offsets, out, err */
static PyObject* mx_gemm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor qa, sa, qb, sb, off, out, err;
    int64_t rows, K, all, Kb;
    void* s;
    if (count(n, 9) < 0 || read_mx(a[0], a[1], a[2], "a", &qa, &sa, &rows, &K) < 0 || read_mx(a[3], a[4], a[5], "b", &qb, &sb, &all, &Kb) < 0)
        return NULL;
    if (qa.dims != 2 || qb.dims < 2 || qb.dims > 3 || K != Kb) {
        fail("matmul", "a [rows, K] and b [N, K] or [G, N, K]");
        return NULL;
    }
    if (K % 32) {
        fail("matmul", "K must be a multiple of 32");
        return NULL;
    }
    const int64_t G = qb.dims == 3 ? qb.size[0] : 1, N = qb.size[qb.dims - 2];
    off.p = err.p = NULL;
    if (a[6] != Py_None) {
        if (read_tensor(a[6], "offsets", &off, 0) < 0) return NULL;
        int64_t m = 1;
        for (int i = 0; i < off.dims; ++i) m *= off.size[i];
        if (off.type != t_i32 || m != G + 1) {
            fail("matmul", "offsets are int32 [G+1]");
            return NULL;
        }
    }
    if (a[8] != Py_None) {
        if (read_tensor(a[8], "err", &err, 0) < 0) return NULL;
        int64_t m = 1;
        for (int i = 0; i < err.dims; ++i) m *= err.size[i];
        if (err.type != t_i32 || m < 4) { /* the kernel writes four words */
            fail("err", "int32 [4]");
            return NULL;
        }
    }
    if (read_rows(a[7], "out", &out, NULL) < 0) return NULL;
    if (out.size[0] != rows || out.size[1] != N) {
        PyErr_Format(PyExc_ValueError, "out: shape (%lld, %lld), not (%lld, %lld)", (long long)rows, (long long)N, (long long)out.size[0],
                     (long long)out.size[1]);
        return NULL;
    }
    if (G > INT32_MAX || K > INT32_MAX) {
        fail("matmul", "G and K below 2^31");
        return NULL;
    }
    if (read_stream(&s) < 0) return NULL;
    CALL(p_gemm((const uint8_t*)qa.p, (const uint8_t*)sa.p, (const uint8_t*)qb.p, (const uint8_t*)sb.p, (const int32_t*)off.p,
                (int32_t)rows, (int32_t)G, (int32_t)N, (int32_t)K, out.p, out.dtype, out.stride[0], (uint32_t*)err.p, s));
}

/* ------------------------------------------------ the experts' products */

/* The stream as read_stream, and every one of the n tensors (or None) on the current device: a kernel would be launched there. */
static int read_stream_of(PyObject* const* t, int n, void** s) {
    PyObject* d = PyObject_CallNoArgs(f_device);
    if (!d) return -1;
    for (int i = 0; i < n; ++i) {
        if (t[i] == Py_None) continue;
        PyObject* o = PyObject_CallMethodNoArgs(t[i], s_get_device);
        const int same = o ? PyObject_RichCompareBool(o, d, Py_EQ) : -1;
        Py_XDECREF(o);
        if (same <= 0) {
            Py_DECREF(d);
            if (same == 0) PyErr_SetString(PyExc_ValueError, "a tensor is not on the current device");
            return -1;
        }
    }
    PyObject* o = PyObject_CallOneArg(f_stream, d);
    Py_DECREF(d);
    if (!o) return -1;
    *s = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    return PyErr_Occurred() ? -1 : 0;
}

/* Offsets of G groups (or None with one group) and an error word (or None). */
static int read_groups(PyObject* offsets, PyObject* word, int64_t G, const int32_t** off, uint32_t** err) {
    Tensor t;
    *off = NULL;
    *err = NULL;
    if (offsets != Py_None) {
        if (read_tensor(offsets, "offsets", &t, 0) < 0) return -1;
        if (t.type != t_i32 || t.dims != 1 || t.size[0] != G + 1) return fail("offsets", "int32 [G+1]");
        *off = (const int32_t*)t.p;
    } else if (G != 1) {
        return fail("offsets", "needed for several groups");
    }
    if (word != Py_None) {
        if (read_tensor(word, "err", &t, 0) < 0) return -1;
        if (t.type != t_i32 || t.dims != 1 || t.size[0] < 4) return fail("err", "int32 [4]");
        *err = (uint32_t*)t.p;
    }
    return 0;
}

/* Contiguous [G, N, K] (or [N, K], one group). */
static int read_matrices(PyObject* t, const char* what, Tensor* r, int64_t* G, int64_t* N, int64_t* K) {
    if (read_tensor(t, what, r, 0) < 0) return -1;
    if (r->dims != 2 && r->dims != 3) return fail(what, "[N, K] or [G, N, K]");
    *G = r->dims == 3 ? r->size[0] : 1;
    *N = r->size[r->dims - 2];
    *K = r->size[r->dims - 1];
    if (*G > INT32_MAX || *N > INT32_MAX || *K > INT32_MAX) return fail(what, "sizes below 2^31");
    return 0;
}

static int columns(const Tensor* r, int64_t cols, const char* what) {
    if (r->size[1] == cols) return 0;
    PyErr_Format(PyExc_ValueError, "%s: %lld columns, not %lld", what, (long long)cols, (long long)r->size[1]);
    return -1;
}

/* direction (0 product, 1 gradient by the rows), rows, weights, offsets, out, err */
static PyObject* grouped(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor x, w, out;
    int64_t G, N, K;
    const int32_t* off;
    uint32_t* err;
    void* s;
    if (count(n, 6) < 0) return NULL;
    const long dir = PyLong_AsLong(a[0]);
    if (PyErr_Occurred() || read_rows(a[1], dir ? "dy" : "x", &x, NULL) < 0 || read_matrices(a[2], "w", &w, &G, &N, &K) < 0 ||
        read_rows(a[4], "out", &out, NULL) < 0 || columns(&x, dir ? N : K, dir ? "dy" : "x") < 0 || columns(&out, dir ? K : N, "out") < 0 ||
        read_groups(a[3], a[5], G, &off, &err) < 0 || read_stream_of(a + 1, 5, &s) < 0)
        return NULL;
    if (w.dtype != x.dtype || out.size[0] != x.size[0]) {
        fail("matmul", w.dtype != x.dtype ? "rows and weights of one type" : "out has a row for each row");
        return NULL;
    }
    CALL(p_grouped[dir != 0](x.p, x.stride[0], w.p, x.dtype, off, (int32_t)x.size[0], (int32_t)G, (int32_t)N, (int32_t)K, out.p, out.dtype,
                             out.stride[0], err, s));
}

/* dy, x, offsets, out, accumulate, err */
static PyObject* grouped_dw(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor dy, x, out;
    int64_t G, N, K;
    const int32_t* off;
    uint32_t* err;
    void* s;
    if (count(n, 6) < 0 || read_rows(a[0], "dy", &dy, NULL) < 0 || read_rows(a[1], "x", &x, NULL) < 0 ||
        read_matrices(a[3], "out", &out, &G, &N, &K) < 0 || columns(&dy, N, "dy") < 0 || columns(&x, K, "x") < 0 ||
        read_groups(a[2], a[5], G, &off, &err) < 0)
        return NULL;
    const int acc = PyObject_IsTrue(a[4]);
    PyObject* const t[5] = {a[0], a[1], a[2], a[3], a[5]};
    if (acc < 0 || read_stream_of(t, 5, &s) < 0) return NULL;
    if (dy.dtype != x.dtype || dy.size[0] != x.size[0] || out.dtype < 0) {
        fail("matmul_dw", out.dtype < 0 ? "out is fp32 or bf16" : "dy and x of one type, a row each");
        return NULL;
    }
    CALL(p_dw(dy.p, dy.stride[0], x.p, x.stride[0], x.dtype, off, (int32_t)x.size[0], (int32_t)G, (int32_t)N, (int32_t)K, out.p, out.dtype,
              acc, err, s));
}

/* A factor for each row: fp32 [rows], or None. */
static int read_factor(PyObject* t, int64_t rows, const char* what, float** p) {
    Tensor r;
    *p = NULL;
    if (t == Py_None) return 0;
    if (read_vector(t, rows, what, &r) < 0) return -1;
    if (r.dtype != MOE_F32) return fail(what, "fp32");
    *p = (float*)r.p;
    return 0;
}

/* gate, up, weight, out */
static PyObject* swiglu(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor g, u, out;
    float* w;
    void* s;
    if (count(n, 4) < 0 || read_rows(a[0], "gate", &g, NULL) < 0 || read_rows(a[1], "up", &u, &g) < 0 ||
        read_rows(a[3], "out", &out, &g) < 0 || read_factor(a[2], g.size[0], "weight", &w) < 0 || read_stream_of(a, 4, &s) < 0)
        return NULL;
    if (g.dtype != u.dtype) {
        fail("up", "the type of gate");
        return NULL;
    }
    CALL(p_swiglu(g.p, g.stride[0], u.p, u.stride[0], g.dtype, w, (int32_t)g.size[0], (int32_t)g.size[1], out.p, out.dtype, out.stride[0], s));
}

/* dh, gate, up, weight, dgate, dup, dweight */
static PyObject* swiglu_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor d, g, u, dg, du;
    float *w, *dw;
    void* s;
    if (count(n, 7) < 0 || read_rows(a[0], "dh", &d, NULL) < 0 || read_rows(a[1], "gate", &g, &d) < 0 || read_rows(a[2], "up", &u, &d) < 0 ||
        read_rows(a[4], "dgate", &dg, &d) < 0 || read_rows(a[5], "dup", &du, &d) < 0 || read_factor(a[3], d.size[0], "weight", &w) < 0 ||
        read_factor(a[6], d.size[0], "dweight", &dw) < 0 || read_stream_of(a, 7, &s) < 0)
        return NULL;
    if (g.dtype != d.dtype || u.dtype != d.dtype || dg.dtype != d.dtype || du.dtype != d.dtype) {
        fail("swiglu_grad", "tensors of one type");
        return NULL;
    }
    CALL(p_swiglu_grad(d.p, d.stride[0], g.p, g.stride[0], u.p, u.stride[0], d.dtype, w, (int32_t)d.size[0], (int32_t)d.size[1], dg.p,
                       dg.stride[0], du.p, du.stride[0], dw, s));
}

typedef struct {
    Tensor codes, scales;
    uint8_t* zeros;
    int64_t rows, cols, group; /* rows: of all leading dimensions */
} Coded;

/* codes, scales, zeros (or None), cols, group */
static int read_int4(PyObject* const* a, const char* what, Coded* c) {
    Tensor z;
    if (read_tensor(a[0], what, &c->codes, 0) < 0 || read_tensor(a[1], what, &c->scales, 0) < 0) return -1;
    c->cols = PyLong_AsLongLong(a[3]);
    c->group = PyLong_AsLongLong(a[4]);
    if (PyErr_Occurred()) return -1;
    if (c->group != 32 && c->group != 64 && c->group != 128) return fail(what, "groups of 32, 64 or 128 columns");
    if (c->cols < 32 || c->cols % 32 || c->cols > INT32_MAX) return fail(what, "a multiple of 32 columns");
    const int d = c->codes.dims;
    const int64_t nb = (c->cols + c->group - 1) / c->group;
    int ok = c->codes.type == t_u8 && c->scales.dtype >= 0 && d == c->scales.dims && d >= 2 && c->codes.size[d - 1] == c->cols / 2 &&
             c->scales.size[d - 1] == nb;
    c->rows = 1;
    for (int i = 0; ok && i < d - 1; ++i) {
        ok = c->codes.size[i] == c->scales.size[i];
        c->rows *= c->codes.size[i];
    }
    c->zeros = NULL;
    if (ok && a[2] != Py_None) {
        if (read_tensor(a[2], what, &z, 0) < 0) return -1;
        ok = z.type == t_u8 && z.dims == d;
        for (int i = 0; ok && i < d; ++i) ok = z.size[i] == c->scales.size[i];
        c->zeros = (uint8_t*)z.p;
    }
    return ok ? 0 : fail(what, "uint8 codes, fp32 or bf16 scales, and uint8 zeros or None, of its columns");
}

/* x, codes, scales, zeros, cols, group */
static PyObject* int4_quantize(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor x;
    Coded c;
    void* s;
    if (count(n, 6) < 0 || read_rows(a[0], "x", &x, NULL) < 0 || read_int4(a + 1, "out", &c) < 0 || held(&x, c.rows, c.cols, "out") < 0 ||
        read_stream_of(a, 4, &s) < 0)
        return NULL;
    CALL(p_int4_quantize(x.p, x.dtype, x.stride[0], c.rows, (int32_t)c.cols, (int32_t)c.group, (uint8_t*)c.codes.p, c.scales.p,
                         c.scales.dtype, c.zeros, s));
}

/* codes, scales, zeros, cols, group, out */
static PyObject* int4_dequantize(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor out;
    Coded c;
    void* s;
    if (count(n, 6) < 0 || read_int4(a, "q", &c) < 0 || read_rows(a[5], "out", &out, NULL) < 0 || held(&out, c.rows, c.cols, "q") < 0)
        return NULL;
    PyObject* const t[4] = {a[0], a[1], a[2], a[5]};
    if (read_stream_of(t, 4, &s) < 0) return NULL;
    CALL(p_int4_dequantize((const uint8_t*)c.codes.p, c.scales.p, c.scales.dtype, c.zeros, (int32_t)c.group, c.rows, (int32_t)c.cols, out.p,
                           out.dtype, out.stride[0], s));
}

/* x, codes, scales, zeros, cols, group, offsets, out, err */
static PyObject* int4_gemm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Tensor x, out;
    Coded c;
    const int32_t* off;
    uint32_t* err;
    void* s;
    if (count(n, 9) < 0 || read_rows(a[0], "x", &x, NULL) < 0 || read_int4(a + 1, "w", &c) < 0 || read_rows(a[7], "out", &out, NULL) < 0)
        return NULL;
    if (c.codes.dims > 3) {
        fail("w", "[N, K] or [G, N, K]");
        return NULL;
    }
    const int64_t G = c.codes.dims == 3 ? c.codes.size[0] : 1, N = c.codes.size[c.codes.dims - 2];
    if (G > INT32_MAX || N > INT32_MAX) {
        fail("w", "sizes below 2^31");
        return NULL;
    }
    if (columns(&x, c.cols, "x") < 0 || columns(&out, N, "out") < 0 || read_groups(a[6], a[8], G, &off, &err) < 0) return NULL;
    if (out.size[0] != x.size[0]) {
        fail("matmul", "out has a row for each row");
        return NULL;
    }
    PyObject* const t[7] = {a[0], a[1], a[2], a[3], a[6], a[7], a[8]};
    if (read_stream_of(t, 7, &s) < 0) return NULL;
    CALL(p_int4_gemm(x.p, x.dtype, x.stride[0], (const uint8_t*)c.codes.p, c.scales.p, c.scales.dtype, c.zeros, (int32_t)c.group, off,
                     (int32_t)x.size[0], (int32_t)G, (int32_t)N, (int32_t)c.cols, out.p, out.dtype, out.stride[0], err, s));
}

/* init(types (fp32, bf16, uint8, int32), current device, raw stream of a device, addresses of the block's five entry points,
 * addresses of the experts' products' eight) */
static PyObject* init(PyObject* self, PyObject* args) {
    unsigned long long f[5], e[8] = {0};
    if (!PyArg_ParseTuple(args, "(OOOO)OO(KKKKK)|(KKKKKKKK)", &t_f32, &t_bf16, &t_u8, &t_i32, &f_device, &f_stream, f, f + 1, f + 2, f + 3,
                          f + 4, e, e + 1, e + 2, e + 3, e + 4, e + 5, e + 6, e + 7))
        return NULL;
    Py_INCREF(t_f32), Py_INCREF(t_bf16), Py_INCREF(t_u8), Py_INCREF(t_i32), Py_INCREF(f_device), Py_INCREF(f_stream);
    *(void**)&p_norm_pre = (void*)f[0];
    *(void**)&p_norm_post = (void*)f[1];
    *(void**)&p_quantize = (void*)f[2];
    *(void**)&p_dequantize = (void*)f[3];
    *(void**)&p_gemm = (void*)f[4];
    *(void**)&p_grouped[0] = (void*)e[0];
    *(void**)&p_grouped[1] = (void*)e[1];
    *(void**)&p_dw = (void*)e[2];
    *(void**)&p_swiglu = (void*)e[3];
    *(void**)&p_swiglu_grad = (void*)e[4];
    *(void**)&p_int4_quantize = (void*)e[5];
    *(void**)&p_int4_dequantize = (void*)e[6];
    *(void**)&p_int4_gemm = (void*)e[7];
    Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {{"init", init, METH_VARARGS, NULL}, FAST(norm_pre), FAST(norm_post), FAST(mx_quantize), FAST(mx_dequantize),
                                FAST(mx_gemm), FAST(grouped), FAST(grouped_dw), FAST(swiglu), FAST(swiglu_grad), FAST(int4_quantize),
                                FAST(int4_dequantize), FAST(int4_gemm), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods};

PyMODINIT_FUNC PyInit__fastcall(void) {
    if (!(s_dtype = PyUnicode_InternFromString("dtype")) || !(s_is_cuda = PyUnicode_InternFromString("is_cuda")) ||
        !(s_shape = PyUnicode_InternFromString("shape")) || !(s_stride = PyUnicode_InternFromString("stride")) ||
        !(s_data_ptr = PyUnicode_InternFromString("data_ptr")) || !(s_is_contiguous = PyUnicode_InternFromString("is_contiguous")) ||
        !(s_get_device = PyUnicode_InternFromString("get_device")))
        return NULL;
    return PyModule_Create(&module);
}
