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

static PyObject *s_dtype, *s_is_cuda, *s_shape, *s_stride, *s_data_ptr, *s_is_contiguous;
static PyObject *t_f32, *t_bf16, *t_u8, *t_i32, *f_device, *f_stream;

static moe_status (*p_norm_pre)(const moe_norm*, const void*, int32_t, int64_t, int32_t, int32_t, void*, int32_t, int64_t, void*);
static moe_status (*p_norm_post)(const moe_post*, const void*, int32_t, int64_t, const void*, int32_t, int64_t, int32_t, int32_t, void*,
                                 int64_t, void*, int32_t, int64_t, void*);
static moe_status (*p_quantize)(const void*, int32_t, int64_t, int64_t, int32_t, uint8_t*, uint8_t*, void*);
static moe_status (*p_dequantize)(const uint8_t*, const uint8_t*, int64_t, int32_t, void*, int32_t, int64_t, void*);
static moe_status (*p_gemm)(const uint8_t*, const uint8_t*, const uint8_t*, const uint8_t*, const int32_t*, int32_t, int32_t, int32_t,
                            int32_t, void*, int32_t, int64_t, uint32_t*, void*);

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

/* init(types (fp32, bf16, uint8, int32), current device, raw stream of a device, addresses of the five entry points) */
static PyObject* init(PyObject* self, PyObject* args) {
    unsigned long long f[5];
    if (!PyArg_ParseTuple(args, "(OOOO)OO(KKKKK)", &t_f32, &t_bf16, &t_u8, &t_i32, &f_device, &f_stream, f, f + 1, f + 2, f + 3, f + 4)) return NULL;
    Py_INCREF(t_f32), Py_INCREF(t_bf16), Py_INCREF(t_u8), Py_INCREF(t_i32), Py_INCREF(f_device), Py_INCREF(f_stream);
    *(void**)&p_norm_pre = (void*)f[0];
    *(void**)&p_norm_post = (void*)f[1];
    *(void**)&p_quantize = (void*)f[2];
    *(void**)&p_dequantize = (void*)f[3];
    *(void**)&p_gemm = (void*)f[4];
    Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {{"init", init, METH_VARARGS, NULL}, FAST(norm_pre), FAST(norm_post), FAST(mx_quantize), FAST(mx_dequantize),
                                FAST(mx_gemm), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods};

PyMODINIT_FUNC PyInit__fastcall(void) {
    if (!(s_dtype = PyUnicode_InternFromString("dtype")) || !(s_is_cuda = PyUnicode_InternFromString("is_cuda")) ||
        !(s_shape = PyUnicode_InternFromString("shape")) || !(s_stride = PyUnicode_InternFromString("stride")) ||
        !(s_data_ptr = PyUnicode_InternFromString("data_ptr")) || !(s_is_contiguous = PyUnicode_InternFromString("is_contiguous")))
        return NULL;
    return PyModule_Create(&module);
}
