/* Argument checks and marshalling of the operators around the routed experts
 * (include/wna16_moe_block.h) and of routed experts in 8-bit floats
 * (include/wna16_moe_f8.h), as a CPython module: a decode step makes several
 * small calls, and the checks of seven tensors in Python took longer than the
 * kernel (a norm call on the Grace cores: 14.5 us, and 8.4 us with lean checks
 * through ctypes).  The entry points come in as addresses, so the module serves
 * any build of the library.  Nothing is computed or kept here. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>
#include <stdint.h>

#include "../../include/wna16_moe_f8.h"

enum { BF16, FP16, FP32, INT8, E4M3, INT32, UINT8, TYPES };
static const char* const kTypeNames[TYPES] = {"bfloat16", "float16", "float32", "int8", "float8_e4m3fn", "int32", "uint8"};
enum { FLOATS = 1 << BF16 | 1 << FP16 | 1 << FP32, CODES = 1 << INT8 | 1 << E4M3 };

static PyObject *g_types[TYPES], *g_device, *g_raw_stream; /* torch dtypes; current device; (device) -> current stream */
static PyObject *s_get_device, *s_dtype, *s_shape, *s_stride, *s_is_contiguous, *s_data_ptr, *s_cuda_stream;

typedef struct {
    char* ptr;
    int64_t n0, n1, ld; /* sizes ([n0] or [n0, n1]), distance of rows */
    int dims, type;
    int64_t n[3], st[3]; /* of up to three dims: sizes, and (layout ANY) strides */
} Tensor;

enum { WHOLE, ROWS, ANY }; /* what has to be contiguous: all of it, its rows, nothing */

/* Checks one tensor and takes it apart.  dev < 0: any CUDA device, returned in
 * *dev_out.  types: mask of allowed types; most: dims allowed. */
static int take_dims(PyObject* t, const char* name, long dev, long* dev_out, unsigned types, int layout, int most, Tensor* o) {
    PyObject* v = PyObject_CallMethodNoArgs(t, s_get_device);
    long d = -1;
    if (v) {
        d = PyLong_AsLong(v);
        Py_DECREF(v);
    }
    if (PyErr_Occurred()) PyErr_Clear();
    if (d < 0) {
        PyErr_Format(PyExc_TypeError, "%s must be a CUDA tensor", name);
        return -1;
    }
    if (dev >= 0 && d != dev) {
        PyErr_Format(PyExc_ValueError, "%s is on cuda:%ld, not on cuda:%ld", name, d, dev);
        return -1;
    }
    if (dev_out) *dev_out = d;
    if (!(v = PyObject_GetAttr(t, s_dtype))) return -1;
    o->type = -1;
    for (int i = 0; i < TYPES; ++i)
        if (v == g_types[i]) o->type = i;
    if (o->type < 0 || !(types >> o->type & 1)) {
        char want[96] = "";
        for (int i = 0; i < TYPES; ++i)
            if (types >> i & 1) {
                if (want[0]) strcat(want, " or ");
                strcat(want, kTypeNames[i]);
            }
        PyErr_Format(PyExc_TypeError, "%s must be %s, got %R", name, want, v);
        Py_DECREF(v);
        return -1;
    }
    Py_DECREF(v);
    if (!(v = PyObject_GetAttr(t, s_shape))) return -1;
    o->dims = PyTuple_Check(v) ? (int)PyTuple_GET_SIZE(v) : 0;
    if (o->dims < 1 || o->dims > most) {
        PyErr_Format(PyExc_ValueError, "%s must have %s dims, got %R", name, most == 2 ? "1 or 2" : "1 to 3", v);
        Py_DECREF(v);
        return -1;
    }
    for (int i = 0; i < o->dims; ++i) o->n[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
    o->n0 = PyLong_AsLongLong(PyTuple_GET_ITEM(v, 0));
    o->n1 = o->dims >= 2 ? PyLong_AsLongLong(PyTuple_GET_ITEM(v, 1)) : 1;
    Py_DECREF(v);
    o->ld = o->n1 > 0 ? o->n1 : 1;
    if (layout == ANY) {
        if (!(v = PyObject_CallMethodNoArgs(t, s_stride))) return -1;
        if (PyTuple_Check(v) && PyTuple_GET_SIZE(v) == o->dims)
            for (int i = 0; i < o->dims; ++i) o->st[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
        Py_DECREF(v);
    } else if (layout == ROWS) {
        if (!(v = PyObject_CallMethodNoArgs(t, s_stride))) return -1;
        if (o->dims == 2 && PyTuple_Check(v) && PyTuple_GET_SIZE(v) == 2) {
            if (o->n0 > 1) o->ld = PyLong_AsLongLong(PyTuple_GET_ITEM(v, 0));
            if (o->n1 > 1 && PyLong_AsLongLong(PyTuple_GET_ITEM(v, 1)) != 1) {
                PyErr_Format(PyExc_ValueError, "the rows of %s must be contiguous", name);
                Py_DECREF(v);
                return -1;
            }
        }
        Py_DECREF(v);
    } else {
        if (!(v = PyObject_CallMethodNoArgs(t, s_is_contiguous))) return -1;
        const int ok = v == Py_True;
        Py_DECREF(v);
        if (!ok) {
            PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
            return -1;
        }
    }
    if (!(v = PyObject_CallMethodNoArgs(t, s_data_ptr))) return -1;
    o->ptr = (char*)PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return PyErr_Occurred() ? -1 : 0;
}

static int take(PyObject* t, const char* name, long dev, long* dev_out, unsigned types, int layout, Tensor* o) {
    return take_dims(t, name, dev, dev_out, types, layout, 2, o);
}

static int want_rows(const Tensor* t, const char* name, int64_t n0, int64_t n1) {
    if (t->dims == 2 && t->n0 == n0 && t->n1 == n1) return 0;
    PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld], got [%lld, %lld]", name, (long long)n0, (long long)n1,
                 (long long)t->n0, (long long)t->n1);
    return -1;
}
/* n values, [n] or (column) [n, 1] */
static int want_list(const Tensor* t, const char* name, int64_t n, int column) {
    if (t->n0 == n && (t->dims == 1 || (column && t->n1 == 1))) return 0;
    PyErr_Format(PyExc_ValueError, "%s must hold %lld values, got [%lld, %lld]", name, (long long)n, (long long)t->n0,
                 (long long)t->n1);
    return -1;
}

/* The stream of a call: `stream`'s (a torch stream) or the device's current one, which must be the current device. */
static int stream_of(PyObject* stream, const char* name, long dev, void** out) {
    PyObject* v = PyObject_CallNoArgs(g_device);
    if (!v) return -1;
    const long now = PyLong_AsLong(v);
    Py_DECREF(v);
    if (now != dev) {
        PyErr_Format(PyExc_ValueError, "%s is on cuda:%ld, the current device is cuda:%ld", name, dev, now);
        return -1;
    }
    if (stream == Py_None) {
        PyObject* d = PyLong_FromLong(dev);
        v = d ? PyObject_CallOneArg(g_raw_stream, d) : NULL;
        Py_XDECREF(d);
    } else {
        v = PyObject_GetAttr(stream, s_cuda_stream);
    }
    if (!v) return -1;
    *out = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return PyErr_Occurred() ? -1 : 0;
}

/* Numbers are read before the tensors: with an exception set nothing else may be called. */
static int to_int(PyObject* o, const char* name, int* out) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) return -1;
    if (v < INT_MIN || v > INT_MAX) {
        PyErr_Format(PyExc_OverflowError, "%s=%ld does not fit 32 bits", name, v);
        return -1;
    }
    *out = (int)v;
    return 0;
}
static int to_float(PyObject* o, float* out) {
    const double v = PyFloat_AsDouble(o);
    *out = (float)v;
    return v == -1.0 && PyErr_Occurred() ? -1 : 0;
}

static int arity(Py_ssize_t got, Py_ssize_t want) {
    if (got == want) return 0;
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", got, want);
    return -1;
}
#define ADDRESS(type) ((type)PyLong_AsVoidPtr(a[0]))
#define MAYBE(obj) ((obj) != Py_None)

/* The 8-bit rows [T, K] and their scales [T, groups]. */
static int take_q(PyObject* q, PyObject* s, long dev, int64_t T, int64_t K, int group, Tensor* tq, Tensor* ts) {
    if (take(q, "q", dev, NULL, CODES, 0, tq) || take(s, "scales", dev, NULL, 1 << FP32, 0, ts)) return -1;
    return want_rows(tq, "q", T, K) || want_rows(ts, "scales", T, group > 0 ? K / group : 1) ? -1 : 0;
}

/* (entry, x, weight, residual, residual_out, norm_out, q, scales, eps, group_size, stream); None where absent */
static PyObject* add_rmsnorm_q8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor x, w, r = {0}, ro = {0}, no = {0}, q = {0}, s = {0};
    long dev;
    void* stream;
    int group;
    float eps;
    if (arity(n, 11) || to_float(a[8], &eps) || to_int(a[9], "group_size", &group) ||
        take(a[1], "x", -1, &dev, FLOATS, 1, &x) || want_rows(&x, "x", x.n0, x.n1) ||
        take(a[2], "weight", dev, NULL, 1u << x.type | 1u << FP32, 0, &w))
        return NULL;
    if (w.dims != 1 || w.n0 != x.n1) {
        PyErr_Format(PyExc_ValueError, "weight must be [%lld], got [%lld]", (long long)x.n1, (long long)w.n0);
        return NULL;
    }
    const unsigned same = 1u << x.type;
    if (MAYBE(a[3]) && (take(a[3], "residual", dev, NULL, same, 1, &r) || want_rows(&r, "residual", x.n0, x.n1))) return NULL;
    if (MAYBE(a[4]) && (take(a[4], "residual_out", dev, NULL, same, 0, &ro) || want_rows(&ro, "residual_out", x.n0, x.n1)))
        return NULL;
    if (MAYBE(a[5]) && (take(a[5], "norm_out", dev, NULL, same, 0, &no) || want_rows(&no, "norm_out", x.n0, x.n1))) return NULL;
    if (MAYBE(a[6]) && take_q(a[6], a[7], dev, x.n0, x.n1, group, &q, &s)) return NULL;
    if (stream_of(a[10], "x", dev, &stream)) return NULL;
    return PyLong_FromLong(ADDRESS(__typeof__(&wna16_moe_add_rmsnorm_q8))(
        x.ptr, x.ld, r.ptr, r.ld, w.ptr, w.type, x.n0, x.n1, x.type, eps,
        q.type == E4M3 && MAYBE(a[6]) ? WNA16_Q8_E4M3 : WNA16_Q8_INT8, group, q.ptr, (float*)s.ptr, ro.ptr, no.ptr, stream));
}

/* (entry, gu, q, scales, limit, group_size, stream) */
static PyObject* swiglu_q8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor x, q, s;
    long dev;
    void* stream;
    int group;
    float limit;
    if (arity(n, 7) || to_float(a[4], &limit) || to_int(a[5], "group_size", &group) ||
        take(a[1], "gu", -1, &dev, FLOATS, 1, &x) || want_rows(&x, "gu", x.n0, x.n1))
        return NULL;
    if (x.n1 % 2) {
        PyErr_Format(PyExc_ValueError, "gu must have an even number of columns, got %lld", (long long)x.n1);
        return NULL;
    }
    if (take_q(a[2], a[3], dev, x.n0, x.n1 / 2, group, &q, &s) || stream_of(a[6], "gu", dev, &stream)) return NULL;
    return PyLong_FromLong(ADDRESS(__typeof__(&wna16_moe_swiglu_q8))(
        x.ptr, x.ld, x.n0, x.n1 / 2, x.type, limit, q.type == E4M3 ? WNA16_Q8_E4M3 : WNA16_Q8_INT8, group, q.ptr,
        (float*)s.ptr, stream));
}

/* (entry, x, q, scales, group_size, stream) */
static PyObject* quantize_q8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor x, q, s;
    long dev;
    void* stream;
    int group;
    if (arity(n, 6) || to_int(a[4], "group_size", &group) || take(a[1], "x", -1, &dev, FLOATS, 1, &x) ||
        want_rows(&x, "x", x.n0, x.n1) || take_q(a[2], a[3], dev, x.n0, x.n1, group, &q, &s) || stream_of(a[5], "x", dev, &stream))
        return NULL;
    return PyLong_FromLong(ADDRESS(__typeof__(&wna16_moe_quantize_q8))(
        x.ptr, x.ld, x.n0, x.n1, x.type, q.type == E4M3 ? WNA16_Q8_E4M3 : WNA16_Q8_INT8, group, q.ptr, (float*)s.ptr,
        stream));
}

/* (entry, q, scales, out, stream) */
static PyObject* dequantize_q8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor q, s, o;
    long dev;
    void* stream;
    if (arity(n, 5) || take(a[1], "q", -1, &dev, CODES, 0, &q) || want_rows(&q, "q", q.n0, q.n1) ||
        take(a[2], "scales", dev, NULL, 1 << FP32, 0, &s) || take(a[3], "out", dev, NULL, FLOATS, 0, &o) ||
        want_rows(&o, "out", q.n0, q.n1))
        return NULL;
    if (s.dims != 2 || s.n0 != q.n0 || s.n1 < 1 || q.n1 % s.n1) {
        PyErr_Format(PyExc_ValueError, "scales must be [%lld, groups] with groups dividing %lld, got [%lld, %lld]",
                     (long long)q.n0, (long long)q.n1, (long long)s.n0, (long long)s.n1);
        return NULL;
    }
    const int64_t group = s.n1 > 1 ? q.n1 / s.n1 : 0;
    if (stream_of(a[4], "q", dev, &stream)) return NULL;
    return PyLong_FromLong(ADDRESS(__typeof__(&wna16_moe_dequantize_q8))(
        q.ptr, (const float*)s.ptr, q.n0, q.n1, q.type == E4M3 ? WNA16_Q8_E4M3 : WNA16_Q8_INT8,
        group > 1 << 20 ? -1 : (int)group, o.type, o.ptr, stream));
}

/* (entry, logits, bias, ids, weights, score, groups, topk_groups, group_score, topk, renormalize, scale, stream) */
static PyObject* route_scored(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor x, b = {0}, ids, w;
    long dev;
    void* stream;
    static const char* const names[6] = {"score", "groups", "topk_groups", "group_score", "topk", "renormalize"};
    int v[6];
    float scale;
    if (arity(n, 13) || to_float(a[11], &scale)) return NULL;
    for (int i = 0; i < 6; ++i)
        if (to_int(a[5 + i], names[i], &v[i])) return NULL;
    if (take(a[1], "logits", -1, &dev, FLOATS, 1, &x) || want_rows(&x, "logits", x.n0, x.n1)) return NULL;
    if (MAYBE(a[2]) && (take(a[2], "bias", dev, NULL, 1 << FP32, 0, &b) || want_list(&b, "bias", x.n1, 0))) return NULL;
    if (take(a[3], "ids", dev, NULL, 1 << INT32, 0, &ids) || want_rows(&ids, "ids", x.n0, v[4]) ||
        take(a[4], "weights", dev, NULL, 1 << FP32, 0, &w) || want_rows(&w, "weights", x.n0, v[4]))
        return NULL;
    if (stream_of(a[12], "logits", dev, &stream)) return NULL;
    return PyLong_FromLong(ADDRESS(__typeof__(&wna16_moe_route_scored))(
        x.ptr, x.ld, (const float*)b.ptr, x.n0, x.n1, x.type, v[0], v[1], v[2], v[3], v[4], v[5], scale, (int32_t*)ids.ptr,
        (float*)w.ptr, stream));
}

/* (entry, xq, x_scales, wq, w_scales, bias, addend, out, workspace, stream) */
static PyObject* linear_q8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor x, xs, w, ws, b = {0}, add = {0}, o, work = {0};
    long dev;
    void* stream;
    if (arity(n, 10) || take(a[1], "xq", -1, &dev, 1 << INT8, 0, &x) || want_rows(&x, "xq", x.n0, x.n1) ||
        take(a[3], "wq", dev, NULL, 1 << INT8, 0, &w) || want_rows(&w, "wq", w.n0, x.n1) ||
        take(a[2], "x_scales", dev, NULL, 1 << FP32, 0, &xs) || want_list(&xs, "x_scales", x.n0, 1) ||
        take(a[4], "w_scales", dev, NULL, 1 << FP32, 0, &ws) || want_list(&ws, "w_scales", w.n0, 1) ||
        take(a[7], "out", dev, NULL, FLOATS, 0, &o) || want_rows(&o, "out", x.n0, w.n0))
        return NULL;
    if (MAYBE(a[5]) && (take(a[5], "bias", dev, NULL, 1 << FP32, 0, &b) || want_list(&b, "bias", w.n0, 0))) return NULL;
    if (MAYBE(a[6]) && (take(a[6], "addend", dev, NULL, 1u << o.type, 0, &add) || want_rows(&add, "addend", x.n0, w.n0)))
        return NULL;
    if (MAYBE(a[8]) && (take(a[8], "workspace", dev, NULL, 1 << UINT8, 0, &work))) return NULL;
    if (stream_of(a[9], "xq", dev, &stream)) return NULL;
    return PyLong_FromLong(ADDRESS(__typeof__(&wna16_moe_linear_q8))(
        (const int8_t*)x.ptr, (const float*)xs.ptr, (const int8_t*)w.ptr, (const float*)ws.ptr, (const float*)b.ptr, add.ptr,
        x.n0, x.n1, w.n0, o.type, o.ptr, work.ptr, work.ptr ? (size_t)work.n0 : 0, stream));
}

static int want_shape(const Tensor* t, const char* name, int dims, int64_t a, int64_t b, int64_t c) {
    const int64_t want[3] = {a, b, c};
    int same = t->dims == dims;
    for (int i = 0; same && i < dims; ++i) same = t->n[i] == want[i];
    if (same) return 0;
    if (dims == 3)
        PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld, %lld]", name, (long long)a, (long long)b, (long long)c);
    else
        PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld]", name, (long long)a, (long long)b);
    return -1;
}

/* (entry, x, x_scales, ids, E, expert_begin, rows, row_scales, offsets, inv, stream) */
static PyObject* sort_tokens(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor x = {0}, xs = {0}, ids, rows = {0}, rs = {0}, off, inv;
    long dev;
    void* stream;
    int E, begin;
    if (arity(n, 11) || to_int(a[4], "experts", &E) || to_int(a[5], "expert_begin", &begin) ||
        take(a[3], "topk_ids", -1, &dev, 1 << INT32, WHOLE, &ids) || want_rows(&ids, "topk_ids", ids.n0, ids.n1))
        return NULL;
    if (ids.n1 > 1024 || ids.n0 >= (int64_t)1 << 31) {
        PyErr_Format(PyExc_ValueError, "topk_ids [%lld, %lld] is too large", (long long)ids.n0, (long long)ids.n1);
        return NULL;
    }
    static const struct { int out, in; const char* message; } kPairs[] = {
        {6, 1, "rows without x"}, {2, 1, "scales without x"}, {7, 2, "row_scales without scales"}};
    for (int i = 0; i < 3; ++i)
        if (MAYBE(a[kPairs[i].out]) && !MAYBE(a[kPairs[i].in])) {
            PyErr_SetString(PyExc_ValueError, kPairs[i].message);
            return NULL;
        }
    const int64_t R = ids.n0 * ids.n1;
    if (MAYBE(a[1]) && (take(a[1], "x", dev, NULL, FLOATS | CODES, ROWS, &x) || want_rows(&x, "x", ids.n0, x.n1) ||
                        take(a[6], "rows", dev, NULL, 1u << x.type, WHOLE, &rows) || want_rows(&rows, "rows", R, x.n1)))
        return NULL;
    if (MAYBE(a[2]) && (take(a[2], "scales", dev, NULL, 1 << FP32, WHOLE, &xs) || want_rows(&xs, "scales", ids.n0, xs.n1) ||
                        take(a[7], "row_scales", dev, NULL, 1 << FP32, WHOLE, &rs) || want_rows(&rs, "row_scales", R, xs.n1)))
        return NULL;
    if (take(a[8], "offsets", dev, NULL, 1 << INT32, WHOLE, &off) || want_list(&off, "offsets", (int64_t)E + 1, 0) ||
        take(a[9], "inv", dev, NULL, 1 << INT32, WHOLE, &inv) || want_rows(&inv, "inv", ids.n0, ids.n1) ||
        stream_of(a[10], "topk_ids", dev, &stream))
        return NULL;
    const int type = !MAYBE(a[1]) || x.type == INT8 || x.type == E4M3 ? WNA16_TYPE_Q8 : x.type;
    return PyLong_FromLong(ADDRESS(__typeof__(&wna16_moe_sort_tokens))(
        x.ptr, x.ld, (const float*)xs.ptr, xs.n1, ids.n0, MAYBE(a[1]) ? x.n1 : 1, type, (const int32_t*)ids.ptr, (int)ids.n1,
        E, begin, rows.ptr, (float*)rs.ptr, (int32_t*)off.ptr, (int32_t*)inv.ptr, stream));
}

/* inv [T, topk] and weights of the same sizes */
static int take_slots(PyObject* i, PyObject* w, long dev, int64_t T, Tensor* ti, Tensor* tw) {
    if (take(i, "inv", dev, NULL, 1 << INT32, WHOLE, ti) || want_rows(ti, "inv", T, ti->n1)) return -1;
    if (ti->n1 > 1024) {
        PyErr_Format(PyExc_ValueError, "inv has %lld slots per token, at most 1024", (long long)ti->n1);
        return -1;
    }
    return MAYBE(w) && (take(w, "weights", dev, NULL, 1 << FP32, WHOLE, tw) || want_rows(tw, "weights", T, ti->n1)) ? -1 : 0;
}

/* (entry, y, inv, weights, addend, out, stream) */
static PyObject* unsort_tokens(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor y, inv, w = {0}, add = {0}, o;
    long dev;
    void* stream;
    if (arity(n, 7) || take(a[1], "y", -1, &dev, FLOATS, WHOLE, &y) || want_rows(&y, "y", y.n0, y.n1) ||
        take(a[5], "out", dev, NULL, 1u << y.type, WHOLE, &o) || want_rows(&o, "out", o.n0, y.n1) ||
        take_slots(a[2], a[3], dev, o.n0, &inv, &w))
        return NULL;
    if (MAYBE(a[4]) && (take(a[4], "addend", dev, NULL, 1u << y.type, WHOLE, &add) || want_rows(&add, "addend", o.n0, y.n1)))
        return NULL;
    if (stream_of(a[6], "y", dev, &stream)) return NULL;
    return PyLong_FromLong(ADDRESS(__typeof__(&wna16_moe_unsort_tokens))(
        y.ptr, y.n0, (const int32_t*)inv.ptr, (const float*)w.ptr, add.ptr, o.n0, y.n1, (int)inv.n1, y.type, o.ptr, stream));
}

/* (entry, dout, inv, y, weights, dy, dweights, stream); R is the rows of dy or y */
static PyObject* unsort_tokens_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor d, inv, y = {0}, w = {0}, dy = {0}, dw = {0};
    long dev;
    void* stream;
    if (arity(n, 8) || take(a[1], "dout", -1, &dev, FLOATS, WHOLE, &d) || want_rows(&d, "dout", d.n0, d.n1) ||
        take_slots(a[2], a[4], dev, d.n0, &inv, &w))
        return NULL;
    const unsigned same = 1u << d.type;
    if (!MAYBE(a[5]) && !MAYBE(a[6]) && d.n0 > 0) {   /* (R is not known without them) */
        PyErr_SetString(PyExc_ValueError, "neither dy nor y: no gradient is wanted");
        return NULL;
    }
    if (MAYBE(a[3]) && (take(a[3], "y", dev, NULL, same, WHOLE, &y) || want_rows(&y, "y", y.n0, d.n1))) return NULL;
    if (MAYBE(a[5]) && (take(a[5], "dy", dev, NULL, same, WHOLE, &dy) ||
                        want_rows(&dy, "dy", MAYBE(a[3]) ? y.n0 : dy.n0, d.n1)))
        return NULL;
    if (MAYBE(a[6]) && (take(a[6], "dweights", dev, NULL, 1 << FP32, WHOLE, &dw) || want_rows(&dw, "dweights", d.n0, inv.n1)))
        return NULL;
    if (stream_of(a[7], "dout", dev, &stream)) return NULL;
    return PyLong_FromLong(ADDRESS(__typeof__(&wna16_moe_unsort_tokens_grad))(
        d.ptr, (const int32_t*)inv.ptr, y.ptr, (const float*)w.ptr, d.n0, d.n1, (int)inv.n1, MAYBE(a[3]) ? y.n0 : dy.n0,
        d.type, dy.ptr, (float*)dw.ptr, stream));
}

/* 8-bit float rows [T, K], their scales, weights [(E,) N, K] and theirs */
static int take_f8(PyObject* const* a, int dims, long* dev, Tensor* x, Tensor* xs, Tensor* w, Tensor* ws) {
    if (take(a[1], "xq", -1, dev, 1 << E4M3, WHOLE, x) || want_rows(x, "xq", x->n0, x->n1) ||
        take(a[2], "x_scales", *dev, NULL, 1 << FP32, WHOLE, xs) || want_rows(xs, "x_scales", x->n0, x->n1 / 128) ||
        take_dims(a[3], "wq", *dev, NULL, 1 << E4M3, WHOLE, dims, w))
        return -1;
    const int64_t N = w->n[dims - 2];
    if (dims == 3 ? want_shape(w, "wq", 3, w->n[0], N, x->n1) : want_shape(w, "wq", 2, N, x->n1, 0)) return -1;
    if (take_dims(a[4], "w_scales", *dev, NULL, 1 << FP32, WHOLE, dims, ws)) return -1;
    return dims == 3 ? want_shape(ws, "w_scales", 3, w->n[0], (N + 127) / 128, x->n1 / 128)
                     : want_shape(ws, "w_scales", 2, (N + 127) / 128, x->n1 / 128, 0);
}

/* (entry, xq, x_scales, wq, w_scales, bias, addend, out, workspace, stream) */
static PyObject* linear_f8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor x, xs, w = {0}, ws = {0}, b = {0}, add = {0}, o, work = {0};
    long dev;
    void* stream;
    if (arity(n, 10) || take_f8(a, 2, &dev, &x, &xs, &w, &ws) || take(a[7], "out", dev, NULL, FLOATS, WHOLE, &o) ||
        want_rows(&o, "out", x.n0, w.n[0]))
        return NULL;
    if (MAYBE(a[5]) && (take(a[5], "bias", dev, NULL, 1 << FP32, WHOLE, &b) || want_list(&b, "bias", w.n[0], 0))) return NULL;
    if (MAYBE(a[6]) && (take(a[6], "addend", dev, NULL, 1u << o.type, WHOLE, &add) || want_rows(&add, "addend", x.n0, w.n[0])))
        return NULL;
    if (MAYBE(a[8]) && (take(a[8], "workspace", dev, NULL, 1 << UINT8, WHOLE, &work))) return NULL;
    if (stream_of(a[9], "xq", dev, &stream)) return NULL;
    return PyLong_FromLong(ADDRESS(__typeof__(&wna16_moe_linear_f8))(
        x.ptr, (const float*)xs.ptr, w.ptr, (const float*)ws.ptr, (const float*)b.ptr, add.ptr, x.n0, x.n1, w.n[0], o.type,
        o.ptr, work.ptr, work.ptr ? (size_t)work.n0 : 0, stream));
}

/* (entry, xq, x_scales, wq, w_scales, offsets, out, workspace, stream) */
static PyObject* grouped_linear_f8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor x, xs, w = {0}, ws = {0}, off, o, work = {0};
    long dev;
    void* stream;
    if (arity(n, 9) || take_f8(a, 3, &dev, &x, &xs, &w, &ws) || take(a[5], "offsets", dev, NULL, 1 << INT32, WHOLE, &off) ||
        want_list(&off, "offsets", w.n[0] + 1, 0) || take(a[6], "out", dev, NULL, FLOATS, WHOLE, &o) ||
        want_rows(&o, "out", x.n0, w.n[1]))
        return NULL;
    if (MAYBE(a[7]) && (take(a[7], "workspace", dev, NULL, 1 << UINT8, WHOLE, &work))) return NULL;
    if (stream_of(a[8], "xq", dev, &stream)) return NULL;
    return PyLong_FromLong(ADDRESS(__typeof__(&wna16_moe_grouped_linear_f8))(
        x.ptr, (const float*)xs.ptr, w.ptr, (const float*)ws.ptr, (const int32_t*)off.ptr, w.n[0], x.n0, x.n1, w.n[1], o.type,
        o.ptr, work.ptr, work.ptr ? (size_t)work.n0 : 0, stream));
}

/* (entry, w, q, scales, stream); w and q [N, K] or [E, N, K] */
static PyObject* quantize_blocks_f8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    Tensor w = {0}, q = {0}, s = {0};
    long dev;
    void* stream;
    if (arity(n, 5) || take_dims(a[1], "w", -1, &dev, FLOATS, ANY, 3, &w)) return NULL;
    if (w.dims < 2) {
        PyErr_SetString(PyExc_ValueError, "w must have 2 or 3 dims");
        return NULL;
    }
    const int d = w.dims;
    const int64_t E = d == 3 ? w.n[0] : 1, N = w.n[d - 2], K = w.n[d - 1];
    if (take_dims(a[2], "q", dev, NULL, 1 << E4M3, WHOLE, 3, &q) || want_shape(&q, "q", d, w.n[0], w.n[1], w.n[2]) ||
        take_dims(a[3], "scales", dev, NULL, 1 << FP32, WHOLE, 3, &s) ||
        (d == 3 ? want_shape(&s, "scales", 3, E, (N + 127) / 128, K / 128) : want_shape(&s, "scales", 2, (N + 127) / 128, K / 128, 0)) ||
        stream_of(a[4], "w", dev, &stream))
        return NULL;
    return PyLong_FromLong(ADDRESS(__typeof__(&wna16_moe_quantize_blocks_f8))(
        w.ptr, E, N, K, d == 3 ? w.st[0] : 0, w.st[d - 2], w.st[d - 1], w.type, q.ptr, (float*)s.ptr, stream));
}

/* ((bfloat16, float16, float32, int8, float8_e4m3fn, int32, uint8), current_device, raw_stream) */
static PyObject* setup(PyObject* self, PyObject* args) {
    PyObject *types, *device, *raw;
    (void)self;
    if (!PyArg_ParseTuple(args, "O!OO", &PyTuple_Type, &types, &device, &raw)) return NULL;
    if (PyTuple_GET_SIZE(types) != TYPES) {
        PyErr_SetString(PyExc_ValueError, "types");
        return NULL;
    }
    for (int i = 0; i < TYPES; ++i) {
        Py_XDECREF(g_types[i]);
        g_types[i] = Py_NewRef(PyTuple_GET_ITEM(types, i));
    }
    Py_XDECREF(g_device);
    g_device = Py_NewRef(device);
    Py_XDECREF(g_raw_stream);
    g_raw_stream = Py_NewRef(raw);
    Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef kMethods[] = {{"setup", setup, METH_VARARGS, NULL}, FAST(add_rmsnorm_q8), FAST(swiglu_q8),
                                 FAST(quantize_q8), FAST(dequantize_q8), FAST(route_scored), FAST(linear_q8),
                                 FAST(sort_tokens), FAST(unsort_tokens), FAST(unsort_tokens_grad), FAST(linear_f8),
                                 FAST(grouped_linear_f8), FAST(quantize_blocks_f8),
                                 {NULL, NULL, 0, NULL}};
static struct PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_host", "Argument checks of the block operators.", -1, kMethods,
                                     NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__host(void) {
    s_get_device = PyUnicode_InternFromString("get_device");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    return PyModule_Create(&kModule);
}
