/* _call.c -- the calls of the packed-sequence operators from Python: each checks its tensors
 * (type, shape, layout, device), takes their addresses and calls the C entry point of librr.so.
 * The same checks written in Python cost a call 8 of its 14 microseconds, more than most of
 * these kernels take on a decoding step's sizes.  Plain CPython API; torch's tensors are asked
 * through their methods.  The entry points run without the interpreter's lock: a launch waits
 * while a stream's queue is full, perhaps for a host callback that needs the lock. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

enum { ROPE_FWD, ROPE_BWD, ATTN_FWD, ATTN_BWD, LOGP_FWD, LOGP_BWD, ENTRIES };
static void *entry[ENTRIES];
static PyObject *f32, *bf16, *i32, *get_device, *raw_stream;
static PyObject *s_dtype, *s_shape, *s_stride, *s_contig, *s_ptr, *s_dev;

typedef struct {
    const char *fn;
    long device;
    int bad; /* an error is set */
} Call;
typedef struct {
    void *p;
    int64_t row; /* elements from a row to the next (rows) */
} Tensor;

/* sizes: a negative entry takes the tensor's and is written back. */
static Tensor tensor(Call *c, const char *name, PyObject *t, PyObject *dtype, int nd, int64_t *size,
                     int rows) {
    Tensor out = {NULL, 0};
    if (c->bad || t == Py_None) return out;
    c->bad = 1;
    PyObject *o = PyObject_GetAttr(t, s_dtype);
    if (!o) return out;
    int same = o == dtype;
    if (!same) PyErr_Format(PyExc_TypeError, "%s: %s must be %S, not %S", c->fn, name, dtype, o);
    Py_DECREF(o);
    if (!same) return out;
    if (!(o = PyObject_GetAttr(t, s_shape))) return out;
    int fits = PyTuple_Check(o) && PyTuple_GET_SIZE(o) == nd;
    for (int i = 0; fits && i < nd; ++i) {
        const int64_t n = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
        if (size[i] < 0) size[i] = n;
        fits = size[i] == n;
    }
    if (!fits) {
        PyObject *want = PyTuple_New(nd);
        for (int i = 0; want && i < nd; ++i) PyTuple_SET_ITEM(want, i, PyLong_FromLongLong(size[i]));
        PyErr_Format(PyExc_ValueError, "%s: %s must have shape %S, not %S", c->fn, name, want, o);
        Py_XDECREF(want);
    }
    Py_DECREF(o);
    if (!fits) return out;
    if (rows) {
        if (!(o = PyObject_CallMethodNoArgs(t, s_stride))) return out;
        int64_t width = 1;
        int dense = PyTuple_Check(o) && PyTuple_GET_SIZE(o) == nd;
        for (int i = nd - 1; dense && i >= 1; --i) {
            if (size[i] > 1 && PyLong_AsLongLong(PyTuple_GET_ITEM(o, i)) != width) dense = 0;
            width *= size[i];
        }
        out.row = dense && size[0] > 1 ? PyLong_AsLongLong(PyTuple_GET_ITEM(o, 0)) : width;
        Py_DECREF(o);
        if (!dense) {
            PyErr_Format(PyExc_ValueError, "%s: the rows of %s must be dense", c->fn, name);
            return out;
        }
    } else {
        if (!(o = PyObject_CallMethodNoArgs(t, s_contig))) return out;
        const int dense = o == Py_True;
        Py_DECREF(o);
        if (!dense) {
            PyErr_Format(PyExc_ValueError, "%s: %s must be contiguous", c->fn, name);
            return out;
        }
    }
    if (!(o = PyObject_CallMethodNoArgs(t, s_dev))) return out;
    const long dev = PyLong_AsLong(o);
    Py_DECREF(o);
    if (dev != c->device) {
        PyErr_Format(PyExc_ValueError, "%s: %s must be a CUDA tensor on the current device", c->fn,
                     name);
        return out;
    }
    if (!(o = PyObject_CallMethodNoArgs(t, s_ptr))) return out;
    out.p = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    if (PyErr_Occurred()) return out;
    c->bad = 0;
    return out;
}

static Call begin(const char *fn) {
    Call c = {fn, 0, 1};
    PyObject *o = PyObject_CallNoArgs(get_device);
    if (!o) return c;
    c.device = PyLong_AsLong(o);
    Py_DECREF(o);
    c.bad = PyErr_Occurred() != NULL;
    return c;
}
static void *stream_of(Call *c, PyObject *stream) {
    if (c->bad) return NULL;
    if (stream != Py_None) {
        void *p = PyLong_AsVoidPtr(stream);
        c->bad = PyErr_Occurred() != NULL;
        return p;
    }
    PyObject *d = PyLong_FromLong(c->device);
    PyObject *o = d ? PyObject_CallOneArg(raw_stream, d) : NULL;
    Py_XDECREF(d);
    if (!o) {
        c->bad = 1;
        return NULL;
    }
    void *p = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    c->bad = PyErr_Occurred() != NULL;
    return p;
}
/* The storage type of a tensor: 0 float32, 1 bfloat16. */
static int storage(Call *c, PyObject *t, PyObject **dtype) {
    if (c->bad) return 0;
    c->bad = 1;
    PyObject *o = PyObject_GetAttr(t, s_dtype);
    if (!o) return 0;
    Py_DECREF(o); /* (torch keeps its dtypes alive) */
    if (o != f32 && o != bf16) {
        PyErr_Format(PyExc_TypeError, "unsupported dtype %S", o);
        return 0;
    }
    c->bad = 0;
    *dtype = o;
    return o == bf16;
}
static double number(Call *c, PyObject *o) {
    if (c->bad) return 0;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) c->bad = 1;
    return v;
}
static int truth(Call *c, PyObject *o) {
    if (c->bad) return 0;
    const int v = PyObject_IsTrue(o);
    if (v < 0) c->bad = 1;
    return v;
}
static int32_t whole(Call *c, const char *name, PyObject *o) {
    if (c->bad) return 0;
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        c->bad = 1;
    } else if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_Format(PyExc_ValueError, "%s: %s must fit 32 bits", c->fn, name);
        c->bad = 1;
    }
    return (int32_t)v;
}
/* A workspace: its address and bytes (numel x element_size; uint8 in practice). */
static void *workspace(Call *c, PyObject *t, size_t *bytes) {
    *bytes = 0;
    if (c->bad || t == Py_None) return NULL;
    c->bad = 1;
    PyObject *o = PyObject_CallMethodNoArgs(t, s_contig);
    if (!o) return NULL;
    const int dense = o == Py_True;
    Py_DECREF(o);
    if (!dense) {
        PyErr_Format(PyExc_ValueError, "%s: workspace must be contiguous", c->fn);
        return NULL;
    }
    if (!(o = PyObject_CallMethodNoArgs(t, s_dev))) return NULL;
    const long dev = PyLong_AsLong(o);
    Py_DECREF(o);
    if (dev != c->device) {
        PyErr_Format(PyExc_ValueError, "%s: workspace must be a CUDA tensor on the current device",
                     c->fn);
        return NULL;
    }
    if (!(o = PyObject_GetAttrString(t, "nbytes"))) return NULL;
    *bytes = PyLong_AsSize_t(o);
    Py_DECREF(o);
    if (!(o = PyObject_CallMethodNoArgs(t, s_ptr))) return NULL;
    void *p = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    c->bad = PyErr_Occurred() != NULL;
    return p;
}

#define ARGS(n)                                                                       \
    if (na != (n)) {                                                                  \
        PyErr_Format(PyExc_TypeError, "%d arguments, not %zd", (n), na);              \
        return NULL;                                                                  \
    }

static PyObject *rope_fwd(PyObject *self, PyObject *const *a, Py_ssize_t na) {
    ARGS(13)
    Call c = begin("rr_qk_norm_rope_fwd");
    PyObject *dt = NULL;
    const int st = storage(&c, a[0], &dt);
    int64_t q[3] = {-1, -1, -1};
    const Tensor x = tensor(&c, "q", a[0], dt, 3, q, 1);
    int64_t k[3] = {q[0], -1, q[2]}, d[1] = {q[2]}, n[1] = {q[0]}, one[1] = {1}, tab[2] = {-1, -1};
    const Tensor y = tensor(&c, "k", a[1], dt, 3, k, 1);
    if (k[1] < 0) k[1] = 0;
    const Tensor qw = tensor(&c, "q_weight", a[2], dt, 1, d, 0);
    const Tensor kw = tensor(&c, "k_weight", a[3], dt, 1, d, 0);
    const Tensor cos = tensor(&c, "cos", a[4], f32, 2, tab, 0);
    const Tensor sin = tensor(&c, "sin", a[5], f32, 2, tab, 0);
    const Tensor pos = tensor(&c, "positions", a[6], i32, 1, n, 0);
    const Tensor qo = tensor(&c, "q_out", a[7], dt, 3, q, 1);
    const Tensor ko = tensor(&c, "k_out", a[8], dt, 3, k, 1);
    const float eps = (float)number(&c, a[9]);
    const int inter = truth(&c, a[10]);
    const Tensor bad = tensor(&c, "bad_position_count", a[11], i32, 1, one, 0);
    void *s = stream_of(&c, a[12]);
    if (c.bad) return NULL;
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = ((int (*)(void *, void *, void *, void *, void *, void *, void *, void *, void *,
                  int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                  int64_t, int64_t, float, int, void *, int, void *))entry[ROPE_FWD])(
        x.p, y.p, qw.p, kw.p, cos.p, sin.p, pos.p, qo.p, ko.p, q[0], q[1], k[1], q[2], 2 * tab[1],
        tab[0], x.row, y.row, qo.row, ko.row, eps, inter, bad.p, st, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

static PyObject *rope_bwd(PyObject *self, PyObject *const *a, Py_ssize_t na) {
    ARGS(18)
    Call c = begin("rr_qk_norm_rope_bwd");
    PyObject *dt = NULL;
    const int st = storage(&c, a[2], &dt);
    int64_t q[3] = {-1, -1, -1};
    const Tensor x = tensor(&c, "q", a[2], dt, 3, q, 1);
    int64_t k[3] = {q[0], -1, q[2]}, d[1] = {q[2]}, n[1] = {q[0]}, one[1] = {1}, tab[2] = {-1, -1};
    const Tensor y = tensor(&c, "k", a[3], dt, 3, k, 1);
    if (k[1] < 0) k[1] = 0;
    const Tensor gq = tensor(&c, "dq_out", a[0], dt, 3, q, 1);
    const Tensor gk = tensor(&c, "dk_out", a[1], dt, 3, k, 1);
    const Tensor qw = tensor(&c, "q_weight", a[4], dt, 1, d, 0);
    const Tensor kw = tensor(&c, "k_weight", a[5], dt, 1, d, 0);
    const Tensor cos = tensor(&c, "cos", a[6], f32, 2, tab, 0);
    const Tensor sin = tensor(&c, "sin", a[7], f32, 2, tab, 0);
    const Tensor pos = tensor(&c, "positions", a[8], i32, 1, n, 0);
    const Tensor dq = tensor(&c, "dq", a[9], dt, 3, q, 1);
    const Tensor dk = tensor(&c, "dk", a[10], dt, 3, k, 1);
    const Tensor dqw = tensor(&c, "dq_weight", a[11], dt, 1, d, 0);
    const Tensor dkw = tensor(&c, "dk_weight", a[12], dt, 1, d, 0);
    const float eps = (float)number(&c, a[13]);
    const int inter = truth(&c, a[14]);
    size_t bytes;
    void *ws = workspace(&c, a[15], &bytes);
    const Tensor bad = tensor(&c, "bad_position_count", a[16], i32, 1, one, 0);
    void *s = stream_of(&c, a[17]);
    if (c.bad) return NULL;
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = ((int (*)(void *, void *, void *, void *, void *, void *, void *, void *, void *,
                  void *, void *, void *, void *, void *, size_t, int64_t, int64_t,
                  int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                  int64_t, int64_t, float, int, void *, int, void *))entry[ROPE_BWD])(
        gq.p, gk.p, x.p, y.p, qw.p, kw.p, cos.p, sin.p, pos.p, dq.p, dk.p, dqw.p, dkw.p, ws, bytes,
        q[0], q[1], k[1], q[2], 2 * tab[1], tab[0], gq.row, gk.row, x.row, y.row, dq.row, dk.row,
        eps, inter, bad.p, st, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

/* cu_seqlens: [batch + 1]; batch is written. */
static void *bounds(Call *c, PyObject *t, int64_t *batch) {
    int64_t n[1] = {-1};
    const Tensor cu = tensor(c, "cu_seqlens", t, i32, 1, n, 0);
    if (!c->bad && n[0] < 1) {
        PyErr_Format(PyExc_ValueError, "%s: cu_seqlens must hold batch + 1 bounds", c->fn);
        c->bad = 1;
    }
    *batch = n[0] - 1;
    return cu.p;
}

static PyObject *attn_fwd(PyObject *self, PyObject *const *a, Py_ssize_t na) {
    ARGS(8)
    Call c = begin("rr_attention_packed_fwd");
    PyObject *dt = NULL;
    const int st = storage(&c, a[0], &dt);
    int64_t q[3] = {-1, -1, -1}, batch;
    const Tensor x = tensor(&c, "q", a[0], dt, 3, q, 1);
    int64_t k[3] = {q[0], -1, q[2]}, l[2] = {q[1], q[0]};
    const Tensor y = tensor(&c, "k", a[1], dt, 3, k, 1);
    const Tensor z = tensor(&c, "v", a[2], dt, 3, k, 1);
    void *cu = bounds(&c, a[3], &batch);
    const Tensor o = tensor(&c, "o", a[4], dt, 3, q, 1);
    const Tensor lse = tensor(&c, "lse", a[5], f32, 2, l, 0);
    const float scale = (float)number(&c, a[6]);
    void *s = stream_of(&c, a[7]);
    if (c.bad) return NULL;
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = ((int (*)(void *, void *, void *, void *, void *, void *, int64_t, int64_t,
                  int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, float,
                  int, void *))entry[ATTN_FWD])(
        x.p, y.p, z.p, cu, o.p, lse.p, q[0], batch, q[1], k[1], q[2], x.row, y.row, z.row, o.row,
        scale, st, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

static PyObject *attn_bwd(PyObject *self, PyObject *const *a, Py_ssize_t na) {
    ARGS(13)
    Call c = begin("rr_attention_packed_bwd");
    PyObject *dt = NULL;
    const int st = storage(&c, a[1], &dt);
    int64_t q[3] = {-1, -1, -1}, batch;
    const Tensor x = tensor(&c, "q", a[1], dt, 3, q, 1);
    int64_t k[3] = {q[0], -1, q[2]}, l[2] = {q[1], q[0]};
    const Tensor y = tensor(&c, "k", a[2], dt, 3, k, 1);
    const Tensor z = tensor(&c, "v", a[3], dt, 3, k, 1);
    const Tensor g = tensor(&c, "dout", a[0], dt, 3, q, 1);
    const Tensor o = tensor(&c, "o", a[4], dt, 3, q, 1);
    const Tensor lse = tensor(&c, "lse", a[5], f32, 2, l, 0);
    void *cu = bounds(&c, a[6], &batch);
    const Tensor dq = tensor(&c, "dq", a[7], dt, 3, q, 1);
    const Tensor dk = tensor(&c, "dk", a[8], dt, 3, k, 1);
    const Tensor dv = tensor(&c, "dv", a[9], dt, 3, k, 1);
    const float scale = (float)number(&c, a[10]);
    size_t bytes;
    void *ws = workspace(&c, a[11], &bytes);
    void *s = stream_of(&c, a[12]);
    if (c.bad) return NULL;
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = ((int (*)(void *, void *, void *, void *, void *, void *, void *, void *, void *,
                  void *, void *, size_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                  int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                  float, int, void *))entry[ATTN_BWD])(
        g.p, x.p, y.p, z.p, o.p, lse.p, cu, dq.p, dk.p, dv.p, ws, bytes, q[0], batch, q[1], k[1],
        q[2], g.row, x.row, y.row, z.row, o.row, dq.row, dk.row, dv.row, scale, st, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

static PyObject *logprob_fwd(PyObject *self, PyObject *const *a, Py_ssize_t na) {
    ARGS(13)
    Call c = begin("rr_token_logprob_fwd");
    PyObject *dt = NULL;
    const int st = storage(&c, a[0], &dt);
    int64_t x[2] = {-1, -1};
    const Tensor lg = tensor(&c, "logits", a[0], dt, 2, x, 1);
    int64_t n[1] = {x[0]}, top[2] = {x[0], -1}, one[1] = {1};
    const Tensor t = tensor(&c, "tokens", a[1], i32, 1, n, 0);
    const Tensor lp = tensor(&c, "logprob", a[2], f32, 1, n, 0);
    const Tensor en = tensor(&c, "entropy", a[3], f32, 1, n, 0);
    const Tensor rm = tensor(&c, "row_max", a[4], f32, 1, n, 0);
    const Tensor ls = tensor(&c, "log_sum", a[5], f32, 1, n, 0);
    const Tensor rk = tensor(&c, "rank", a[6], i32, 1, n, 0);
    const Tensor ti = tensor(&c, "top_index", a[7], i32, 2, top, 0);
    const Tensor tl = tensor(&c, "top_logprob", a[8], f32, 2, top, 0);
    if (!c.bad && (a[7] == Py_None) != (a[8] == Py_None)) {
        PyErr_Format(PyExc_ValueError, "%s: top_index and top_logprob: both, or neither", c.fn);
        return NULL;
    }
    const float T = (float)number(&c, a[9]);
    const int32_t ignore = whole(&c, "ignore_index", a[10]);
    const Tensor bad = tensor(&c, "bad_token_count", a[11], i32, 1, one, 0);
    void *s = stream_of(&c, a[12]);
    if (c.bad) return NULL;
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = ((int (*)(void *, void *, void *, void *, void *, void *, void *, void *, void *,
                  int64_t, int64_t, int64_t, int64_t, float, int32_t, void *, int,
                  void *))entry[LOGP_FWD])(
        lg.p, t.p, lp.p, en.p, rm.p, ls.p, rk.p, ti.p, tl.p, x[0], x[1], lg.row,
        top[1] < 0 ? 0 : top[1], T, ignore, bad.p, st, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

static PyObject *logprob_bwd(PyObject *self, PyObject *const *a, Py_ssize_t na) {
    ARGS(11)
    Call c = begin("rr_token_logprob_bwd");
    PyObject *dt = NULL;
    const int st = storage(&c, a[0], &dt);
    int64_t x[2] = {-1, -1};
    const Tensor lg = tensor(&c, "logits", a[0], dt, 2, x, 1);
    int64_t n[1] = {x[0]};
    const Tensor t = tensor(&c, "tokens", a[1], i32, 1, n, 0);
    const Tensor rm = tensor(&c, "row_max", a[2], f32, 1, n, 0);
    const Tensor ls = tensor(&c, "log_sum", a[3], f32, 1, n, 0);
    const Tensor g = tensor(&c, "grad_logprob", a[4], f32, 1, n, 0);
    const Tensor dl = tensor(&c, "dlogits", a[5], dt, 2, x, 1);
    const Tensor en = tensor(&c, "entropy", a[6], f32, 1, n, 0);
    const Tensor h = tensor(&c, "grad_entropy", a[7], f32, 1, n, 0);
    const float T = (float)number(&c, a[8]);
    const int32_t ignore = whole(&c, "ignore_index", a[9]);
    void *s = stream_of(&c, a[10]);
    if (c.bad) return NULL;
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = ((int (*)(void *, void *, void *, void *, void *, void *, void *, void *, int64_t,
                  int64_t, int64_t, int64_t, float, int32_t, int, void *))entry[LOGP_BWD])(
        lg.p, t.p, rm.p, ls.p, en.p, g.p, h.p, dl.p, x[0], x[1], lg.row, dl.row, T, ignore, st, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

/* setup(float32, bfloat16, int32, get_device, raw_stream, addresses in the order of `entry`) */
static PyObject *setup(PyObject *self, PyObject *const *a, Py_ssize_t na) {
    ARGS(6)
    if (!PyTuple_Check(a[5]) || PyTuple_GET_SIZE(a[5]) != ENTRIES) {
        PyErr_SetString(PyExc_TypeError, "addresses: a tuple of one for each entry point");
        return NULL;
    }
    for (int i = 0; i < ENTRIES; ++i) {
        entry[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[5], i));
        if (PyErr_Occurred()) return NULL;
    }
    PyObject **keep[] = {&f32, &bf16, &i32, &get_device, &raw_stream};
    for (int i = 0; i < 5; ++i) {
        Py_INCREF(a[i]);
        Py_XSETREF(*keep[i], a[i]);
    }
    Py_RETURN_NONE;
}

#define M(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {M(setup),    M(rope_fwd),    M(rope_bwd),    M(attn_fwd),
                                M(attn_bwd), M(logprob_fwd), M(logprob_bwd), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__call(void) {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_contig = PyUnicode_InternFromString("is_contiguous");
    s_ptr = PyUnicode_InternFromString("data_ptr");
    s_dev = PyUnicode_InternFromString("get_device");
    return PyModule_Create(&module);
}
