/*
 * binding.c -- the short way from Python into the serving calls.
 *
 * A decode step's kernels take a few microseconds, less than Python takes to
 * look at six tensors and ctypes to pass sixteen arguments.  These functions
 * do both in C: they look at the tensors through the same methods that the
 * Python side calls (dtype, shape, get_device, is_contiguous, stride,
 * data_ptr), and where every one is as the call wants it, make the call.
 * Where anything is not -- another type, another device, a shape that does not
 * fit -- they return None without having called anything, and the Python side
 * goes through its own checks, which say what is wrong.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/mercury_attn.h"

typedef long long ll;

/* what init() was given */
static PyObject *g_bf16, *g_fp32, *g_int32, *g_device, *g_stream;
static int (*g_rope)(const void *, const ll *, const int *, ll, ll, int, int, int, int, int, const mercury_rope_plan *, int,
                     void *, const ll *, void *);
static int (*g_append)(const void *, const ll *, const void *, const ll *, int, int, const mercury_paged_cache *, const int *,
                       const int *, const mercury_rope_plan *, const void *, const ll *, int, void *, const ll *, void *);
static int (*g_attn)(const void *, const ll *, const mercury_paged_cache *, const int *, const int *, int, int, int, int,
                     float *, float *, void *);
static int (*g_attn_bf16)(const void *, const ll *, const mercury_paged_cache *, const int *, const int *, int, int, int, int,
                          void *, float *, void *);
static PyObject *s_dtype, *s_shape, *s_get_device, *s_is_contiguous, *s_stride, *s_data_ptr;

/* A tensor as a call sees it. */
typedef struct {
    void *p;
    Py_ssize_t n[4];  /* shape */
    ll st[3];
    const ll *strides;  /* st, or NULL where contiguous */
} View;

static int is_true_call(PyObject *t, PyObject *name)
{
    PyObject *r = PyObject_CallMethodNoArgs(t, name);
    const int yes = r ? PyObject_IsTrue(r) : -1;
    Py_XDECREF(r);
    return yes;
}

/* 1 where t is a tensor of this dtype on device dev with `dim` axes, its last
 * one contiguous if `strided`, all of it if not; 0 otherwise (no exception is
 * left behind). */
static int look(PyObject *t, PyObject *dtype, long dev, int dim, int strided, View *v)
{
    PyObject *a = PyObject_GetAttr(t, s_dtype), *r;
    int ok = a == dtype, contiguous;
    Py_XDECREF(a);
    if (!ok)
        goto no;
    r = PyObject_CallMethodNoArgs(t, s_get_device);
    ok = r && PyLong_AsLong(r) == dev;
    Py_XDECREF(r);
    if (!ok || PyErr_Occurred())
        goto no;
    r = PyObject_GetAttr(t, s_shape);
    ok = r && PyTuple_Check(r) && PyTuple_GET_SIZE(r) == dim;
    if (ok)
        for (int i = 0; i < dim; ++i)
            v->n[i] = PyLong_AsSsize_t(PyTuple_GET_ITEM(r, i));
    Py_XDECREF(r);
    if (!ok || PyErr_Occurred())
        goto no;
    v->strides = NULL;
    contiguous = is_true_call(t, s_is_contiguous);
    if (contiguous != 1) {
        if (contiguous < 0 || !strided)
            goto no;
        r = PyObject_CallMethodNoArgs(t, s_stride);
        ok = r && PyTuple_Check(r) && PyTuple_GET_SIZE(r) == dim && dim == 4 &&
             (v->n[3] == 1 || PyLong_AsLongLong(PyTuple_GET_ITEM(r, 3)) == 1);
        if (ok)
            for (int i = 0; i < 3; ++i)
                v->st[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(r, i));
        Py_XDECREF(r);
        if (!ok || PyErr_Occurred())
            goto no;
        v->strides = v->st;
    }
    r = PyObject_CallMethodNoArgs(t, s_data_ptr);
    v->p = r ? PyLong_AsVoidPtr(r) : NULL;
    Py_XDECREF(r);
    if (PyErr_Occurred())
        goto no;
    return 1;
no:
    PyErr_Clear();
    return 0;
}

/* The current device is dev; its current stream. */
static int on_device(long dev, void **stream)
{
    PyObject *r = PyObject_CallNoArgs(g_device), *d;
    int ok = r && PyLong_AsLong(r) == dev;
    Py_XDECREF(r);
    if (ok) {
        d = PyLong_FromLong(dev);
        r = d ? PyObject_CallOneArg(g_stream, d) : NULL;
        Py_XDECREF(d);
        ok = r != NULL;
        if (ok)
            *stream = PyLong_AsVoidPtr(r);
        Py_XDECREF(r);
    }
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return 0;
    }
    return ok;
}

static int fits(const View *v, int i) { return v->n[i] >= 0 && v->n[i] <= 0x7fffffff; }

/* A [B] int32 tensor, or None (NULL). */
static int look_lens(PyObject *t, long dev, Py_ssize_t B, const int **p)
{
    View v;
    *p = NULL;
    if (t == Py_None)
        return 1;
    if (!look(t, g_int32, dev, 1, 0, &v) || v.n[0] != B)
        return 0;
    *p = (const int *)v.p;
    return 1;
}

/* rope(x, plan address, positions or None, start, inverse, out) -> status or None */
static PyObject *py_rope(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    View x, o, pos;
    void *stream, *plan;
    const int *pp = NULL;
    ll row = 0, start;
    long dev;
    int rc, inverse, elem;
    PyObject *r, *dtype;
    if (n != 6)
        Py_RETURN_NONE;
    plan = PyLong_AsVoidPtr(a[1]);
    start = PyErr_Occurred() ? 0 : PyLong_AsLongLong(a[3]);
    inverse = PyErr_Occurred() ? 0 : PyObject_IsTrue(a[4]);
    r = PyErr_Occurred() ? NULL : PyObject_CallMethodNoArgs(a[0], s_get_device);
    dev = r ? PyLong_AsLong(r) : -1;
    Py_XDECREF(r);
    dtype = dev < 0 ? NULL : PyObject_GetAttr(a[0], s_dtype);
    elem = dtype == g_bf16 ? MERCURY_ELEM_BF16 : MERCURY_ELEM_FP32;
    Py_XDECREF(dtype);
    if (dev < 0 || PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    dtype = elem == MERCURY_ELEM_BF16 ? g_bf16 : g_fp32;
    if (!look(a[0], dtype, dev, 4, 1, &x) || !look(a[5], dtype, dev, 4, 1, &o))
        Py_RETURN_NONE;
    for (int i = 0; i < 4; ++i)
        if (!fits(&x, i) || x.n[i] != o.n[i])
            Py_RETURN_NONE;
    if (a[2] != Py_None) {
        if (look(a[2], g_int32, dev, 2, 0, &pos) && pos.n[0] == x.n[0] && pos.n[1] == x.n[2])
            row = x.n[2];
        else if (!look(a[2], g_int32, dev, 1, 0, &pos) || pos.n[0] != x.n[2])
            Py_RETURN_NONE;
        pp = (const int *)pos.p;
    }
    if (!on_device(dev, &stream))
        Py_RETURN_NONE;
    Py_BEGIN_ALLOW_THREADS
    rc = g_rope(x.p, x.strides, pp, row, start, (int)x.n[0], (int)x.n[1], (int)x.n[2], (int)x.n[3], elem,
                (const mercury_rope_plan *)plan, inverse, o.p, o.strides, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* append(cache address, device, k, v, past_lens, new_lens or None, plan address or 0, q or None, q_out or None)
 * -> status or None */
static PyObject *py_append(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    View k, v, q = {0}, o = {0};
    const mercury_paged_cache *c;
    const int *past, *fresh;
    void *stream, *plan;
    long dev;
    int rc;
    if (n != 9)
        Py_RETURN_NONE;
    c = (const mercury_paged_cache *)PyLong_AsVoidPtr(a[0]);
    dev = PyErr_Occurred() ? -1 : PyLong_AsLong(a[1]);
    plan = PyErr_Occurred() ? NULL : PyLong_AsVoidPtr(a[6]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    if (!look(a[2], g_bf16, dev, 4, 1, &k) || !look(a[3], g_bf16, dev, 4, 1, &v) || k.n[0] != c->B || k.n[1] != c->Hkv ||
        k.n[3] != c->d || !fits(&k, 2))
        Py_RETURN_NONE;
    for (int i = 0; i < 4; ++i)
        if (k.n[i] != v.n[i])
            Py_RETURN_NONE;
    if (a[4] == Py_None || !look_lens(a[4], dev, c->B, &past) || !look_lens(a[5], dev, c->B, &fresh))
        Py_RETURN_NONE;
    if (a[7] != Py_None) {
        if (!look(a[7], g_bf16, dev, 4, 1, &q) || !look(a[8], g_bf16, dev, 4, 1, &o) || q.n[0] != k.n[0] || q.n[2] != k.n[2] ||
            q.n[3] != k.n[3] || !fits(&q, 1))
            Py_RETURN_NONE;
        for (int i = 0; i < 4; ++i)
            if (q.n[i] != o.n[i])
                Py_RETURN_NONE;
    } else if (a[8] != Py_None) {
        Py_RETURN_NONE;
    }
    if (!on_device(dev, &stream))
        Py_RETURN_NONE;
    Py_BEGIN_ALLOW_THREADS
    rc = g_append(k.p, k.strides, v.p, v.strides, c->B, (int)k.n[2], c, past, fresh, (const mercury_rope_plan *)plan, q.p,
                  q.strides, (int)q.n[1], o.p, o.strides, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* attn(bf16 output?, q, cache address, device, seq_lens, new_lens or None, causal, out, lse) -> status or None */
static PyObject *py_attn(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    View q, o, l;
    const mercury_paged_cache *c;
    const int *lens, *fresh;
    void *stream;
    long dev;
    int rc, bf16, causal;
    if (n != 9)
        Py_RETURN_NONE;
    bf16 = PyObject_IsTrue(a[0]);
    c = PyErr_Occurred() ? NULL : (const mercury_paged_cache *)PyLong_AsVoidPtr(a[2]);
    dev = PyErr_Occurred() ? -1 : PyLong_AsLong(a[3]);
    causal = PyErr_Occurred() ? 0 : PyObject_IsTrue(a[6]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    if (!look(a[1], g_bf16, dev, 4, 1, &q) || q.n[0] != c->B || q.n[3] != c->d || !fits(&q, 1) || !fits(&q, 2))
        Py_RETURN_NONE;
    if (a[4] == Py_None || !look_lens(a[4], dev, c->B, &lens) || !look_lens(a[5], dev, c->B, &fresh))
        Py_RETURN_NONE;
    if (!look(a[7], bf16 ? g_bf16 : g_fp32, dev, 4, 0, &o) || !look(a[8], g_fp32, dev, 3, 0, &l))
        Py_RETURN_NONE;
    for (int i = 0; i < 4; ++i)
        if (q.n[i] != o.n[i] || (i < 3 && q.n[i] != l.n[i]))
            Py_RETURN_NONE;
    if (!on_device(dev, &stream))
        Py_RETURN_NONE;
    Py_BEGIN_ALLOW_THREADS
    rc = bf16 ? g_attn_bf16(q.p, q.strides, c, lens, fresh, c->B, (int)q.n[1], (int)q.n[2], causal, o.p, (float *)l.p, stream)
              : g_attn(q.p, q.strides, c, lens, fresh, c->B, (int)q.n[1], (int)q.n[2], causal, (float *)o.p, (float *)l.p, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* init(bf16, fp32, int32, current_device, current_stream, addresses of the four library functions) */
static PyObject *py_init(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    if (n != 9) {
        PyErr_SetString(PyExc_TypeError, "init takes nine arguments");
        return NULL;
    }
    g_bf16 = Py_NewRef(a[0]);
    g_fp32 = Py_NewRef(a[1]);
    g_int32 = Py_NewRef(a[2]);
    g_device = Py_NewRef(a[3]);
    g_stream = Py_NewRef(a[4]);
    *(void **)&g_rope = PyLong_AsVoidPtr(a[5]);
    *(void **)&g_append = PyLong_AsVoidPtr(a[6]);
    *(void **)&g_attn = PyLong_AsVoidPtr(a[7]);
    *(void **)&g_attn_bf16 = PyLong_AsVoidPtr(a[8]);
    if (PyErr_Occurred())
        return NULL;
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))py_init, METH_FASTCALL, "torch names and library functions"},
    {"rope", (PyCFunction)(void (*)(void))py_rope, METH_FASTCALL, "mercury_rope, or None"},
    {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, "mercury_kv_append, or None"},
    {"attn", (PyCFunction)(void (*)(void))py_attn, METH_FASTCALL, "mercury_attn_paged, or None"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "mercury_binding", "the serving calls, from tensors", -1, methods};

PyMODINIT_FUNC PyInit_mercury_binding(void)
{
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    if (!s_dtype || !s_shape || !s_get_device || !s_is_contiguous || !s_stride || !s_data_ptr)
        return NULL;
    return PyModule_Create(&module);
}
