/* The tensor-level calls of the 4-bit cache, of attention over it and of key weights:
 * checks of the tensors, allocation of outputs, and the call into libfa.so, as a
 * CPython extension.  A decode step's kernels take a few microseconds; the same
 * steps in Python took 10 to 20 more (a tensor attribute costs 60 to 150 ns,
 * marshalling a dozen arguments through ctypes 3 us).  The library is not linked:
 * _binding.py hands over the addresses of its functions, so there is one copy of
 * it in the process.  No arithmetic here; every refusal raises. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>
#include <stdint.h>

#include "fa.h"

static PyObject *s_dtype, *s_shape, *s_device, *s_contig, *s_ptr;                 /* attribute names */
static PyObject *t_u8, *t_bf16, *t_f32, *t_i32, *f_empty, *f_stream, *f_current, *c_error;
static PyObject *kw_empty, *a_keep_refs;

static int (*p_append)(const fa_kv4_cache *, const void *, const void *, const float *, const int32_t *, const int32_t *,
                       const int32_t *, int64_t, int64_t, int64_t, void *);
static int (*p_read)(const fa_kv4_cache *, const int32_t *, const int32_t *, const int32_t *, int64_t, int64_t, int64_t,
                     void *, void *, void *);
static int (*p_fwd)(const void *, const fa_kv4_cache *, const int32_t *, const int32_t *, void *, float *, int64_t, int64_t,
                    int64_t, int64_t, float, int, void *, int64_t, void *);
static int64_t (*p_fwd_bytes)(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int);
static int (*p_evict)(const fa_kv4_cache *, const int32_t *, const int32_t *, int64_t, const fa_kv4_cache *, const int32_t *,
                      int64_t, int64_t, int64_t, int64_t, int32_t *, int32_t *, void *);
static int (*p_weights)(const void *, const void *, const float *, float *, int64_t, int64_t, int64_t, int64_t, int64_t,
                        float, int, int64_t, void *);

typedef struct {
    int nd;
    int64_t dim[4];
    void *ptr;
    long dev;
} Tensor;

static long call_long(PyObject *o, PyObject *name)
{
    PyObject *r = PyObject_CallMethodNoArgs(o, name);
    if (r == NULL) return -1;
    const long v = PyLong_AsLong(r);
    Py_DECREF(r);
    return v;
}

/* A contiguous tensor of `dtype` and `nd` dimensions on CUDA device `dev` (any where dev < 0); 0, or -1 with `what` raised. */
static int get_tensor(PyObject *o, PyObject *dtype, int nd, long dev, Tensor *t, const char *what)
{
    PyObject *x = PyObject_GetAttr(o, s_dtype);
    if (x == NULL) return -1;
    int good = x == dtype;
    Py_DECREF(x);
    t->dev = call_long(o, s_device);
    if (t->dev == -1 && PyErr_Occurred()) return -1;
    good = good && t->dev >= 0 && (dev < 0 || t->dev == dev);
    if (good) {
        x = PyObject_CallMethodNoArgs(o, s_contig);
        if (x == NULL) return -1;
        good = x == Py_True;
        Py_DECREF(x);
    }
    if (good) {
        x = PyObject_GetAttr(o, s_shape);
        if (x == NULL) return -1;
        good = PyTuple_Check(x) && PyTuple_GET_SIZE(x) == nd;
        for (int i = 0; good && i < nd; ++i) t->dim[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(x, i));
        Py_DECREF(x);
        if (PyErr_Occurred()) return -1;
    }
    if (!good) {
        PyErr_Format(PyExc_ValueError, "%s", what);
        return -1;
    }
    t->nd = nd;
    x = PyObject_CallMethodNoArgs(o, s_ptr);
    if (x == NULL) return -1;
    t->ptr = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(x);
    Py_DECREF(x);
    return PyErr_Occurred() ? -1 : 0;
}

static int refuse(const char *what)
{
    PyErr_SetString(PyExc_ValueError, what);
    return -1;
}

/* A KV4Cache as the library's struct; *dev is its device. */
static int get_cache(PyObject *o, fa_kv4_cache *c, long *dev)
{
    static const char *const codes = "k and v of a cache must be contiguous uint8 tensors [n_pages, Hkv, page_size, d/2] on one CUDA device";
    static const char *const scales = "k_scale and v_scale of a cache must be contiguous uint8 tensors [n_pages, Hkv, page_size, d/32] and "
                                      "[n_pages, Hkv, page_size] on its device";
    static const char *const weights = "weights of a cache must be a contiguous fp32 tensor [n_pages, Hkv, page_size] on its device";
    Tensor k, t;
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5) return refuse("the cache must be a KV4Cache");
    if (get_tensor(PyTuple_GET_ITEM(o, 0), t_u8, 4, -1, &k, codes)) return -1;
    c->k = k.ptr;
    c->n_pages = k.dim[0];
    c->Hkv = k.dim[1];
    c->page_size = k.dim[2];
    c->d = 2 * k.dim[3];
    *dev = k.dev;
    if (get_tensor(PyTuple_GET_ITEM(o, 1), t_u8, 4, k.dev, &t, codes)) return -1;
    for (int i = 0; i < 4; ++i)
        if (t.dim[i] != k.dim[i]) return refuse(codes);
    c->v = t.ptr;
    if (get_tensor(PyTuple_GET_ITEM(o, 2), t_u8, 4, k.dev, &t, scales)) return -1;
    if (t.dim[0] != k.dim[0] || t.dim[1] != k.dim[1] || t.dim[2] != k.dim[2] || t.dim[3] != k.dim[3] / 16) return refuse(scales);
    c->k_scale = t.ptr;
    if (get_tensor(PyTuple_GET_ITEM(o, 3), t_u8, 3, k.dev, &t, scales)) return -1;
    if (t.dim[0] != k.dim[0] || t.dim[1] != k.dim[1] || t.dim[2] != k.dim[2]) return refuse(scales);
    c->v_scale = t.ptr;
    c->weights = NULL;
    if (PyTuple_GET_ITEM(o, 4) != Py_None) {
        if (get_tensor(PyTuple_GET_ITEM(o, 4), t_f32, 3, k.dev, &t, weights)) return -1;
        if (t.dim[0] != k.dim[0] || t.dim[1] != k.dim[1] || t.dim[2] != k.dim[2]) return refuse(weights);
        c->weights = (float *)t.ptr;
    }
    return 0;
}

/* int32 index tensors: [B], or [B, columns]; B < 0 is set. */
static int get_index(PyObject *o, int nd, int64_t *B, long dev, Tensor *t, const char *what)
{
    if (get_tensor(o, t_i32, nd, dev, t, what)) return -1;
    if (*B < 0) *B = t->dim[0];
    return t->dim[0] == *B ? 0 : refuse(what);
}
#define LENS "lens must be a contiguous int32 tensor [B] on the cache's device"
#define TABLE "page_table must be a contiguous int32 tensor [B, pages] on the cache's device"

/* The current stream of `dev`, and whether that is the current device (else the caller makes it so and calls again). */
static int get_stream(long dev, void **s, int *here)
{
    PyObject *r = PyObject_CallNoArgs(f_current);
    if (r == NULL) return -1;
    *here = PyLong_AsLong(r) == dev;
    Py_DECREF(r);
    PyObject *d = PyLong_FromLong(dev);
    if (d == NULL) return -1;
    r = PyObject_CallOneArg(f_stream, d);
    Py_DECREF(d);
    if (r == NULL) return -1;
    *s = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(r);
    Py_DECREF(r);
    return PyErr_Occurred() ? -1 : 0;
}

/* torch.empty(dims, dtype=dtype, device=dev), and its address. */
static PyObject *empty(int nd, const int64_t *dim, PyObject *dtype, long dev, void **ptr)
{
    PyObject *shape = PyTuple_New(nd), *d = PyLong_FromLong(dev), *r = NULL;
    for (int i = 0; shape != NULL && i < nd; ++i) {
        PyObject *n = PyLong_FromLongLong(dim[i]);
        if (n == NULL) Py_CLEAR(shape);
        else PyTuple_SET_ITEM(shape, i, n);
    }
    if (shape != NULL && d != NULL) {
        PyObject *args[4] = {NULL, shape, dtype, d};
        r = PyObject_Vectorcall(f_empty, args + 1, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, kw_empty);
    }
    Py_XDECREF(shape);
    Py_XDECREF(d);
    if (r == NULL) return NULL;
    PyObject *p = PyObject_CallMethodNoArgs(r, s_ptr);
    *ptr = p == NULL ? NULL : (void *)(uintptr_t)PyLong_AsUnsignedLongLong(p);
    Py_XDECREF(p);
    if (PyErr_Occurred()) Py_CLEAR(r);
    return r;
}

static PyObject *fail(int status, const char *where)
{
    PyObject *e = PyObject_CallFunction(c_error, "is", status, where);
    if (e != NULL) {
        PyErr_SetObject(c_error, e);
        Py_DECREF(e);
    }
    return NULL;
}

static int nargs_is(Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return 1;
    PyErr_Format(PyExc_TypeError, "%zd arguments are needed, not %zd", want, n);
    return 0;
}

/* (cache, k, v, lens, page_table, n_new, weights) */
static PyObject *kv4_append(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    fa_kv4_cache c;
    Tensor k, v, lens, table, extra;
    long dev;
    void *s, *p_new = NULL, *p_w = NULL;
    int here, st;
    static const char *const kv = "k and v must be contiguous bf16 tensors [B, Hkv, S, d], with the cache's Hkv and d, on its device";
    static const char *const w = "weights must be a contiguous fp32 tensor [B, Hkv, S] on the cache's device";
    if (!nargs_is(n, 7) || get_cache(a[0], &c, &dev)) return NULL;
    if (get_tensor(a[1], t_bf16, 4, dev, &k, kv) || get_tensor(a[2], t_bf16, 4, dev, &v, kv)) return NULL;
    for (int i = 0; i < 4; ++i)
        if (k.dim[i] != v.dim[i]) return refuse(kv), NULL;
    if (k.dim[1] != c.Hkv || k.dim[3] != c.d) return refuse(kv), NULL;
    int64_t B = k.dim[0];
    if (get_index(a[3], 1, &B, dev, &lens, LENS) || get_index(a[4], 2, &B, dev, &table, TABLE)) return NULL;
    if (a[5] != Py_None) {
        if (get_index(a[5], 1, &B, dev, &extra, "n_new must be a contiguous int32 tensor [B] on the cache's device")) return NULL;
        p_new = extra.ptr;
    }
    if (a[6] != Py_None) {
        if (get_tensor(a[6], t_f32, 3, dev, &extra, w)) return NULL;
        if (extra.dim[0] != B || extra.dim[1] != c.Hkv || extra.dim[2] != k.dim[2]) return refuse(w), NULL;
        if (c.weights == NULL) return refuse("the cache holds no weights"), NULL;
        p_w = extra.ptr;
    }
    if (get_stream(dev, &s, &here)) return NULL;
    if (!here) Py_RETURN_NOTIMPLEMENTED;
    Py_BEGIN_ALLOW_THREADS
    st = p_append(&c, k.ptr, v.ptr, (const float *)p_w, (const int32_t *)p_new, (const int32_t *)lens.ptr,
                  (const int32_t *)table.ptr, B, k.dim[2], table.dim[1], s);
    Py_END_ALLOW_THREADS
    if (st != FA_OK) return fail(st, "fa_kv4_append");
    Py_RETURN_NONE;
}

/* (cache, lens, page_table, count, first) -> (k, v) */
static PyObject *kv4_read(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    fa_kv4_cache c;
    Tensor lens, table, first;
    long dev;
    void *s, *pk, *pv, *pf = NULL;
    int here, st;
    int64_t B = -1;
    if (!nargs_is(n, 5) || get_cache(a[0], &c, &dev)) return NULL;
    if (get_index(a[1], 1, &B, dev, &lens, LENS) || get_index(a[2], 2, &B, dev, &table, TABLE)) return NULL;
    const int64_t count = PyLong_AsLongLong(a[3]);
    if (count == -1 && PyErr_Occurred()) return NULL;
    if (count < 1) return refuse("count must be at least 1"), NULL;
    if (a[4] != Py_None) {
        if (get_index(a[4], 1, &B, dev, &first, "first must be a contiguous int32 tensor [B] on the cache's device")) return NULL;
        pf = first.ptr;
    }
    if (get_stream(dev, &s, &here)) return NULL;
    if (!here) Py_RETURN_NOTIMPLEMENTED;
    const int64_t dim[4] = {B, c.Hkv, count, c.d};
    PyObject *k = empty(4, dim, t_bf16, dev, &pk);
    PyObject *v = k == NULL ? NULL : empty(4, dim, t_bf16, dev, &pv);
    if (v == NULL) {
        Py_XDECREF(k);
        return NULL;
    }
    Py_BEGIN_ALLOW_THREADS
    st = p_read(&c, (const int32_t *)pf, (const int32_t *)lens.ptr, (const int32_t *)table.ptr, B, table.dim[1], count, pk, pv, s);
    Py_END_ALLOW_THREADS
    PyObject *r = st == FA_OK ? PyTuple_Pack(2, k, v) : fail(st, "fa_kv4_read");
    Py_DECREF(k);
    Py_DECREF(v);
    return r;
}

/* scale argument: None is fp32 1 / sqrt(d) */
static int get_scale(PyObject *o, int64_t d, float *scale)
{
    const double x = o == Py_None ? 1.0 / sqrt((double)d) : PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) return -1;
    *scale = (float)x;
    return 0;
}

/* (q, cache, lens, page_table, scale, accumulate, workspace) -> (o, lse) */
static PyObject *forward_kv4(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    fa_kv4_cache c;
    Tensor q, lens, table, ws;
    long dev;
    float scale;
    void *s, *po, *pl, *pw = NULL;
    int here, st;
    static const char *const what = "q must be a contiguous bf16 tensor [B, H, n_q, d], with the cache's d and H a multiple of its key heads, on its device";
    if (!nargs_is(n, 7) || get_cache(a[1], &c, &dev)) return NULL;
    if (get_tensor(a[0], t_bf16, 4, dev, &q, what)) return NULL;
    if (q.dim[3] != c.d || c.Hkv < 1 || q.dim[1] % c.Hkv != 0) return refuse(what), NULL;
    int64_t B = q.dim[0], size;
    if (get_index(a[2], 1, &B, dev, &lens, LENS) || get_index(a[3], 2, &B, dev, &table, TABLE)) return NULL;
    const int acc = PyObject_IsTrue(a[5]);
    if (acc < 0 || get_scale(a[4], c.d, &scale)) return NULL;
    if (acc && c.weights == NULL) return refuse("the cache holds no weights"), NULL;
    const int64_t need = p_fwd_bytes(B, q.dim[1], c.Hkv, q.dim[2], c.d, table.dim[1] * c.page_size, acc);
    if (need < 0) return fail(c.d == 64 || c.d == 128 ? FA_ERR_INVALID_ARG : FA_ERR_UNSUPPORTED, "fa_fwd_kv4_workspace_bytes");
    if (get_stream(dev, &s, &here)) return NULL;
    if (!here) Py_RETURN_NOTIMPLEMENTED;
    PyObject *own = NULL, *o = NULL, *lse = NULL, *r = NULL;
    if (a[6] == Py_None) {
        own = empty(1, &need, t_u8, dev, &pw);
        if (own == NULL) return NULL;
        size = need;
    } else {
        if (get_tensor(a[6], t_u8, 1, dev, &ws, "workspace must be a contiguous uint8 tensor [bytes] on the cache's device")) return NULL;
        pw = ws.ptr;
        size = ws.dim[0];
    }
    o = empty(4, q.dim, t_bf16, dev, &po);
    lse = o == NULL ? NULL : empty(3, q.dim, t_f32, dev, &pl);
    if (lse != NULL) {
        Py_BEGIN_ALLOW_THREADS
        st = p_fwd(q.ptr, &c, (const int32_t *)lens.ptr, (const int32_t *)table.ptr, po, (float *)pl, B, q.dim[1], q.dim[2],
                   table.dim[1], scale, acc, pw, size, s);
        Py_END_ALLOW_THREADS
        r = st == FA_OK ? PyTuple_Pack(2, o, lse) : fail(st, "fa_fwd_kv4");
    }
    Py_XDECREF(own);
    Py_XDECREF(o);
    Py_XDECREF(lse);
    return r;
}

/* (cache, lens, page_table, to, to_table, keep, recent) -> (kept, new_lens) */
static PyObject *kv4_evict(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    fa_kv4_cache c, t;
    Tensor lens, table, to_table;
    long dev, dev_to;
    void *s, *pk, *pn;
    int here, st;
    int64_t B = -1;
    if (!nargs_is(n, 7) || get_cache(a[0], &c, &dev)) return NULL;
    if (a[3] == a[0]) {
        t = c;
    } else {
        if (get_cache(a[3], &t, &dev_to)) return NULL;
        if (dev_to != dev || t.Hkv != c.Hkv || t.page_size != c.page_size || t.d != c.d)
            return refuse("both caches must have the same key heads, page size, d and device"), NULL;
    }
    if (c.weights == NULL || t.weights == NULL) return refuse("eviction needs the weights of both caches"), NULL;
    if (get_index(a[1], 1, &B, dev, &lens, LENS) || get_index(a[2], 2, &B, dev, &table, TABLE) ||
        get_index(a[4], 2, &B, dev, &to_table, "to_table must be a contiguous int32 tensor [B, pages] on the cache's device"))
        return NULL;
    const int64_t keep = PyLong_AsLongLong(a[5]), recent = PyLong_AsLongLong(a[6]);
    if (PyErr_Occurred()) return NULL;
    if (keep < 1 || recent < 0 || recent > keep || keep > to_table.dim[1] * c.page_size)
        return refuse("need 1 <= keep <= the tokens of to_table's pages, and 0 <= recent <= keep"), NULL;
    if (get_stream(dev, &s, &here)) return NULL;
    if (!here) Py_RETURN_NOTIMPLEMENTED;
    const int64_t dim[3] = {B, c.Hkv, keep};
    PyObject *kept = empty(3, dim, t_i32, dev, &pk), *now = kept == NULL ? NULL : empty(1, &B, t_i32, dev, &pn), *r = NULL;
    if (now != NULL) {
        Py_BEGIN_ALLOW_THREADS
        st = p_evict(&c, (const int32_t *)lens.ptr, (const int32_t *)table.ptr, table.dim[1], &t, (const int32_t *)to_table.ptr,
                     to_table.dim[1], B, keep, recent, (int32_t *)pk, (int32_t *)pn, s);
        Py_END_ALLOW_THREADS
        r = st == FA_OK ? PyTuple_Pack(2, kept, now) : fail(st, "fa_kv4_evict");
    }
    Py_XDECREF(kept);
    Py_XDECREF(now);
    return r;
}

/* (q, k, lse, scale, causal, first_query) -> weights */
static PyObject *key_weights(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Tensor q, k, lse;
    float scale;
    void *s, *pw;
    int here, st;
    static const char *const qk = "q and k must be contiguous bf16 tensors [B, H, N, d] and [B, Hkv, N, d], H a multiple of Hkv, on one CUDA device";
    if (!nargs_is(n, 6) || get_tensor(a[0], t_bf16, 4, -1, &q, qk) || get_tensor(a[1], t_bf16, 4, q.dev, &k, qk)) return NULL;
    if (k.dim[0] != q.dim[0] || k.dim[2] != q.dim[2] || k.dim[3] != q.dim[3] || k.dim[1] < 1 || q.dim[1] % k.dim[1] != 0)
        return refuse(qk), NULL;
    static const char *const what = "lse must be a contiguous fp32 tensor [B, H, N] on q's device";
    if (get_tensor(a[2], t_f32, 3, q.dev, &lse, what)) return NULL;
    for (int i = 0; i < 3; ++i)
        if (lse.dim[i] != q.dim[i]) return refuse(what), NULL;
    const int causal = PyObject_IsTrue(a[4]);
    const int64_t first = PyLong_AsLongLong(a[5]);
    if (causal < 0 || PyErr_Occurred() || get_scale(a[3], q.dim[3], &scale)) return NULL;
    if (first < 0 || first >= q.dim[2]) return refuse("first_query must lie in [0, N)"), NULL;
    if (get_stream(q.dev, &s, &here)) return NULL;
    if (!here) Py_RETURN_NOTIMPLEMENTED;
    const int64_t dim[3] = {q.dim[0], k.dim[1], q.dim[2]};
    PyObject *w = empty(3, dim, t_f32, q.dev, &pw);
    if (w == NULL) return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = p_weights(q.ptr, k.ptr, (const float *)lse.ptr, (float *)pw, q.dim[0], q.dim[1], k.dim[1], q.dim[2], q.dim[3], scale,
                   causal, first, s);
    Py_END_ALLOW_THREADS
    if (st == FA_OK) return w;
    Py_DECREF(w);
    return fail(st, "fa_key_weights");
}

/* setup(uint8, bfloat16, float32, int32, torch.empty, current raw stream, current device, FAError, addresses: a tuple of
 * fa_kv4_append, fa_kv4_read, fa_fwd_kv4, fa_fwd_kv4_workspace_bytes, fa_kv4_evict, fa_key_weights) */
static PyObject *setup(PyObject *self, PyObject *args)
{
    PyObject *p;
    unsigned long long f[6];
    if (!PyArg_ParseTuple(args, "OOOOOOOO(KKKKKK)", &t_u8, &t_bf16, &t_f32, &t_i32, &f_empty, &f_stream, &f_current, &c_error, &f[0],
                          &f[1], &f[2], &f[3], &f[4], &f[5]))
        return NULL;
    p = a_keep_refs;
    Py_INCREF(args);
    a_keep_refs = args; /* the objects above live as long as the module */
    Py_XDECREF(p);
    p_append = (void *)(uintptr_t)f[0];
    p_read = (void *)(uintptr_t)f[1];
    p_fwd = (void *)(uintptr_t)f[2];
    p_fwd_bytes = (void *)(uintptr_t)f[3];
    p_evict = (void *)(uintptr_t)f[4];
    p_weights = (void *)(uintptr_t)f[5];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "types, functions and addresses the calls use"},
    {"kv4_append", (PyCFunction)(void (*)(void))kv4_append, METH_FASTCALL, NULL},
    {"kv4_read", (PyCFunction)(void (*)(void))kv4_read, METH_FASTCALL, NULL},
    {"forward_kv4", (PyCFunction)(void (*)(void))forward_kv4, METH_FASTCALL, NULL},
    {"kv4_evict", (PyCFunction)(void (*)(void))kv4_evict, METH_FASTCALL, NULL},
    {"key_weights", (PyCFunction)(void (*)(void))key_weights, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void)
{
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_device = PyUnicode_InternFromString("get_device");
    s_contig = PyUnicode_InternFromString("is_contiguous");
    s_ptr = PyUnicode_InternFromString("data_ptr");
    PyObject *d = PyUnicode_InternFromString("dtype"), *v = PyUnicode_InternFromString("device");
    if (!s_dtype || !s_shape || !s_device || !s_contig || !s_ptr || !d || !v) return NULL;
    kw_empty = PyTuple_Pack(2, d, v);
    Py_DECREF(d);
    Py_DECREF(v);
    return kw_empty == NULL ? NULL : PyModule_Create(&module);
}
