// The tensor-level calls of the 4-bit cache, of attention over it and of key weights:
// checks of the tensors, allocation of outputs, and the call into libfa.so, as a
// CPython extension over torch's C++ tensors.  A decode step's kernels take a few
// microseconds; the same steps in Python took 10 to 30 more (a tensor attribute costs
// 60 to 250 ns, marshalling a dozen arguments through ctypes 3 us), and reading the
// attributes through the Python objects from C still 5 to 15.  The library is not linked:
// _binding.py hands over the addresses of its functions, so there is one copy of
// it in the process.  No arithmetic here; every refusal raises.
#include <Python.h>
#include <math.h>
#include <stdint.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include "fa.h"

namespace {

PyObject *c_error;

decltype(&fa_kv4_append) p_append;
decltype(&fa_kv4_read) p_read;
decltype(&fa_fwd_kv4) p_fwd;
decltype(&fa_fwd_kv4_workspace_bytes) p_fwd_bytes;
decltype(&fa_kv4_evict) p_evict;
decltype(&fa_key_weights) p_weights;

constexpr at::ScalarType t_u8 = at::kByte, t_bf16 = at::kBFloat16, t_f32 = at::kFloat, t_i32 = at::kInt;

struct Tensor {
    int64_t dim[4];
    void *ptr;
    int dev;
};

int refuse(const char *what)
{
    PyErr_SetString(PyExc_ValueError, what);
    return -1;
}

// A contiguous tensor of `dtype` and `nd` dimensions on CUDA device `dev` (any where dev < 0); 0, or -1 with `what` raised.
int get_tensor(PyObject *o, at::ScalarType dtype, int nd, int dev, Tensor *t, const char *what)
{
    if (!THPVariable_Check(o)) return refuse(what);
    const at::Tensor &x = THPVariable_Unpack(o);
    if (!x.is_cuda() || x.layout() != at::kStrided || x.scalar_type() != dtype || x.dim() != nd || x.is_neg() || !x.is_contiguous())
        return refuse(what);
    t->dev = x.get_device();
    if (dev >= 0 && t->dev != dev) return refuse(what);
    for (int i = 0; i < nd; ++i) t->dim[i] = x.size(i);
    t->ptr = x.data_ptr();
    return 0;
}

// A KV4Cache as the library's struct; *dev is its device.
int get_cache(PyObject *o, fa_kv4_cache *c, int *dev)
{
    const char *const codes = "k and v of a cache must be contiguous uint8 tensors [n_pages, Hkv, page_size, d/2] on one CUDA device";
    const char *const scales = "k_scale and v_scale of a cache must be contiguous uint8 tensors [n_pages, Hkv, page_size, d/32] and "
                                      "[n_pages, Hkv, page_size] on its device";
    const char *const weights = "weights of a cache must be a contiguous fp32 tensor [n_pages, Hkv, page_size] on its device";
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
    c->weights = nullptr;
    if (PyTuple_GET_ITEM(o, 4) != Py_None) {
        if (get_tensor(PyTuple_GET_ITEM(o, 4), t_f32, 3, k.dev, &t, weights)) return -1;
        if (t.dim[0] != k.dim[0] || t.dim[1] != k.dim[1] || t.dim[2] != k.dim[2]) return refuse(weights);
        c->weights = static_cast<float *>(t.ptr);
    }
    return 0;
}

// int32 index tensors: [B], or [B, columns]; B < 0 is set.
int get_index(PyObject *o, int nd, int64_t *B, int dev, Tensor *t, const char *what)
{
    if (get_tensor(o, t_i32, nd, dev, t, what)) return -1;
    if (*B < 0) *B = t->dim[0];
    return t->dim[0] == *B ? 0 : refuse(what);
}
#define LENS "lens must be a contiguous int32 tensor [B] on the cache's device"
#define TABLE "page_table must be a contiguous int32 tensor [B, pages] on the cache's device"

const int32_t *i32(const Tensor &t) { return static_cast<const int32_t *>(t.ptr); }

// Whether `dev` is the current device (else the caller makes it so and calls again).
bool here(int dev) { return c10::cuda::current_device() == dev; }
void *stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

at::Tensor empty(at::IntArrayRef dim, at::ScalarType dtype, int dev)
{
    return at::empty(dim, at::TensorOptions().dtype(dtype).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
}

// (a, b) as a Python tuple
PyObject *pair(at::Tensor a, at::Tensor b)
{
    PyObject *x = THPVariable_Wrap(std::move(a)), *y = x == nullptr ? nullptr : THPVariable_Wrap(std::move(b));
    PyObject *r = y == nullptr ? nullptr : PyTuple_Pack(2, x, y);
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

PyObject *fail(int status, const char *where)
{
    PyObject *e = PyObject_CallFunction(c_error, "is", status, where);
    if (e != nullptr) {
        PyErr_SetObject(c_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

int nargs_is(Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return 1;
    PyErr_Format(PyExc_TypeError, "%zd arguments are needed, not %zd", want, n);
    return 0;
}

// (cache, k, v, lens, page_table, n_new, weights)
PyObject *kv4_append(PyObject *const *a, Py_ssize_t n)
{
    fa_kv4_cache c;
    Tensor k, v, lens, table, extra;
    int dev;
    void *p_new = nullptr, *p_w = nullptr;
    int st;
    const char *const kv = "k and v must be contiguous bf16 tensors [B, Hkv, S, d], with the cache's Hkv and d, on its device";
    const char *const w = "weights must be a contiguous fp32 tensor [B, Hkv, S] on the cache's device";
    if (!nargs_is(n, 7) || get_cache(a[0], &c, &dev)) return nullptr;
    if (get_tensor(a[1], t_bf16, 4, dev, &k, kv) || get_tensor(a[2], t_bf16, 4, dev, &v, kv)) return nullptr;
    for (int i = 0; i < 4; ++i)
        if (k.dim[i] != v.dim[i]) return refuse(kv), nullptr;
    if (k.dim[1] != c.Hkv || k.dim[3] != c.d) return refuse(kv), nullptr;
    int64_t B = k.dim[0];
    if (get_index(a[3], 1, &B, dev, &lens, LENS) || get_index(a[4], 2, &B, dev, &table, TABLE)) return nullptr;
    if (a[5] != Py_None) {
        if (get_index(a[5], 1, &B, dev, &extra, "n_new must be a contiguous int32 tensor [B] on the cache's device")) return nullptr;
        p_new = extra.ptr;
    }
    if (a[6] != Py_None) {
        if (get_tensor(a[6], t_f32, 3, dev, &extra, w)) return nullptr;
        if (extra.dim[0] != B || extra.dim[1] != c.Hkv || extra.dim[2] != k.dim[2]) return refuse(w), nullptr;
        if (c.weights == nullptr) return refuse("the cache holds no weights"), nullptr;
        p_w = extra.ptr;
    }
    if (!here(dev)) Py_RETURN_NOTIMPLEMENTED;
    {
        pybind11::gil_scoped_release free;
        st = p_append(&c, k.ptr, v.ptr, static_cast<const float *>(p_w), static_cast<const int32_t *>(p_new), i32(lens), i32(table),
                      B, k.dim[2], table.dim[1], stream_of(dev));
    }
    if (st != FA_OK) return fail(st, "fa_kv4_append");
    Py_RETURN_NONE;
}

// (cache, lens, page_table, count, first) -> (k, v)
PyObject *kv4_read(PyObject *const *a, Py_ssize_t n)
{
    fa_kv4_cache c;
    Tensor lens, table, first;
    int dev;
    void *pf = nullptr;
    int st;
    int64_t B = -1;
    if (!nargs_is(n, 5) || get_cache(a[0], &c, &dev)) return nullptr;
    if (get_index(a[1], 1, &B, dev, &lens, LENS) || get_index(a[2], 2, &B, dev, &table, TABLE)) return nullptr;
    const int64_t count = PyLong_AsLongLong(a[3]);
    if (count == -1 && PyErr_Occurred()) return nullptr;
    if (count < 1) return refuse("count must be at least 1"), nullptr;
    if (a[4] != Py_None) {
        if (get_index(a[4], 1, &B, dev, &first, "first must be a contiguous int32 tensor [B] on the cache's device")) return nullptr;
        pf = first.ptr;
    }
    if (!here(dev)) Py_RETURN_NOTIMPLEMENTED;
    at::Tensor k, v;
    {
        pybind11::gil_scoped_release free;
        k = empty({B, c.Hkv, count, c.d}, t_bf16, dev);
        v = empty({B, c.Hkv, count, c.d}, t_bf16, dev);
        st = p_read(&c, static_cast<const int32_t *>(pf), i32(lens), i32(table), B, table.dim[1], count, k.data_ptr(), v.data_ptr(),
                    stream_of(dev));
    }
    return st == FA_OK ? pair(std::move(k), std::move(v)) : fail(st, "fa_kv4_read");
}

// scale argument: None is fp32 1 / sqrt(d)
int get_scale(PyObject *o, int64_t d, float *scale)
{
    const double x = o == Py_None ? 1.0 / sqrt(static_cast<double>(d)) : PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) return -1;
    *scale = static_cast<float>(x);
    return 0;
}

// (q, cache, lens, page_table, scale, accumulate, workspace) -> (o, lse)
PyObject *forward_kv4(PyObject *const *a, Py_ssize_t n)
{
    fa_kv4_cache c;
    Tensor q, lens, table, ws;
    int dev;
    float scale;
    int st;
    const char *const what = "q must be a contiguous bf16 tensor [B, H, n_q, d], with the cache's d and H a multiple of its key heads, on its device";
    if (!nargs_is(n, 7) || get_cache(a[1], &c, &dev)) return nullptr;
    if (get_tensor(a[0], t_bf16, 4, dev, &q, what)) return nullptr;
    if (q.dim[3] != c.d || c.Hkv < 1 || q.dim[1] % c.Hkv != 0) return refuse(what), nullptr;
    int64_t B = q.dim[0];
    if (get_index(a[2], 1, &B, dev, &lens, LENS) || get_index(a[3], 2, &B, dev, &table, TABLE)) return nullptr;
    const int acc = PyObject_IsTrue(a[5]);
    if (acc < 0 || get_scale(a[4], c.d, &scale)) return nullptr;
    if (acc && c.weights == nullptr) return refuse("the cache holds no weights"), nullptr;
    const int64_t need = p_fwd_bytes(B, q.dim[1], c.Hkv, q.dim[2], c.d, table.dim[1] * c.page_size, acc);
    if (need < 0) return fail(c.d == 64 || c.d == 128 ? FA_ERR_INVALID_ARG : FA_ERR_UNSUPPORTED, "fa_fwd_kv4_workspace_bytes");
    if (!here(dev)) Py_RETURN_NOTIMPLEMENTED;
    if (a[6] != Py_None &&
        get_tensor(a[6], t_u8, 1, dev, &ws, "workspace must be a contiguous uint8 tensor [bytes] on the cache's device"))
        return nullptr;
    at::Tensor own, o, lse;
    {
        pybind11::gil_scoped_release free;
        if (a[6] == Py_None) {
            own = empty({need}, t_u8, dev);
            ws.ptr = own.data_ptr();
            ws.dim[0] = need;
        }
        o = empty({B, q.dim[1], q.dim[2], q.dim[3]}, t_bf16, dev);
        lse = empty({B, q.dim[1], q.dim[2]}, t_f32, dev);
        st = p_fwd(q.ptr, &c, i32(lens), i32(table), o.data_ptr(), static_cast<float *>(lse.data_ptr()), B, q.dim[1], q.dim[2],
                   table.dim[1], scale, acc, ws.ptr, ws.dim[0], stream_of(dev));
    }
    return st == FA_OK ? pair(std::move(o), std::move(lse)) : fail(st, "fa_fwd_kv4");
}

// (cache, lens, page_table, to, to_table, keep, recent) -> (kept, new_lens)
PyObject *kv4_evict(PyObject *const *a, Py_ssize_t n)
{
    fa_kv4_cache c, t;
    Tensor lens, table, to_table;
    int dev, dev_to;
    int st;
    int64_t B = -1;
    if (!nargs_is(n, 7) || get_cache(a[0], &c, &dev)) return nullptr;
    if (a[3] == a[0]) {
        t = c;
    } else {
        if (get_cache(a[3], &t, &dev_to)) return nullptr;
        if (dev_to != dev || t.Hkv != c.Hkv || t.page_size != c.page_size || t.d != c.d)
            return refuse("both caches must have the same key heads, page size, d and device"), nullptr;
    }
    if (c.weights == nullptr || t.weights == nullptr) return refuse("eviction needs the weights of both caches"), nullptr;
    if (get_index(a[1], 1, &B, dev, &lens, LENS) || get_index(a[2], 2, &B, dev, &table, TABLE) ||
        get_index(a[4], 2, &B, dev, &to_table, "to_table must be a contiguous int32 tensor [B, pages] on the cache's device"))
        return nullptr;
    const int64_t keep = PyLong_AsLongLong(a[5]), recent = PyLong_AsLongLong(a[6]);
    if (PyErr_Occurred()) return nullptr;
    if (keep < 1 || recent < 0 || recent > keep || keep > to_table.dim[1] * c.page_size)
        return refuse("need 1 <= keep <= the tokens of to_table's pages, and 0 <= recent <= keep"), nullptr;
    if (!here(dev)) Py_RETURN_NOTIMPLEMENTED;
    at::Tensor kept, now;
    {
        pybind11::gil_scoped_release free;
        kept = empty({B, c.Hkv, keep}, t_i32, dev);
        now = empty({B}, t_i32, dev);
        st = p_evict(&c, i32(lens), i32(table), table.dim[1], &t, i32(to_table), to_table.dim[1], B, keep, recent,
                     static_cast<int32_t *>(kept.data_ptr()), static_cast<int32_t *>(now.data_ptr()), stream_of(dev));
    }
    return st == FA_OK ? pair(std::move(kept), std::move(now)) : fail(st, "fa_kv4_evict");
}

// (q, k, lse, scale, causal, first_query) -> weights
PyObject *key_weights(PyObject *const *a, Py_ssize_t n)
{
    Tensor q, k, lse;
    float scale;
    int st;
    const char *const qk = "q and k must be contiguous bf16 tensors [B, H, N, d] and [B, Hkv, N, d], H a multiple of Hkv, on one CUDA device";
    if (!nargs_is(n, 6) || get_tensor(a[0], t_bf16, 4, -1, &q, qk) || get_tensor(a[1], t_bf16, 4, q.dev, &k, qk)) return nullptr;
    if (k.dim[0] != q.dim[0] || k.dim[2] != q.dim[2] || k.dim[3] != q.dim[3] || k.dim[1] < 1 || q.dim[1] % k.dim[1] != 0)
        return refuse(qk), nullptr;
    const char *const what = "lse must be a contiguous fp32 tensor [B, H, N] on q's device";
    if (get_tensor(a[2], t_f32, 3, q.dev, &lse, what)) return nullptr;
    for (int i = 0; i < 3; ++i)
        if (lse.dim[i] != q.dim[i]) return refuse(what), nullptr;
    const int causal = PyObject_IsTrue(a[4]);
    const int64_t first = PyLong_AsLongLong(a[5]);
    if (causal < 0 || PyErr_Occurred() || get_scale(a[3], q.dim[3], &scale)) return nullptr;
    if (first < 0 || first >= q.dim[2]) return refuse("first_query must lie in [0, N)"), nullptr;
    if (!here(q.dev)) Py_RETURN_NOTIMPLEMENTED;
    at::Tensor w;
    {
        pybind11::gil_scoped_release free;
        w = empty({q.dim[0], k.dim[1], q.dim[2]}, t_f32, q.dev);
        st = p_weights(q.ptr, k.ptr, static_cast<const float *>(lse.ptr), static_cast<float *>(w.data_ptr()), q.dim[0], q.dim[1],
                       k.dim[1], q.dim[2], q.dim[3], scale, causal, first, stream_of(q.dev));
    }
    return st == FA_OK ? THPVariable_Wrap(std::move(w)) : fail(st, "fa_key_weights");
}

// setup(FAError, addresses: a tuple of fa_kv4_append, fa_kv4_read, fa_fwd_kv4, fa_fwd_kv4_workspace_bytes, fa_kv4_evict,
// fa_key_weights)
PyObject *setup(PyObject *, PyObject *args)
{
    PyObject *e;
    unsigned long long f[6];
    if (!PyArg_ParseTuple(args, "O(KKKKKK)", &e, &f[0], &f[1], &f[2], &f[3], &f[4], &f[5])) return nullptr;
    Py_INCREF(e);  // (lives as long as the module)
    Py_XSETREF(c_error, e);
    p_append = reinterpret_cast<decltype(p_append)>(f[0]);
    p_read = reinterpret_cast<decltype(p_read)>(f[1]);
    p_fwd = reinterpret_cast<decltype(p_fwd)>(f[2]);
    p_fwd_bytes = reinterpret_cast<decltype(p_fwd_bytes)>(f[3]);
    p_evict = reinterpret_cast<decltype(p_evict)>(f[4]);
    p_weights = reinterpret_cast<decltype(p_weights)>(f[5]);
    Py_RETURN_NONE;
}

// A C++ exception (an allocation that fails, a tensor without memory) leaves a call as torch's Python exception for it.
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *call(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    return F(a, n);
    END_HANDLE_TH_ERRORS
}

#define CALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<f>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"setup", setup, METH_VARARGS, "the error class and the addresses the calls use"},
                         CALL(kv4_append),
                         CALL(kv4_read),
                         CALL(forward_kv4),
                         CALL(kv4_evict),
                         CALL(key_weights),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
