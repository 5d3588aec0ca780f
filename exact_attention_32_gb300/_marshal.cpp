// The tensor-level calls of packed sequences, of the 4-bit cache, of attention over it and of key weights:
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

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/full.h>
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
decltype(&fa_fwd_kv4_tree) p_tree;
decltype(&fa_kv4_keep) p_keep;
decltype(&fa_kv4_copy_pages) p_copy;
decltype(&fa_packed_plan) p_plan;
decltype(&fa_packed_plan_bytes) p_plan_bytes;
decltype(&fa_fwd_packed) p_fwd_packed;
decltype(&fa_bwd_packed) p_bwd_packed;
decltype(&fa_bwd_packed_workspace_bytes) p_bwd_packed_bytes;
decltype(&fa_fwd_kv4_tree_workspace_bytes) p_tree_bytes;

constexpr at::ScalarType t_u8 = at::kByte, t_bf16 = at::kBFloat16, t_f32 = at::kFloat, t_i32 = at::kInt, t_i64 = at::kLong;

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
int get_index(PyObject *o, int nd, int64_t *B, int dev, Tensor *t, const char *what, at::ScalarType dtype = t_i32)
{
    if (get_tensor(o, dtype, nd, dev, t, what)) return -1;
    if (*B < 0) *B = t->dim[0];
    return t->dim[0] == *B ? 0 : refuse(what);
}
#define LENS "lens must be a contiguous int32 tensor [B] on the cache's device"
#define N_NEW "n_new must be a contiguous int32 tensor [B] on the cache's device"
#define SAME_LAYOUT "both caches must have the same key heads, page size, d and device"
#define TABLE "page_table must be a contiguous int32 tensor [B, pages] on the cache's device"

const int32_t *i32(const Tensor &t) { return static_cast<const int32_t *>(t.ptr); }

// Whether `dev` is the current device (else the caller makes it so and calls again).
bool here(int dev) { return c10::cuda::current_device() == dev; }
void *stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

// (at::empty goes by the dispatcher first, a third of its time)
at::Tensor empty(at::IntArrayRef dim, at::ScalarType dtype, int dev)
{
    return at::Tensor(at::detail::empty_cuda(dim, dtype, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt));
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
        if (get_index(a[5], 1, &B, dev, &extra, N_NEW)) return nullptr;
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

// Attention over a cache; with tree (and n_new, or None) of drafts.
PyObject *attend(PyObject *const *a, PyObject *tree_arg, PyObject *n_new_arg)
{
    fa_kv4_cache c;
    Tensor q, lens, table, ws, tree, n_new;
    int dev;
    float scale;
    int st;
    const char *const what = "q must be a contiguous bf16 tensor [B, H, n_q, d], with the cache's d and H a multiple of its key heads, on its device";
    if (get_cache(a[1], &c, &dev)) return nullptr;
    if (get_tensor(a[0], t_bf16, 4, dev, &q, what)) return nullptr;
    if (q.dim[3] != c.d || c.Hkv < 1 || q.dim[1] % c.Hkv != 0) return refuse(what), nullptr;
    int64_t B = q.dim[0];
    if (get_index(a[2], 1, &B, dev, &lens, LENS) || get_index(a[3], 2, &B, dev, &table, TABLE)) return nullptr;
    const int acc = PyObject_IsTrue(a[5]);
    if (acc < 0 || get_scale(a[4], c.d, &scale)) return nullptr;
    if (acc && c.weights == nullptr) return refuse("the cache holds no weights"), nullptr;
    tree.ptr = n_new.ptr = nullptr;
    if (tree_arg != nullptr) {
        const char *const masks = "tree must be a contiguous int64 tensor [B, n_q] on the cache's device";
        if (get_index(tree_arg, 2, &B, dev, &tree, masks, t_i64)) return nullptr;
        if (tree.dim[1] != q.dim[2]) return refuse(masks), nullptr;
        if (n_new_arg != Py_None && get_index(n_new_arg, 1, &B, dev, &n_new, N_NEW)) return nullptr;
    }
    const int64_t room = table.dim[1] * c.page_size;
    const int64_t need = tree_arg == nullptr ? p_fwd_bytes(B, q.dim[1], c.Hkv, q.dim[2], c.d, room, acc)
                                             : p_tree_bytes(B, q.dim[1], c.Hkv, q.dim[2], c.d, room);
    if (need < 0)
        return fail(c.d == 64 || c.d == 128 ? FA_ERR_INVALID_ARG : FA_ERR_UNSUPPORTED,
                    tree_arg == nullptr ? "fa_fwd_kv4_workspace_bytes" : "fa_fwd_kv4_tree_workspace_bytes");
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
        if (tree_arg == nullptr)
            st = p_fwd(q.ptr, &c, i32(lens), i32(table), o.data_ptr(), static_cast<float *>(lse.data_ptr()), B, q.dim[1], q.dim[2],
                       table.dim[1], scale, acc, ws.ptr, ws.dim[0], stream_of(dev));
        else
            st = p_tree(q.ptr, &c, i32(lens), i32(table), static_cast<const uint64_t *>(tree.ptr), i32(n_new), o.data_ptr(),
                        static_cast<float *>(lse.data_ptr()), B, q.dim[1], q.dim[2], table.dim[1], scale, ws.ptr, ws.dim[0],
                        stream_of(dev));
    }
    return st == FA_OK ? pair(std::move(o), std::move(lse)) : fail(st, tree_arg == nullptr ? "fa_fwd_kv4" : "fa_fwd_kv4_tree");
}

// (q, cache, lens, page_table, scale, accumulate, workspace) -> (o, lse)
PyObject *forward_kv4(PyObject *const *a, Py_ssize_t n) { return nargs_is(n, 7) ? attend(a, nullptr, nullptr) : nullptr; }

// (q, cache, lens, page_table, tree, n_new, scale, workspace) -> (o, lse)
PyObject *forward_kv4_tree(PyObject *const *a, Py_ssize_t n)
{
    if (!nargs_is(n, 8)) return nullptr;
    PyObject *const args[7] = {a[0], a[1], a[2], a[3], a[6], Py_False, a[7]};
    return attend(args, a[4], a[5]);
}

// (cache, lens, page_table, path, n_path, n_new) -> new_lens
PyObject *kv4_keep(PyObject *const *a, Py_ssize_t n)
{
    fa_kv4_cache c;
    Tensor lens, table, path, n_path, n_new;
    int dev;
    int st;
    int64_t B = -1;
    if (!nargs_is(n, 6) || get_cache(a[0], &c, &dev)) return nullptr;
    if (get_index(a[1], 1, &B, dev, &lens, LENS) || get_index(a[2], 2, &B, dev, &table, TABLE) ||
        get_index(a[3], 2, &B, dev, &path, "path must be a contiguous int32 tensor [B, drafts] on the cache's device") ||
        get_index(a[4], 1, &B, dev, &n_path, "n_path must be a contiguous int32 tensor [B] on the cache's device"))
        return nullptr;
    n_new.ptr = nullptr;
    if (a[5] != Py_None && get_index(a[5], 1, &B, dev, &n_new, N_NEW)) return nullptr;
    if (path.dim[1] < 1 || path.dim[1] > 64) return refuse("path must have 1 to 64 columns"), nullptr;
    if (!here(dev)) Py_RETURN_NOTIMPLEMENTED;
    at::Tensor now;
    {
        pybind11::gil_scoped_release free;
        now = empty({B}, t_i32, dev);
        st = p_keep(&c, i32(lens), i32(table), table.dim[1], i32(path), i32(n_path), i32(n_new), B, path.dim[1],
                    static_cast<int32_t *>(now.data_ptr()), stream_of(dev));
    }
    return st == FA_OK ? THPVariable_Wrap(std::move(now)) : fail(st, "fa_kv4_keep");
}

// (cache, pages, to, to_pages)
PyObject *kv4_copy_pages(PyObject *const *a, Py_ssize_t n)
{
    fa_kv4_cache c, t;
    Tensor pages, to_pages;
    int dev, dev_to;
    int st;
    int64_t count = -1;
    const char *const what = "pages and to_pages must be contiguous int32 tensors of one length on the cache's device";
    if (!nargs_is(n, 4) || get_cache(a[0], &c, &dev) || get_cache(a[2], &t, &dev_to)) return nullptr;
    if (dev_to != dev || t.Hkv != c.Hkv || t.page_size != c.page_size || t.d != c.d) return refuse(SAME_LAYOUT), nullptr;
    if (get_index(a[1], 1, &count, dev, &pages, what) || get_index(a[3], 1, &count, dev, &to_pages, what)) return nullptr;
    if (!here(dev)) Py_RETURN_NOTIMPLEMENTED;
    if (count == 0) Py_RETURN_NONE;
    {
        pybind11::gil_scoped_release free;
        st = p_copy(&c, i32(pages), &t, i32(to_pages), count, stream_of(dev));
    }
    if (st != FA_OK) return fail(st, "fa_kv4_copy_pages");
    Py_RETURN_NONE;
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
            return refuse(SAME_LAYOUT), nullptr;
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

// A packed bf16 tensor [T, heads, d], d contiguous, on CUDA device `dev` (any where dev < 0); T, heads and d below 0 are set.
struct Packed {
    fa_rows r;
    int64_t T, heads, d;
    int dev;
};
int get_packed(PyObject *o, int dev, int64_t T, int64_t heads, int64_t d, Packed *t, const char *what)
{
    if (!THPVariable_Check(o)) return refuse(what);
    const at::Tensor &x = THPVariable_Unpack(o);
    if (!x.is_cuda() || x.layout() != at::kStrided || x.scalar_type() != t_bf16 || x.dim() != 3 || x.is_neg() || x.stride(2) != 1)
        return refuse(what);
    t->dev = x.get_device();
    t->T = x.size(0);
    t->heads = x.size(1);
    t->d = x.size(2);
    if ((dev >= 0 && t->dev != dev) || (T >= 0 && t->T != T) || (heads >= 0 && t->heads != heads) || (d >= 0 && t->d != d))
        return refuse(what);
    for (int i = 0; i < 2; ++i)
        if (x.size(i) > 1 && (x.stride(i) < t->d || x.stride(i) % 8 != 0))
            return refuse("a packed tensor's tokens and heads must lie at least d and a multiple of 8 elements apart "
                          "(what expand() makes has to be made contiguous)");
    t->r = {x.data_ptr(), x.stride(0), x.stride(1)};
    return 0;
}
#define QKV "q, k and v must be bf16 tensors [T, H, d], [T, Hkv, d] and [T, Hkv, d], H a multiple of Hkv, the last axis contiguous, on one CUDA device"
#define CU "cu_seqlens must be a contiguous int32 tensor [sequences + 1] on the tensors' device"

// q, k, v, and the offsets of B sequences.
int get_batch(PyObject *const *qkv, PyObject *cu_arg, Packed (&x)[3], Tensor *cu, int64_t *B)
{
    if (get_packed(qkv[0], -1, -1, -1, -1, &x[0], QKV) || get_packed(qkv[1], x[0].dev, x[0].T, -1, x[0].d, &x[1], QKV) ||
        get_packed(qkv[2], x[0].dev, x[0].T, x[1].heads, x[0].d, &x[2], QKV))
        return -1;
    if (x[1].heads < 1 || x[0].heads % x[1].heads != 0) return refuse(QKV);
    if (get_tensor(cu_arg, t_i32, 1, x[0].dev, cu, CU)) return -1;
    *B = cu->dim[0] - 1;
    return *B >= 1 ? 0 : refuse(CU);
}

// A plan's memory: given (a PackedPlan, held to this batch), or null with the bytes that one needs.
int get_plan(PyObject *o, int64_t B, int64_t T, int causal, int dev, void **ptr, int64_t *bytes)
{
    *ptr = nullptr;
    *bytes = p_plan_bytes(B, T);
    if (*bytes < 0) return fail(FA_ERR_INVALID_ARG, "fa_packed_plan_bytes"), -1;
    if (o == Py_None) return 0;
    const char *const what = "plan must be packed_plan's for these cu_seqlens, this number of tokens and this causal";
    Tensor t;
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4 || get_tensor(PyTuple_GET_ITEM(o, 0), t_u8, 1, dev, &t, what)) return refuse(what);
    const int64_t tokens = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 1)), sequences = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 2));
    const int same = PyObject_IsTrue(PyTuple_GET_ITEM(o, 3));
    if (PyErr_Occurred()) return -1;
    if (tokens != T || sequences != B || same != causal || t.dim[0] < *bytes) return refuse(what);
    *ptr = t.ptr;
    return 0;
}

// (cu_seqlens, tokens, causal) -> plan
PyObject *packed_plan(PyObject *const *a, Py_ssize_t n)
{
    Tensor cu;
    int st;
    if (!nargs_is(n, 3) || get_tensor(a[0], t_i32, 1, -1, &cu, CU)) return nullptr;
    const int64_t T = PyLong_AsLongLong(a[1]), B = cu.dim[0] - 1;
    const int causal = PyObject_IsTrue(a[2]);
    if (causal < 0 || PyErr_Occurred()) return nullptr;
    if (B < 1) return refuse(CU), nullptr;
    const int64_t bytes = p_plan_bytes(B, T);
    if (bytes < 0) return fail(FA_ERR_INVALID_ARG, "fa_packed_plan_bytes");
    if (!here(cu.dev)) Py_RETURN_NOTIMPLEMENTED;
    at::Tensor plan;
    {
        pybind11::gil_scoped_release free;
        plan = empty({bytes}, t_u8, cu.dev);
        st = p_plan(i32(cu), B, T, causal, plan.data_ptr(), bytes, stream_of(cu.dev));
    }
    return st == FA_OK ? THPVariable_Wrap(std::move(plan)) : fail(st, "fa_packed_plan");
}

// (q, k, v, cu_seqlens, scale, causal, plan, out, lse) -> (o, lse)
PyObject *forward_packed(PyObject *const *a, Py_ssize_t n)
{
    Packed x[3], out;
    Tensor cu, lse_t;
    float scale;
    int st;
    int64_t B, bytes;
    void *plan;
    if (!nargs_is(n, 9) || get_batch(a, a[3], x, &cu, &B)) return nullptr;
    const int dev = x[0].dev;
    const int64_t T = x[0].T, H = x[0].heads, d = x[0].d;
    const int causal = PyObject_IsTrue(a[5]);
    if (causal < 0 || get_scale(a[4], d, &scale) || get_plan(a[6], B, T, causal, dev, &plan, &bytes)) return nullptr;
    at::Tensor o, lse, own;
    if (a[7] != Py_None) {
        if (get_packed(a[7], dev, T, H, d, &out, "out must be a bf16 tensor [T, H, d], the last axis contiguous, on q's device")) return nullptr;
        o = THPVariable_Unpack(a[7]);
    }
    if (a[8] != Py_None) {
        const char *const what = "lse must be a contiguous fp32 tensor [H, T] on q's device";
        if (get_tensor(a[8], t_f32, 2, dev, &lse_t, what)) return nullptr;
        if (lse_t.dim[0] != H || lse_t.dim[1] != T) return refuse(what), nullptr;
        lse = THPVariable_Unpack(a[8]);
    }
    if (!here(dev)) Py_RETURN_NOTIMPLEMENTED;
    {
        pybind11::gil_scoped_release free;
        // rows of no sequence: filled in tensors of this call's own, left alone in given ones
        const int fill = a[7] == Py_None && a[8] == Py_None;
        const auto opt = [&](at::ScalarType t) { return at::TensorOptions().dtype(t).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)); };
        if (a[7] == Py_None) {
            o = fill ? empty({T, H, d}, t_bf16, dev) : at::full({T, H, d}, 0, opt(t_bf16));
            out.r = {o.data_ptr(), H * d, d};
        }
        if (a[8] == Py_None) lse = fill ? empty({H, T}, t_f32, dev) : at::full({H, T}, -INFINITY, opt(t_f32));
        st = FA_OK;
        if (plan == nullptr) {
            own = empty({bytes}, t_u8, dev);
            plan = own.data_ptr();
            st = p_plan(i32(cu), B, T, causal, plan, bytes, stream_of(dev));
        }
        if (st == FA_OK)
            st = p_fwd_packed(&x[0].r, &x[1].r, &x[2].r, &out.r, static_cast<float *>(lse.data_ptr()), plan, B, T, H, x[1].heads, d,
                              scale, causal, fill, stream_of(dev));
    }
    return st == FA_OK ? pair(std::move(o), std::move(lse)) : fail(st, "fa_fwd_packed");
}

// (q, k, v, o, lse, dout, cu_seqlens, scale, causal, plan, workspace, (dq, dk, dv) or None) -> (dq, dk, dv)
PyObject *backward_packed(PyObject *const *a, Py_ssize_t n)
{
    Packed x[3], o, dout, g[3];
    Tensor cu, lse, ws;
    float scale;
    int st;
    int64_t B, bytes;
    void *plan;
    if (!nargs_is(n, 12) || get_batch(a, a[6], x, &cu, &B)) return nullptr;
    const int dev = x[0].dev;
    const int64_t T = x[0].T, H = x[0].heads, Hkv = x[1].heads, d = x[0].d;
    const char *const what = "o and dout must be bf16 tensors like q, the last axis contiguous";
    if (get_packed(a[3], dev, T, H, d, &o, what) || get_packed(a[5], dev, T, H, d, &dout, what)) return nullptr;
    const char *const lse_what = "lse must be a contiguous fp32 tensor [H, T] on q's device";
    if (get_tensor(a[4], t_f32, 2, dev, &lse, lse_what)) return nullptr;
    if (lse.dim[0] != H || lse.dim[1] != T) return refuse(lse_what), nullptr;
    const int causal = PyObject_IsTrue(a[8]);
    if (causal < 0 || get_scale(a[7], d, &scale) || get_plan(a[9], B, T, causal, dev, &plan, &bytes)) return nullptr;
    const int64_t need = p_bwd_packed_bytes(B, T, H, Hkv, d);
    if (need < 0) return fail(d == 64 || d == 128 ? FA_ERR_INVALID_ARG : FA_ERR_UNSUPPORTED, "fa_bwd_packed_workspace_bytes");
    if (a[10] != Py_None && get_tensor(a[10], t_u8, 1, dev, &ws, "workspace must be a contiguous uint8 tensor [bytes] on q's device"))
        return nullptr;
    at::Tensor grad[3], own, own_plan;
    if (a[11] != Py_None) {
        const char *const grads = "out must be (dq, dk, dv), bf16 tensors like q, k and v, the last axis contiguous";
        if (!PyTuple_Check(a[11]) || PyTuple_GET_SIZE(a[11]) != 3) return refuse(grads), nullptr;
        for (int i = 0; i < 3; ++i) {
            if (get_packed(PyTuple_GET_ITEM(a[11], i), dev, T, x[i].heads, d, &g[i], grads)) return nullptr;
            grad[i] = THPVariable_Unpack(PyTuple_GET_ITEM(a[11], i));
        }
    }
    if (!here(dev)) Py_RETURN_NOTIMPLEMENTED;
    {
        pybind11::gil_scoped_release free;
        const int fill = a[11] == Py_None;  // (as in forward_packed)
        for (int i = 0; fill && i < 3; ++i) {
            grad[i] = empty({T, x[i].heads, d}, t_bf16, dev);
            g[i].r = {grad[i].data_ptr(), x[i].heads * d, d};
        }
        if (a[10] == Py_None) {
            own = empty({need}, t_u8, dev);
            ws.ptr = own.data_ptr();
            ws.dim[0] = need;
        }
        st = FA_OK;
        if (plan == nullptr) {
            own_plan = empty({bytes}, t_u8, dev);
            plan = own_plan.data_ptr();
            st = p_plan(i32(cu), B, T, causal, plan, bytes, stream_of(dev));
        }
        if (st == FA_OK)
            st = p_bwd_packed(&x[0].r, &x[1].r, &x[2].r, &o.r, static_cast<const float *>(lse.ptr), &dout.r, &g[0].r, &g[1].r, &g[2].r,
                              plan, B, T, H, Hkv, d, scale, causal, fill, ws.ptr, ws.dim[0], stream_of(dev));
    }
    if (st != FA_OK) return fail(st, "fa_bwd_packed");
    PyObject *r = PyTuple_New(3);
    for (int i = 0; r != nullptr && i < 3; ++i) {
        PyObject *t = THPVariable_Wrap(std::move(grad[i]));
        if (t == nullptr) Py_CLEAR(r);
        else PyTuple_SET_ITEM(r, i, t);
    }
    return r;
}

// setup(FAError, addresses: a tuple of fa_kv4_append, fa_kv4_read, fa_fwd_kv4, fa_fwd_kv4_workspace_bytes, fa_kv4_evict,
// fa_key_weights, fa_fwd_kv4_tree, fa_kv4_keep, fa_kv4_copy_pages, fa_packed_plan, fa_packed_plan_bytes, fa_fwd_packed,
// fa_bwd_packed, fa_bwd_packed_workspace_bytes, fa_fwd_kv4_tree_workspace_bytes)
PyObject *setup(PyObject *, PyObject *args)
{
    PyObject *e;
    unsigned long long f[15];
    if (!PyArg_ParseTuple(args, "O(KKKKKKKKKKKKKKK)", &e, &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &f[7], &f[8], &f[9], &f[10],
                          &f[11], &f[12], &f[13], &f[14]))
        return nullptr;
    Py_INCREF(e);  // (lives as long as the module)
    Py_XSETREF(c_error, e);
    p_append = reinterpret_cast<decltype(p_append)>(f[0]);
    p_read = reinterpret_cast<decltype(p_read)>(f[1]);
    p_fwd = reinterpret_cast<decltype(p_fwd)>(f[2]);
    p_fwd_bytes = reinterpret_cast<decltype(p_fwd_bytes)>(f[3]);
    p_evict = reinterpret_cast<decltype(p_evict)>(f[4]);
    p_weights = reinterpret_cast<decltype(p_weights)>(f[5]);
    p_tree = reinterpret_cast<decltype(p_tree)>(f[6]);
    p_keep = reinterpret_cast<decltype(p_keep)>(f[7]);
    p_copy = reinterpret_cast<decltype(p_copy)>(f[8]);
    p_plan = reinterpret_cast<decltype(p_plan)>(f[9]);
    p_plan_bytes = reinterpret_cast<decltype(p_plan_bytes)>(f[10]);
    p_fwd_packed = reinterpret_cast<decltype(p_fwd_packed)>(f[11]);
    p_bwd_packed = reinterpret_cast<decltype(p_bwd_packed)>(f[12]);
    p_bwd_packed_bytes = reinterpret_cast<decltype(p_bwd_packed_bytes)>(f[13]);
    p_tree_bytes = reinterpret_cast<decltype(p_tree_bytes)>(f[14]);
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
                         CALL(forward_kv4_tree),
                         CALL(kv4_keep),
                         CALL(kv4_copy_pages),
                         CALL(packed_plan),
                         CALL(forward_packed),
                         CALL(backward_packed),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
