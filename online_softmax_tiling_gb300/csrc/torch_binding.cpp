// torch_binding.cpp - torch tensors to the C ABI of include/fa_paged.h.
//
// Argument checks, allocation of outputs and workspaces, and the call; the
// functions' documentation is in paged.py, their only caller.  A decode step's
// kernels take a few microseconds, less than the same marshalling costs in
// Python (20 us a call on the GB300's host), so it is done here.
// Every function returns its outputs, or the FA_ERR_* status of the call as an
// int; wrong tensors raise TypeError or ValueError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <optional>

#include "../../include/fa.h"
#include "../../include/fa_paged.h"

namespace {

// A Python exception is set; unwinds to the function's entry.
struct Raised {};

[[noreturn]] void refuse(PyObject* kind, const char* name, const char* what) {
    PyErr_Format(kind, "%s %s", name, what);
    throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, "must be a tensor");
    return THPVariable_Unpack(o);
}

int device_of(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse(PyExc_ValueError, name, "must be on a CUDA device");
    return t.get_device();
}

void on_device(const at::Tensor& t, const char* name, int dev) {
    if (!t.is_cuda() || t.get_device() != dev) refuse(PyExc_ValueError, name, "must be on the device of the other tensors");
}

// Address of a contiguous tensor of this type and shape on device `dev`.
template <typename T = void>
T* need(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
    const at::Tensor& t = tensor(o, name);
    on_device(t, name, dev);
    if (t.scalar_type() != type) {
        PyErr_Format(PyExc_ValueError, "%s must be of type %s", name, c10::toString(type));
        throw Raised{};
    }
    if (t.sizes() != shape) {
        std::string want = c10::str(shape), got = c10::str(t.sizes());
        PyErr_Format(PyExc_ValueError, "%s must have the shape %s, got %s", name, want.c_str(), got.c_str());
        throw Raised{};
    }
    if (!t.is_contiguous()) refuse(PyExc_ValueError, name, "must be contiguous");
    return static_cast<T*>(t.data_ptr());
}

int dtype_of(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kHalf) return FA_FP16;
    if (t.scalar_type() == at::kBFloat16) return FA_BF16;
    refuse(PyExc_TypeError, name, "must be float16 or bfloat16");
}

// {token, head} strides of a [rows, heads, d] tensor with contiguous d.  The
// stride of a dimension of at most one element is never used: any valid one will do.
struct Strides {
    long long s[2];
};
Strides rows16(const at::Tensor& t, const char* name, at::ScalarType type, int dev) {
    on_device(t, name, dev);
    if (t.dim() != 3) refuse(PyExc_ValueError, name, "must be [tokens, heads, d]");
    if (t.scalar_type() != type) refuse(PyExc_TypeError, name, "must have the type of the other 16-bit tensors");
    if (t.stride(2) != 1 && t.size(2) > 1) refuse(PyExc_ValueError, name, "must have a contiguous last dimension");
    return {{t.size(0) > 1 ? t.stride(0) : 8, t.size(1) > 1 ? t.stride(1) : 8}};
}

int integer(PyObject* o, const char* name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v != static_cast<int>(v)) refuse(PyExc_ValueError, name, "does not fit 32 bits");
    return static_cast<int>(v);
}

int dim32(int64_t n, const char* name) {
    if (n > INT32_MAX) refuse(PyExc_ValueError, name, "has a dimension beyond 32 bits");
    return static_cast<int>(n);
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int dev) {
    return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<at::DeviceIndex>(dev)), std::nullopt);
}

// The cache's sizes from k_cache [num_pages, Hk, P, d].
fa_kv_cache cache_of(PyObject* k, PyObject* v, PyObject* ks, PyObject* vs, PyObject* bounds, int dev) {
    const at::Tensor& t = tensor(k, "k_cache");
    if (t.dim() != 4) refuse(PyExc_ValueError, "k_cache", "must be [num_pages, Hk, page_size, d]");
    const int64_t N = t.size(0), H = t.size(1), d = t.size(3);
    fa_kv_cache c;
    c.k = need<>(k, "k_cache", at::kFloat8_e4m3fn, t.sizes(), dev);
    c.v = need<>(v, "v_cache", at::kFloat8_e4m3fn, t.sizes(), dev);
    c.k_scale = need<float>(ks, "k_scale", at::kFloat, {N, H}, dev);
    c.v_scale = need<float>(vs, "v_scale", at::kFloat, {N, H}, dev);
    c.k_bounds = bounds == Py_None ? nullptr : need<signed char>(bounds, "k_bounds", at::kChar, {N, H, 2, d}, dev);
    c.num_pages = dim32(N, "k_cache"), c.Hk = dim32(H, "k_cache");
    c.page_size = dim32(t.size(2), "k_cache"), c.d = dim32(d, "k_cache");
    return c;
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
    PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (!r) throw Raised{};
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) {
        PyObject* w = THPVariable_Wrap(t);
        if (!w) {
            Py_DECREF(r);
            throw Raised{};
        }
        PyTuple_SET_ITEM(r, i++, w);
    }
    return r;
}

// new_tokens, lens, block_table, free_pages, free_count, page_size, max_tokens
PyObject* tables_step(PyObject* const* a) {
    const at::Tensor& nt = tensor(a[0], "new_tokens");
    const at::Tensor& bt = tensor(a[2], "block_table");
    const at::Tensor& fp = tensor(a[3], "free_pages");
    const int dev = device_of(nt, "new_tokens");
    if (nt.dim() != 1) refuse(PyExc_ValueError, "new_tokens", "must be [B]");
    if (bt.dim() != 2) refuse(PyExc_ValueError, "block_table", "must be [B, max_pages]");
    if (fp.dim() != 1) refuse(PyExc_ValueError, "free_pages", "must be [capacity]");
    const int64_t B = nt.size(0), M = bt.size(1);
    const int P = integer(a[5], "page_size"), T = integer(a[6], "max_tokens");
    if (T < 0) refuse(PyExc_ValueError, "max_tokens", "must not be negative");
    const int* new_tokens = need<int>(a[0], "new_tokens", at::kInt, {B}, dev);
    const int* lens = need<int>(a[1], "lens", at::kInt, {B}, dev);
    int* table = need<int>(a[2], "block_table", at::kInt, {B, M}, dev);
    int* free_pages = need<int>(a[3], "free_pages", at::kInt, fp.sizes(), dev);
    const int* count = need<int>(a[4], "free_count", at::kInt, {1}, dev);
    c10::cuda::OptionalCUDAGuard guard;
    guard.set_index(static_cast<c10::DeviceIndex>(dev));
    // one allocation for the five outputs
    const at::Tensor all = empty({T + 2 * B + 3}, at::kInt, dev);
    int64_t used = 0;
    auto part = [&](int64_t n) {
        auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
        impl->set_storage_offset(used);
        impl->set_sizes_contiguous({n});
        used += n;
        return at::Tensor(std::move(impl));
    };
    at::Tensor slots = part(T), cu = part(B + 1), lens_out = part(B), count_out = part(1), status = part(1);
    auto at_int = [](at::Tensor& t) { return static_cast<int*>(t.data_ptr()); };
    const int st = fa_kv_tables_step(new_tokens, lens, table, free_pages, count, dim32(B, "new_tokens"), dim32(M, "block_table"),
                                     dim32(fp.size(0), "free_pages"), P, T, at_int(slots), at_int(cu), at_int(lens_out),
                                     at_int(count_out), at_int(status), stream_of(dev));
    if (st != FA_OK) return PyLong_FromLong(st);
    return tuple_of({slots, cu, lens_out, count_out, status});
}

// k, v, slots, k_cache, v_cache, k_scale, v_scale, k_bounds
PyObject* append(PyObject* const* a) {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const int dev = device_of(k, "k"), dtype = dtype_of(k, "k");
    const Strides ks = rows16(k, "k", k.scalar_type(), dev), vs = rows16(v, "v", k.scalar_type(), dev);
    const fa_kv_cache c = cache_of(a[3], a[4], a[5], a[6], a[7], dev);
    const int64_t T = k.size(0);
    if (k.size(1) != c.Hk || k.size(2) != c.d) refuse(PyExc_ValueError, "k", "must be [T, Hk, d] with the cache's Hk and d");
    if (v.sizes() != k.sizes()) refuse(PyExc_ValueError, "v", "must have the shape of k");
    const int* slots = need<int>(a[2], "slots", at::kInt, {T}, dev);
    if (T == 0) Py_RETURN_NONE;
    c10::cuda::OptionalCUDAGuard guard;
    guard.set_index(static_cast<c10::DeviceIndex>(dev));
    const int st = fa_kv_cache_append(&c, k.data_ptr(), v.data_ptr(), slots, dim32(T, "k"), ks.s, vs.s, dtype, stream_of(dev));
    if (st != FA_OK) return PyLong_FromLong(st);
    Py_RETURN_NONE;
}

// q, k_cache, v_cache, k_scale, v_scale, block_table, lens, cu_q, max_q, scale, causal, selected,
// selected_count, out, lse, num_splits, workspace
PyObject* attend(PyObject* const* a) {
    const at::Tensor& q = tensor(a[0], "q");
    const at::Tensor& bt = tensor(a[5], "block_table");
    const int dev = device_of(q, "q");
    fa_paged_args p = {};
    p.dtype = dtype_of(q, "q");
    const Strides qs = rows16(q, "q", q.scalar_type(), dev);
    p.cache = cache_of(a[1], a[2], a[3], a[4], Py_None, dev);
    if (q.size(2) != p.cache.d) refuse(PyExc_ValueError, "q", "must be [T, Hq, d] with the cache's d");
    if (bt.dim() != 2) refuse(PyExc_ValueError, "block_table", "must be [B, max_pages]");
    const int64_t T = q.size(0), Hq = q.size(1), B = bt.size(0), M = bt.size(1);
    p.q = q.data_ptr();
    p.block_table = need<int>(a[5], "block_table", at::kInt, {B, M}, dev);
    p.lens = need<int>(a[6], "lens", at::kInt, {B}, dev);
    p.cu_q = a[7] == Py_None ? nullptr : need<int>(a[7], "cu_q", at::kInt, {B + 1}, dev);
    p.max_q = integer(a[8], "max_q");
    const double scale = PyFloat_AsDouble(a[9]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    p.scale = static_cast<float>(scale);
    p.causal = PyObject_IsTrue(a[10]);
    if (p.causal < 0) throw Raised{};
    if (a[11] != Py_None || a[12] != Py_None) {
        const at::Tensor& sel = tensor(a[11], "selected");
        if (sel.dim() != 3) refuse(PyExc_ValueError, "selected", "must be [B, Hk, keep]");
        p.selected = need<int>(a[11], "selected", at::kInt, {B, p.cache.Hk, sel.size(2)}, dev);
        p.selected_count = need<int>(a[12], "selected_count", at::kInt, {B, p.cache.Hk}, dev);
        p.num_selected = dim32(sel.size(2), "selected");
    }
    p.num_splits = integer(a[15], "num_splits");
    p.T = dim32(T, "q"), p.Hq = dim32(Hq, "q"), p.B = dim32(B, "block_table"), p.max_pages = dim32(M, "block_table");
    p.q_stride[0] = qs.s[0], p.q_stride[1] = qs.s[1];

    c10::cuda::OptionalCUDAGuard guard;
    guard.set_index(static_cast<c10::DeviceIndex>(dev));
    at::Tensor out, lse, ws;
    Strides os = {{Hq * p.cache.d, p.cache.d}};
    if (a[13] == Py_None) {
        out = empty({T, Hq, p.cache.d}, q.scalar_type(), dev);
    } else {
        out = tensor(a[13], "out");
        os = rows16(out, "out", q.scalar_type(), dev);
        if (out.sizes() != q.sizes()) refuse(PyExc_ValueError, "out", "must have the shape of q");
    }
    if (a[14] == Py_None) {
        lse = empty({T, Hq}, at::kFloat, dev);
        p.lse = static_cast<float*>(lse.data_ptr());
    } else {
        p.lse = need<float>(a[14], "lse", at::kFloat, {T, Hq}, dev);
    }
    p.o = out.data_ptr();
    p.o_stride[0] = os.s[0], p.o_stride[1] = os.s[1];
    p.stream = stream_of(dev);
    if (const size_t bytes = fa_paged_workspace_size(&p)) {
        if (a[16] == Py_None) {
            ws = empty({static_cast<int64_t>(bytes)}, at::kByte, dev);
        } else {
            ws = tensor(a[16], "workspace");
            on_device(ws, "workspace", dev);
            if (!ws.is_contiguous()) refuse(PyExc_ValueError, "workspace", "must be contiguous");
        }
        p.workspace = ws.data_ptr();
        p.workspace_bytes = ws.nbytes();
    }
    const int st = fa_paged_fwd(&p);
    if (st != FA_OK) return PyLong_FromLong(st);
    if (a[13] == Py_None && a[14] == Py_None) return tuple_of({out, lse});
    PyObject* wo = a[13] == Py_None ? THPVariable_Wrap(out) : Py_NewRef(a[13]);
    PyObject* wl = a[14] == Py_None ? THPVariable_Wrap(lse) : Py_NewRef(a[14]);
    PyObject* r = wo && wl ? PyTuple_Pack(2, wo, wl) : nullptr;
    Py_XDECREF(wo);
    Py_XDECREF(wl);
    return r;
}

// q, k_bounds, k_scale, block_table, lens, page_size, num_selected
PyObject* page_select(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q"), &bd = tensor(a[1], "k_bounds"), &bt = tensor(a[3], "block_table");
    const int dev = device_of(q, "q"), dtype = dtype_of(q, "q");
    const Strides qs = rows16(q, "q", q.scalar_type(), dev);
    if (bd.dim() != 4) refuse(PyExc_ValueError, "k_bounds", "must be [num_pages, Hk, 2, d]");
    if (bt.dim() != 2) refuse(PyExc_ValueError, "block_table", "must be [B, max_pages]");
    const int64_t N = bd.size(0), H = bd.size(1), d = bd.size(3), B = bt.size(0), M = bt.size(1), Hq = q.size(1);
    if (q.size(0) != B || q.size(2) != d) refuse(PyExc_ValueError, "q", "must be [B, Hq, d]");
    fa_kv_cache c = {};
    c.k_bounds = need<signed char>(a[1], "k_bounds", at::kChar, {N, H, 2, d}, dev);
    c.k_scale = need<float>(a[2], "k_scale", at::kFloat, {N, H}, dev);
    c.num_pages = dim32(N, "k_bounds"), c.Hk = dim32(H, "k_bounds"), c.d = dim32(d, "k_bounds");
    c.page_size = integer(a[5], "page_size");
    const int* table = need<int>(a[3], "block_table", at::kInt, {B, M}, dev);
    const int* lens = need<int>(a[4], "lens", at::kInt, {B}, dev);
    const int keep = integer(a[6], "num_selected");
    if (keep < 1) refuse(PyExc_ValueError, "num_selected", "must be at least 1");
    c10::cuda::OptionalCUDAGuard guard;
    guard.set_index(static_cast<c10::DeviceIndex>(dev));
    at::Tensor sel = empty({B, H, keep}, at::kInt, dev), count = empty({B, H}, at::kInt, dev);
    if (B == 0) return tuple_of({sel, count});
    const int st = fa_kv_page_select(&c, q.data_ptr(), qs.s, table, lens, dim32(B, "block_table"), dim32(Hq, "q"),
                                     dim32(M, "block_table"), keep, dtype, static_cast<int*>(sel.data_ptr()),
                                     static_cast<int*>(count.data_ptr()), stream_of(dev));
    if (st != FA_OK) return PyLong_FromLong(st);
    return tuple_of({sel, count});
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define FA_METHOD(name, f, n) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FA_METHOD("tables_step", tables_step, 7), FA_METHOD("append", append, 8),
                         FA_METHOD("attend", attend, 17), FA_METHOD("page_select", page_select, 7),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding() { return PyModule_Create(&module); }
