// torch_binding.cpp - torch tensors to the C ABI of include/fa_paged.h, fa_rotary.h and fa_latent.h.
//
// Argument checks, allocation of outputs and workspaces, and the call; the
// functions' documentation is in paged.py, rotary.py and latent.py, their only callers.  A decode step's
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
#include "../../include/fa_latent.h"
#include "../../include/fa_paged.h"
#include "../../include/fa_rotary.h"

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

// True or false of a Python object.
int truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v;
}
float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return static_cast<float>(v);
}
void guard_device(c10::cuda::OptionalCUDAGuard& g, int dev) { g.set_index(static_cast<c10::DeviceIndex>(dev)); }
PyObject* wrap(const at::Tensor& t) {
    PyObject* r = THPVariable_Wrap(t);
    if (!r) throw Raised{};
    return r;
}
// The given output (an object) or the one made here, as the function returns it.
PyObject* given_or(PyObject* o, const at::Tensor& t) { return o == Py_None ? wrap(t) : Py_NewRef(o); }
PyObject* pair_of(PyObject* a, PyObject* b) {
    PyObject* r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
}

fa_rotary rotary_of(PyObject* positions, PyObject* table, PyObject* interleaved, int64_t T, int dev) {
    const at::Tensor& t = tensor(table, "table");
    if (t.dim() != 2) refuse(PyExc_ValueError, "table", "must be [num_positions, dim]");
    fa_rotary r = {};
    r.table = need<float>(table, "table", at::kFloat, t.sizes(), dev);
    r.positions = need<int>(positions, "positions", at::kInt, {T}, dev);
    r.num_positions = dim32(t.size(0), "table"), r.dim = dim32(t.size(1), "table");
    r.interleaved = truth(interleaved);
    return r;
}
// x as a part to turn; its output is `out` (None: a new tensor, left in `made`).
fa_rotary_part part_of(const at::Tensor& x, const char* name, PyObject* out, const char* out_name, at::ScalarType type, int dev, at::Tensor& made) {
    fa_rotary_part p = {};
    const Strides xs = rows16(x, name, type, dev);
    Strides ys;
    if (out == Py_None) {
        made = empty(x.sizes(), type, dev);
        ys = rows16(made, out_name, type, dev);
    } else {
        const at::Tensor& o = tensor(out, out_name);
        ys = rows16(o, out_name, type, dev);
        if (o.sizes() != x.sizes()) refuse(PyExc_ValueError, out_name, "must have the shape of its input");
        // (strides that are used: those of dimensions of one element may differ)
        if (o.data_ptr() == x.data_ptr() && (xs.s[0] != ys.s[0] || xs.s[1] != ys.s[1]) && x.numel() > 0)
            refuse(PyExc_ValueError, out_name, "must be its input or not overlap it");
        made = o;
    }
    p.x = x.data_ptr(), p.y = made.data_ptr(), p.heads = dim32(x.size(1), name);
    for (int i = 0; i < 2; ++i) p.x_stride[i] = xs.s[i], p.y_stride[i] = ys.s[i];
    return p;
}

// q, k, positions, table, interleaved, inverse, q_out, k_out
PyObject* rotary_embed(PyObject* const* a) {
    const at::Tensor& q = tensor(a[0], "q");
    const int dev = device_of(q, "q"), dtype = dtype_of(q, "q");
    rows16(q, "q", q.scalar_type(), dev);
    const int64_t T = q.size(0), d = q.size(2);
    fa_rotary r = rotary_of(a[2], a[3], a[4], T, dev);
    r.inverse = truth(a[5]);
    c10::cuda::OptionalCUDAGuard guard;
    guard_device(guard, dev);
    at::Tensor qo, ko;
    const fa_rotary_part qp = part_of(q, "q", a[6], "q_out", q.scalar_type(), dev, qo);
    fa_rotary_part kp = {};
    const bool two = a[1] != Py_None;
    if (two) {
        const at::Tensor& k = tensor(a[1], "k");
        rows16(k, "k", q.scalar_type(), dev);
        if (k.size(0) != T || k.size(2) != d) refuse(PyExc_ValueError, "k", "must have the tokens and the width of q");
        kp = part_of(k, "k", a[7], "k_out", q.scalar_type(), dev, ko);
    } else if (a[7] != Py_None) {
        refuse(PyExc_ValueError, "k_out", "is given without k");
    }
    const int st = fa_rotary_embed(&r, &qp, two ? &kp : nullptr, dim32(T, "q"), dim32(d, "q"), dtype, stream_of(dev));
    if (st != FA_OK) return PyLong_FromLong(st);
    return pair_of(given_or(a[6], qo), two ? given_or(a[7], ko) : Py_NewRef(Py_None));
}

// q, k, v, positions, table, slots, k_cache, v_cache, k_scale, v_scale, k_bounds, interleaved, q_out
PyObject* append_rotary(PyObject* const* a) {
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const int dev = device_of(k, "k"), dtype = dtype_of(k, "k");
    const Strides ks = rows16(k, "k", k.scalar_type(), dev), vs = rows16(v, "v", k.scalar_type(), dev);
    const fa_kv_cache c = cache_of(a[6], a[7], a[8], a[9], a[10], dev);
    const int64_t T = k.size(0);
    if (k.size(1) != c.Hk || k.size(2) != c.d) refuse(PyExc_ValueError, "k", "must be [T, Hk, d] with the cache's Hk and d");
    if (v.sizes() != k.sizes()) refuse(PyExc_ValueError, "v", "must have the shape of k");
    const int* slots = need<int>(a[5], "slots", at::kInt, {T}, dev);
    const fa_rotary r = rotary_of(a[3], a[4], a[11], T, dev);
    c10::cuda::OptionalCUDAGuard guard;
    guard_device(guard, dev);
    at::Tensor qo;
    fa_rotary_part qp = {};
    const bool with_q = a[0] != Py_None;
    if (with_q) {
        const at::Tensor& q = tensor(a[0], "q");
        rows16(q, "q", k.scalar_type(), dev);
        if (q.size(0) != T || q.size(2) != c.d) refuse(PyExc_ValueError, "q", "must be [T, Hq, d] with the tokens and the width of k");
        qp = part_of(q, "q", a[12], "q_out", k.scalar_type(), dev, qo);
    } else if (a[12] != Py_None) {
        refuse(PyExc_ValueError, "q_out", "is given without q");
    }
    const int st = T == 0 ? FA_OK
                          : fa_kv_cache_append_rotary(&c, k.data_ptr(), v.data_ptr(), slots, dim32(T, "k"), ks.s, vs.s, &r,
                                                      with_q ? &qp : nullptr, dtype, stream_of(dev));
    if (st != FA_OK) return PyLong_FromLong(st);
    return with_q ? given_or(a[12], qo) : Py_NewRef(Py_None);
}

fa_latent_cache latent_cache_of(PyObject* cache, int64_t value_dim, at::ScalarType type, int dev) {
    const at::Tensor& t = tensor(cache, "cache");
    if (t.dim() != 3) refuse(PyExc_ValueError, "cache", "must be [num_pages, page_size, value_dim + rope_dim]");
    fa_latent_cache c = {};
    c.rows = need<>(cache, "cache", type, t.sizes(), dev);
    c.num_pages = dim32(t.size(0), "cache"), c.page_size = dim32(t.size(1), "cache");
    if (value_dim < 0 || value_dim > t.size(2)) refuse(PyExc_ValueError, "cache", "must have rows of at least value_dim channels");
    c.value_dim = static_cast<int>(value_dim), c.rope_dim = dim32(t.size(2), "cache") - c.value_dim;
    return c;
}
// Token stride of a [T, n] tensor with contiguous channels.
long long rows2(const at::Tensor& t, const char* name, at::ScalarType type, int64_t T, int dev) {
    on_device(t, name, dev);
    if (t.dim() != 2 || t.size(0) != T) refuse(PyExc_ValueError, name, "must be [tokens, channels]");
    if (t.scalar_type() != type) refuse(PyExc_TypeError, name, "must have the type of the other 16-bit tensors");
    if (t.stride(1) != 1 && t.size(1) > 1) refuse(PyExc_ValueError, name, "must have a contiguous last dimension");
    return T > 1 ? t.stride(0) : 8;
}

// latent, rope, slots, cache, q_rope, positions, table, interleaved, q_out
PyObject* latent_append(PyObject* const* a) {
    const at::Tensor& latent = tensor(a[0], "latent");
    const int dev = device_of(latent, "latent"), dtype = dtype_of(latent, "latent");
    const at::ScalarType type = latent.scalar_type();
    if (latent.dim() != 2) refuse(PyExc_ValueError, "latent", "must be [T, value_dim]");
    const int64_t T = latent.size(0);
    const long long ls = rows2(latent, "latent", type, T, dev);
    const fa_latent_cache c = latent_cache_of(a[3], latent.size(1), type, dev);
    const void* rope = nullptr;
    long long rs = 8;
    if (a[1] != Py_None) {
        const at::Tensor& t = tensor(a[1], "rope");
        rs = rows2(t, "rope", type, T, dev);
        if (t.size(1) != c.rope_dim) refuse(PyExc_ValueError, "rope", "must have the channels that the cache has behind the latent's");
        rope = t.data_ptr();
    } else if (c.rope_dim != 0) {
        refuse(PyExc_ValueError, "rope", "is missing: the cache's rows are wider than the latent");
    }
    const int* slots = need<int>(a[2], "slots", at::kInt, {T}, dev);
    const bool turned = a[5] != Py_None || a[6] != Py_None, with_q = a[4] != Py_None;
    if (with_q && !turned) refuse(PyExc_ValueError, "q_rope", "is given without positions and table");
    if (!with_q && a[8] != Py_None) refuse(PyExc_ValueError, "q_out", "is given without q_rope");
    c10::cuda::OptionalCUDAGuard guard;
    guard_device(guard, dev);
    fa_rotary r = {};
    if (turned) r = rotary_of(a[5], a[6], a[7], T, dev);
    at::Tensor qo;
    fa_rotary_part qp = {};
    if (with_q) {
        const at::Tensor& q = tensor(a[4], "q_rope");
        rows16(q, "q_rope", type, dev);
        if (q.size(0) != T || q.size(2) != c.rope_dim) refuse(PyExc_ValueError, "q_rope", "must be [T, H, rope_dim]");
        qp = part_of(q, "q_rope", a[8], "q_out", type, dev, qo);
    }
    const int st = fa_latent_cache_append(&c, latent.data_ptr(), ls, rope, rs, slots, dim32(T, "latent"), turned ? &r : nullptr,
                                          with_q ? &qp : nullptr, dtype, stream_of(dev));
    if (st != FA_OK) return PyLong_FromLong(st);
    return with_q ? given_or(a[8], qo) : Py_NewRef(Py_None);
}

// Output [T, H, width] and LSE [T, H], given or new.
struct Outputs {
    at::Tensor out, lse;
    Strides os;
    float* l;
};
Outputs outputs_of(PyObject* out, PyObject* lse, int64_t T, int64_t H, int64_t width, at::ScalarType type, int dev) {
    Outputs r;
    r.os = {{H * width, width}};
    if (out == Py_None) {
        r.out = empty({T, H, width}, type, dev);
    } else {
        r.out = tensor(out, "out");
        r.os = rows16(r.out, "out", type, dev);
        if (r.out.sizes() != at::IntArrayRef({T, H, width})) refuse(PyExc_ValueError, "out", "must be [T, H, value channels]");
    }
    if (lse == Py_None) {
        r.lse = empty({T, H}, at::kFloat, dev);
        r.l = static_cast<float*>(r.lse.data_ptr());
    } else {
        r.l = need<float>(lse, "lse", at::kFloat, {T, H}, dev);
    }
    return r;
}

// q, cache, block_table, lens, value_dim, cu_q, max_q, scale, causal, out, lse, workspace
PyObject* latent_paged(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q"), &bt = tensor(a[2], "block_table");
    const int dev = device_of(q, "q");
    fa_latent_paged_args p = {};
    p.dtype = dtype_of(q, "q");
    const Strides qs = rows16(q, "q", q.scalar_type(), dev);
    p.cache = latent_cache_of(a[1], integer(a[4], "value_dim"), q.scalar_type(), dev);
    const int C = p.cache.value_dim;
    if (q.size(2) != C + p.cache.rope_dim) refuse(PyExc_ValueError, "q", "must be [T, H, width of the cache's rows]");
    if (bt.dim() != 2) refuse(PyExc_ValueError, "block_table", "must be [B, max_pages]");
    const int64_t T = q.size(0), H = q.size(1), B = bt.size(0), M = bt.size(1);
    p.q = q.data_ptr();
    p.block_table = need<int>(a[2], "block_table", at::kInt, {B, M}, dev);
    p.lens = need<int>(a[3], "lens", at::kInt, {B}, dev);
    p.cu_q = a[5] == Py_None ? nullptr : need<int>(a[5], "cu_q", at::kInt, {B + 1}, dev);
    p.max_q = integer(a[6], "max_q");
    p.scale = number(a[7]);
    p.causal = truth(a[8]);
    p.T = dim32(T, "q"), p.H = dim32(H, "q"), p.B = dim32(B, "block_table"), p.max_pages = dim32(M, "block_table");
    p.q_stride[0] = qs.s[0], p.q_stride[1] = qs.s[1];
    c10::cuda::OptionalCUDAGuard guard;
    guard_device(guard, dev);
    const Outputs o = outputs_of(a[9], a[10], T, H, C, q.scalar_type(), dev);
    p.o = o.out.data_ptr(), p.lse = o.l, p.o_stride[0] = o.os.s[0], p.o_stride[1] = o.os.s[1];
    p.stream = stream_of(dev);
    at::Tensor ws;
    if (const size_t bytes = fa_latent_paged_workspace_size(&p)) {
        if (a[11] == Py_None) {
            ws = empty({static_cast<int64_t>(bytes)}, at::kByte, dev);
        } else {
            ws = tensor(a[11], "workspace");
            on_device(ws, "workspace", dev);
            if (!ws.is_contiguous()) refuse(PyExc_ValueError, "workspace", "must be contiguous");
        }
        p.workspace = ws.data_ptr();
        p.workspace_bytes = ws.nbytes();
    }
    const int st = fa_latent_paged_fwd(&p);
    if (st != FA_OK) return PyLong_FromLong(st);
    return pair_of(given_or(a[9], o.out), given_or(a[10], o.lse));
}

// q, k, k_rope, v, cu_q, cu_k, max_q, max_k, scale, causal, out, lse
PyObject* latent_fwd(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &kr = tensor(a[2], "k_rope"), &v = tensor(a[3], "v");
    const at::Tensor& cq = tensor(a[4], "cu_q");
    const int dev = device_of(q, "q");
    const at::ScalarType type = q.scalar_type();
    fa_latent_args p = {};
    p.dtype = dtype_of(q, "q");
    const Strides qs = rows16(q, "q", type, dev), ks = rows16(k, "k", type, dev), vs = rows16(v, "v", type, dev);
    const int64_t T = q.size(0), H = q.size(1), Tk = k.size(0);
    p.k_rope_stride = rows2(kr, "k_rope", type, Tk, dev);
    if (k.size(1) != H) refuse(PyExc_ValueError, "k", "must have the heads of q");
    if (q.size(2) != k.size(2) + kr.size(1)) refuse(PyExc_ValueError, "q", "must have the channels of k and k_rope together");
    if (v.size(0) != Tk || v.size(1) != H) refuse(PyExc_ValueError, "v", "must have the tokens and heads of k");
    if (cq.dim() != 1 || cq.size(0) < 1) refuse(PyExc_ValueError, "cu_q", "must be [B + 1]");
    const int64_t B = cq.size(0) - 1;
    p.cu_q = need<int>(a[4], "cu_q", at::kInt, {B + 1}, dev);
    p.cu_k = need<int>(a[5], "cu_k", at::kInt, {B + 1}, dev);
    p.q = q.data_ptr(), p.k = k.data_ptr(), p.k_rope = kr.data_ptr(), p.v = v.data_ptr();
    p.max_q = integer(a[6], "max_q"), p.max_k = integer(a[7], "max_k");
    p.scale = number(a[8]);
    p.causal = truth(a[9]);
    p.T = dim32(T, "q"), p.Tk = dim32(Tk, "k"), p.B = dim32(B, "cu_q"), p.H = dim32(H, "q");
    p.Dn = dim32(k.size(2), "k"), p.R = dim32(kr.size(1), "k_rope"), p.Dv = dim32(v.size(2), "v");
    for (int i = 0; i < 2; ++i) p.q_stride[i] = qs.s[i], p.k_stride[i] = ks.s[i], p.v_stride[i] = vs.s[i];
    c10::cuda::OptionalCUDAGuard guard;
    guard_device(guard, dev);
    const Outputs o = outputs_of(a[10], a[11], T, H, p.Dv, type, dev);
    p.o = o.out.data_ptr(), p.lse = o.l, p.o_stride[0] = o.os.s[0], p.o_stride[1] = o.os.s[1];
    p.stream = stream_of(dev);
    if (Tk == 0 && T > 0) {  // no key has an address; nothing is read from these
        p.k = p.k_rope = p.v = p.q;
    }
    const int st = fa_latent_fwd(&p);
    if (st != FA_OK) return PyLong_FromLong(st);
    return pair_of(given_or(a[10], o.out), given_or(a[11], o.lse));
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
                         FA_METHOD("rotary_embed", rotary_embed, 8), FA_METHOD("append_rotary", append_rotary, 13),
                         FA_METHOD("latent_append", latent_append, 9), FA_METHOD("latent_paged", latent_paged, 12),
                         FA_METHOD("latent_fwd", latent_fwd, 12),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding() { return PyModule_Create(&module); }
