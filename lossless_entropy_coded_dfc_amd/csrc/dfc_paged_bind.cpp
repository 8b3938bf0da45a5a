// dfc_paged_bind.cpp - the entry points of the paged cache and of the drafts'
// verification for Python: checks of tensors, allocation of what a call returns,
// and the argument structures of dfc.h.
//
// The kernels of a decoding step run for 4 to 12 us.  Done in Python and ctypes
// this took 9 to 11 us a call beside the launch's 3.6 (an append of 64 tokens
// 12.8 us a call among others, now 5.2; one token over 700 16.3, now 11.4).
// Nothing is computed here and nothing kept between calls.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/detail/CUDAHooksInterface.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <exception>
#include <vector>

#include "dfc.h"

namespace {

// An error that is already set, or is to be, as Python's.
struct Failed {};

[[noreturn]] void type_error(const char *text) {
    PyErr_SetString(PyExc_TypeError, text);
    throw Failed();
}
template <typename... A>
[[noreturn]] void type_error(const char *format, A... a) {
    PyErr_Format(PyExc_TypeError, format, a...);
    throw Failed();
}
template <typename... A>
[[noreturn]] void value_error(const char *format, A... a) {
    PyErr_Format(PyExc_ValueError, format, a...);
    throw Failed();
}

PyObject *g_current_stream;  // torch's: device -> handle
decltype(&dfc_paged_plan) g_plan;
decltype(&dfc_paged_append_normed) g_append;
decltype(&dfc_paged_attention_sinks) g_attention;
decltype(&dfc_paged_attention_workspace) g_workspace;
decltype(&dfc_paged_release) g_release;
decltype(&dfc_paged_fork) g_fork;
decltype(&dfc_paged_compact) g_compact;
decltype(&dfc_paged_compact_workspace) g_compact_workspace;
decltype(&dfc_paged_copy) g_copy;
decltype(&dfc_verify_drafts) g_verify;
decltype(&dfc_verify_workspace) g_verify_workspace;

// None of the operators has a backward pass: a tensor that asks for one is
// refused, or its gradient would be lost without a word.
const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) type_error("%s must be a tensor", name);
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.requires_grad() && c10::GradMode::is_enabled())
        value_error("%s requires a gradient, which the serving operators do not compute: detach it, or call under "
                    "torch.no_grad()",
                    name);
    return t;
}

// A given tensor that the call writes: autograd is told, so that it does not
// use a value saved before as if it still stood.
void written(const at::Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

int64_t integer(PyObject *o, const char *name) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error("%s must be an integer", name);
    }
    return x;
}

// A size that the C structures hold in 32 bits.
uint32_t count(PyObject *o, const char *name) {
    const int64_t x = integer(o, name);
    if (x < 0 || x >= int64_t(1) << 31) value_error("%s must be between 0 and 2^31 - 1", name);
    return uint32_t(x);
}

uint32_t narrow(int64_t x, const char *name) {
    if (x < 0 || x >= int64_t(1) << 31) value_error("%s must be between 0 and 2^31 - 1", name);
    return uint32_t(x);
}

float real(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Failed();
    return float(x);
}

bool truth(PyObject *o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw Failed();
    return x != 0;
}

// The device of the call's main tensor, which must be the current one: the
// launch goes to it.
int64_t device_of(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) type_error("%s must be a device (cuda) tensor", name);
    const int64_t dev = t.get_device();
    if (dev != at::detail::getCUDAHooks().getCurrentDevice())
        value_error("%s is on device %d, not the current one", name, int(dev));
    return dev;
}

bool on(const at::Tensor &t, int64_t dev) { return t.is_cuda() && t.get_device() == dev; }

// A contiguous vector of n elements.
template <typename T>
T *vector(const at::Tensor &t, at::ScalarType type, int64_t n, int64_t dev, const char *name) {
    if (t.scalar_type() != type || t.dim() != 1 || !on(t, dev) || !t.is_contiguous())
        type_error("%s must be a contiguous one-dimensional %s tensor on the call's device", name, at::toString(type));
    if (t.size(0) != n) value_error("%s has %lld elements, not %lld", name, (long long)t.size(0), (long long)n);
    return static_cast<T *>(t.data_ptr());
}

// Rows (tokens, heads, head_dim): any strides of the first two dimensions, the
// last one contiguous.
void *rows(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, int64_t dev,
           int64_t (&stride)[2]) {
    if (t.scalar_type() != type || !on(t, dev) || t.dim() != 3)
        type_error("%s must be a %s tensor of shape (tokens, heads, head_dim) on the call's device", name,
                   at::toString(type));
    if (t.sizes() != shape)
        value_error("%s has shape (%lld, %lld, %lld), not (%lld, %lld, %lld)", name, (long long)t.size(0),
                    (long long)t.size(1), (long long)t.size(2), (long long)shape[0], (long long)shape[1],
                    (long long)shape[2]);
    if (t.stride(2) != 1 && t.size(2) != 1) value_error("the values of a head of %s must be contiguous", name);
    stride[0] = t.stride(0);
    stride[1] = t.stride(1);
    return t.data_ptr();
}

void cache_of(const at::Tensor &k, const at::Tensor &v, int64_t dev, dfc_paged_cache &c) {
    if (k.dim() != 4 || k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type() || !on(k, dev) || !on(v, dev))
        type_error("k_cache and v_cache must be tensors of one shape (pages, page size, heads, head_dim) and one "
                   "type on the call's device");
    if (k.scalar_type() != at::kBFloat16 && k.scalar_type() != at::kHalf)
        type_error("the cache must be bfloat16 or float16");
    if (k.stride(3) != 1 || v.stride(3) != 1) value_error("the values of a head must be contiguous in the cache");
    std::memset(&c, 0, sizeof(c));
    c.k_dev = k.data_ptr();
    c.v_dev = v.data_ptr();
    for (int i = 0; i < 3; ++i) {
        c.k_stride[i] = k.stride(i);
        c.v_stride[i] = v.stride(i);
    }
    c.n_pages = narrow(k.size(0), "the cache's pages");
    c.page_size = narrow(k.size(1), "the cache's page size");
    c.kv_heads = narrow(k.size(2), "the cache's heads");
    c.head_dim = narrow(k.size(3), "the cache's head_dim");
    c.dtype = k.scalar_type() == at::kBFloat16 ? DFC_BF16 : DFC_F16;
}

// A block table of n rows.
int32_t *table_of(const at::Tensor &t, int64_t n, int64_t dev, int64_t &stride, uint32_t &width) {
    if (t.dim() != 2 || t.scalar_type() != at::kInt || !on(t, dev))
        type_error("block_table must be an int32 tensor of shape (requests, pages) on the call's device");
    if (t.size(0) != n) value_error("block_table has %lld rows for %lld requests", (long long)t.size(0), (long long)n);
    if (t.stride(1) != 1 && t.size(1) > 1) value_error("the entries of a row of block_table must be contiguous");
    width = narrow(t.size(1), "the width of block_table");
    stride = n > 1 ? t.stride(0) : t.size(1);  // a single row's stride says nothing
    return static_cast<int32_t *>(t.data_ptr());
}

// Weights of a norm: head_dim values, float32 or of the cache's type.
const void *norm_of(PyObject *o, const char *name, at::ScalarType type, int64_t dim, int64_t dev, uint32_t &dtype) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != at::kFloat && t.scalar_type() != type)
        type_error("%s must be float32 or of the cache's type", name);
    dtype = t.scalar_type() == at::kFloat ? DFC_F32 : type == at::kBFloat16 ? DFC_BF16 : DFC_F16;
    return vector<const void>(t, t.scalar_type(), dim, dev, name);
}

uint32_t *status_of(PyObject *o, int64_t dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, "status");
    if (!on(t, dev) || t.element_size() != 4 || t.numel() < 1)
        value_error("status must be a device tensor of at least one 32-bit element");
    written(t);
    return static_cast<uint32_t *>(t.data_ptr());
}

// The given stream's handle, or torch's current one's.
void *stream_of(PyObject *o, int64_t dev) {
    if (o != Py_None) return reinterpret_cast<void *>(uintptr_t(integer(o, "stream")));
    PyObject *d = PyLong_FromLongLong(dev);
    PyObject *h = d ? PyObject_CallOneArg(g_current_stream, d) : nullptr;
    Py_XDECREF(d);
    if (!h) throw Failed();
    const unsigned long long handle = PyLong_AsUnsignedLongLong(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Failed();
    return reinterpret_cast<void *>(uintptr_t(handle));
}

// A launch may wait for room in the queue: other threads run meanwhile.
template <typename F, typename... A>
dfc_status call(F f, A... args) {
    dfc_status s;
    Py_BEGIN_ALLOW_THREADS
    s = f(args...);
    Py_END_ALLOW_THREADS
    return s;
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

// A vector in a part of an allocation (an allocation takes longer).
at::Tensor part(const at::Tensor &of, at::ScalarType type, int64_t offset, int64_t n) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(of.storage()), of.key_set(),
                                                            c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(offset);
    t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    return t;
}

void want(Py_ssize_t n, Py_ssize_t expected) {
    if (n != expected) type_error("wrong number of arguments");
}

template <typename F>
PyObject *guarded(F &&f) {
    try {
        return f();
    } catch (const Failed &) {
    } catch (const std::exception &e) {  // an allocation's, among others
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// A result with its status: (status, tensors ...).
template <size_t N>
PyObject *answer(dfc_status s, const at::Tensor (&t)[N]) {
    PyObject *r = PyTuple_New(N + 1);
    if (!r) throw Failed();
    PyTuple_SET_ITEM(r, 0, PyLong_FromLong(s));
    for (size_t i = 0; i < N; ++i) {
        PyObject *x = t[i].defined() ? THPVariable_Wrap(t[i]) : Py_NewRef(Py_None);
        PyTuple_SET_ITEM(r, Py_ssize_t(i) + 1, x);
        if (!x) {
            Py_DECREF(r);
            throw Failed();
        }
    }
    return r;
}

template <typename F>
void address(F &f, PyObject *o) {
    f = reinterpret_cast<F>(uintptr_t(integer(o, "address")));
}

// setup(current_stream, addresses ...): torch's function for the current
// stream and where dfc.h's functions are, in the order below
PyObject *setup(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        want(n, 12);
        Py_INCREF(a[0]);
        PyObject *before = g_current_stream;
        g_current_stream = a[0];
        Py_XDECREF(before);
        address(g_plan, a[1]);
        address(g_append, a[2]);
        address(g_attention, a[3]);
        address(g_workspace, a[4]);
        address(g_release, a[5]);
        address(g_fork, a[6]);
        address(g_compact, a[7]);
        address(g_compact_workspace, a[8]);
        address(g_copy, a[9]);
        address(g_verify, a[10]);
        address(g_verify_workspace, a[11]);
        Py_RETURN_NONE;
    });
}

// plan(context_lens, new_lens, block_table, free_pages, cursor, page_size,
//      tokens, out or None, status or None, stream)
PyObject *plan(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        want(n_args, 10);
        const at::Tensor &context = tensor(a[0], "context_lens"), &table = tensor(a[2], "block_table");
        const at::Tensor &ring = tensor(a[3], "free_pages");
        const int64_t dev = device_of(table, "block_table");
        const int64_t n = context.dim() == 1 ? context.size(0) : -1;
        dfc_plan_args p;
        std::memset(&p, 0, sizeof(p));
        p.block_table = table_of(table, n, dev, p.table_stride, p.max_pages);
        p.n_requests = narrow(n, "requests");
        p.page_size = count(a[5], "page_size");
        const int64_t tokens = p.tokens = count(a[6], "tokens");
        p.context_lens = vector<int32_t>(context, at::kInt, n, dev, "context_lens");
        p.new_lens = vector<int32_t>(tensor(a[1], "new_lens"), at::kInt, n, dev, "new_lens");
        p.free_pages = vector<int32_t>(ring, at::kInt, ring.dim() == 1 ? ring.size(0) : -1, dev, "free_pages");
        p.n_ring = narrow(ring.size(0), "the length of free_pages");
        p.cursor = vector<int64_t>(tensor(a[4], "cursor"), at::kLong, 2, dev, "cursor");
        p.status_dev = status_of(a[8], dev);
        at::Tensor t[5];  // seq_lens, cu_q, slots, positions, cursor
        if (a[7] == Py_None) {
            const int64_t wide = tokens + 2;  // 64-bit elements, first
            const at::Tensor all = make({8 * wide + 4 * (2 * n + 1 + tokens)}, at::kByte, table);
            t[2] = part(all, at::kLong, 0, tokens);
            t[4] = part(all, at::kLong, tokens, 2);
            t[0] = part(all, at::kInt, 2 * wide, n);
            t[1] = part(all, at::kInt, 2 * wide + n, n + 1);
            t[3] = part(all, at::kInt, 2 * wide + 2 * n + 1, tokens);
        } else {
            if (!PyTuple_Check(a[7]) || PyTuple_GET_SIZE(a[7]) != 5) type_error("out must be a PagedPlan");
            for (int i = 0; i < 5; ++i) written(t[i] = tensor(PyTuple_GET_ITEM(a[7], i), "a field of out"));
        }
        p.seq_lens = vector<int32_t>(t[0], at::kInt, n, dev, "the plan's seq_lens");
        p.cu_q = vector<int32_t>(t[1], at::kInt, n + 1, dev, "the plan's cu_q");
        p.slots = vector<int64_t>(t[2], at::kLong, tokens, dev, "the plan's slots");
        p.positions = vector<int32_t>(t[3], at::kInt, tokens, dev, "the plan's positions");
        p.cursor_out = vector<int64_t>(t[4], at::kLong, 2, dev, "the plan's cursor");
        written(table);
        return answer(call(g_plan, &p, stream_of(a[9], dev)), t);
    });
}

// append(k, v, k_cache, v_cache, slots, q or None, q_out or None, positions or
//        None, rotary or None, interleaved, status or None, q_norm or None,
//        k_norm or None, eps, stream)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        want(n_args, 15);
        const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
        const at::Tensor &kc = tensor(a[2], "k_cache"), &vc = tensor(a[3], "v_cache");
        const int64_t dev = device_of(kc, "k_cache");
        dfc_append_args p;
        std::memset(&p, 0, sizeof(p));
        cache_of(kc, vc, dev, p.cache);
        const at::ScalarType source = k.scalar_type(), type = kc.scalar_type();
        if (source != at::kFloat && source != type) type_error("k and v must be float32 or of the cache's type");
        const int64_t tokens = k.dim() ? k.size(0) : 0, dim = p.cache.head_dim;
        p.tokens = uint64_t(tokens);
        const int64_t shape[3] = {tokens, p.cache.kv_heads, dim};
        p.k_dev = rows(k, "k", source, shape, dev, p.k_src_stride);
        p.v_dev = rows(v, "v", source, shape, dev, p.v_src_stride);
        p.slots = vector<int64_t>(tensor(a[4], "slots"), at::kLong, tokens, dev, "slots");
        p.source_dtype = source == at::kFloat ? DFC_F32 : p.cache.dtype;
        at::Tensor out[1];
        if (a[5] != Py_None) {
            const at::Tensor &q = tensor(a[5], "q");
            if (q.dim() != 3 || q.size(0) != tokens || q.size(2) != dim) value_error("q must have k's tokens and head_dim");
            p.q_heads = narrow(q.size(1), "the heads of q");
            p.q_dev = rows(q, "q", source, q.sizes(), dev, p.q_stride);
            out[0] = a[6] == Py_None ? make(q.sizes(), type, q) : tensor(a[6], "q_out");
            p.q_out_dev = rows(out[0], "q_out", type, q.sizes(), dev, p.q_out_stride);
            written(out[0]);
        }
        if (a[8] != Py_None) {
            const at::Tensor &angles = tensor(a[8], "rotary");
            if (angles.scalar_type() != at::kFloat || angles.dim() != 2 || !on(angles, dev) || !angles.is_contiguous())
                type_error("rotary must be a contiguous float32 tensor of shape (positions, rot_dim) on the call's "
                           "device");
            if (a[7] == Py_None) value_error("rotary needs positions");
            p.max_positions = narrow(angles.size(0), "the positions of rotary");
            p.rot_dim = narrow(angles.size(1), "the rot_dim of rotary");
            p.positions = vector<int32_t>(tensor(a[7], "positions"), at::kInt, tokens, dev, "positions");
            p.rotary_dev = static_cast<float *>(angles.data_ptr());
        }
        p.interleaved = truth(a[9]) ? 1u : 0u;
        p.status_dev = status_of(a[10], dev);
        dfc_norm_args norms;
        std::memset(&norms, 0, sizeof(norms));
        if (a[11] != Py_None && a[5] == Py_None) value_error("q_norm needs q");
        norms.q_norm_dev = norm_of(a[11], "q_norm", type, dim, dev, norms.dtype);
        norms.k_norm_dev = norm_of(a[12], "k_norm", type, dim, dev, norms.dtype);
        const bool both = norms.q_norm_dev && norms.k_norm_dev;
        if (both && tensor(a[11], "q_norm").scalar_type() != tensor(a[12], "k_norm").scalar_type())
            type_error("q_norm and k_norm must be of one type");
        norms.eps = real(a[13]);
        const bool normed = norms.q_norm_dev || norms.k_norm_dev;
        written(kc);
        written(vc);
        return answer(call(g_append, &p, normed ? &norms : nullptr, stream_of(a[14], dev)), out);
    });
}

void sizes_of(const at::Tensor &q, int64_t n, int64_t width, PyObject *max_q_len, dfc_attention_args &p) {
    p.heads = narrow(q.size(1), "the heads of q");
    p.n_requests = narrow(n, "requests");
    p.max_pages = narrow(width, "the width of block_table");
    p.max_q_len = count(max_q_len, "max_q_len");
    p.tokens = uint64_t(q.size(0));
}

// attention(q, k_cache, v_cache, block_table, cu_q, seq_lens, scale or None,
//           causal, window, max_q_len, out or None, lse: None, True or a
//           tensor, workspace or None, status or None, sinks, stream)
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        want(n_args, 16);
        const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &lens = tensor(a[5], "seq_lens");
        const int64_t dev = device_of(q, "q");
        dfc_attention_args p;
        std::memset(&p, 0, sizeof(p));
        cache_of(kc, tensor(a[2], "v_cache"), dev, p.cache);
        const at::ScalarType type = q.scalar_type();
        if (type != kc.scalar_type() || q.dim() != 3)
            type_error("q must be a tensor of shape (tokens, heads, head_dim) of the cache's type");
        const at::IntArrayRef shape = q.sizes();
        if (shape[2] != int64_t(p.cache.head_dim) || !shape[1] || !p.cache.kv_heads || shape[1] % p.cache.kv_heads)
            value_error("q must have the cache's head_dim and a multiple of its heads");
        const int64_t n = lens.dim() == 1 ? lens.size(0) : -1;
        p.block_table = table_of(tensor(a[3], "block_table"), n, dev, p.table_stride, p.max_pages);
        sizes_of(q, n, p.max_pages, a[9], p);
        p.causal = truth(a[7]) ? 1u : 0u;
        p.window = count(a[8], "window");
        const uint32_t sinks = count(a[14], "sinks");
        if (a[6] == Py_None) {
            p.scale = float(1.0 / std::sqrt(double(shape[2])));
        } else {
            p.scale = real(a[6]);
        }
        p.q_dev = rows(q, "q", type, shape, dev, p.q_stride);
        p.cu_q = vector<int32_t>(tensor(a[4], "cu_q"), at::kInt, n + 1, dev, "cu_q");
        p.seq_lens = vector<int32_t>(lens, at::kInt, n, dev, "seq_lens");
        at::Tensor t[2];  // out, lse
        t[0] = a[10] == Py_None ? make(shape, type, q) : tensor(a[10], "out");
        p.out_dev = rows(t[0], "out", type, shape, dev, p.out_stride);
        written(t[0]);
        if (a[11] == Py_True) {
            t[1] = make(shape.slice(0, 2), at::kFloat, q);
        } else if (a[11] != Py_None) {
            t[1] = tensor(a[11], "lse");
            if (t[1].scalar_type() != at::kFloat || t[1].sizes() != shape.slice(0, 2) || !on(t[1], dev) ||
                !t[1].is_contiguous())
                type_error("lse must be a contiguous float32 tensor of shape (tokens, heads) on the call's device");
        }
        if (t[1].defined()) {
            written(t[1]);
            p.lse_dev = static_cast<float *>(t[1].data_ptr());
        }
        at::Tensor work;
        if (a[12] == Py_None) {
            uint64_t bytes = 0;
            const dfc_status s = g_workspace(&p, &bytes);
            if (s != DFC_OK) return answer(s, t);
            work = make({int64_t(bytes)}, at::kByte, q);
        } else {
            work = tensor(a[12], "workspace");
            if (!on(work, dev) || !work.is_contiguous())
                type_error("workspace must be a contiguous tensor on the call's device");
            written(work);
        }
        p.workspace_dev = work.data_ptr();
        p.workspace_bytes = uint64_t(work.nbytes());
        p.status_dev = status_of(a[13], dev);
        return answer(call(g_attention, &p, sinks, stream_of(a[15], dev)), t);
    });
}

// workspace(q, k_cache, v_cache, block_table, seq_lens, max_q_len) ->
// (status, bytes)
PyObject *workspace(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        want(n_args, 6);
        const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &table = tensor(a[3], "block_table");
        const at::Tensor &lens = tensor(a[4], "seq_lens");
        dfc_attention_args p;
        std::memset(&p, 0, sizeof(p));
        cache_of(kc, tensor(a[2], "v_cache"), device_of(q, "q"), p.cache);
        if (q.dim() != 3 || table.dim() != 2 || lens.dim() != 1)
            type_error("q, block_table and seq_lens must have 3, 2 and 1 dimensions");
        sizes_of(q, lens.size(0), table.size(1), a[5], p);
        p.scale = 1.0f;
        uint64_t bytes = 0;
        const dfc_status s = g_workspace(&p, &bytes);
        return Py_BuildValue("iK", int(s), static_cast<unsigned long long>(bytes));
    });
}

// The cursor of a ring, the ring and the holders.
template <typename A>
void pool_of(PyObject *ring, PyObject *cursor, PyObject *shared, int64_t dev, A &p) {
    const at::Tensor &r = tensor(ring, "free_pages"), &s = tensor(shared, "shared");
    p.free_pages = vector<int32_t>(r, at::kInt, r.dim() == 1 ? r.size(0) : -1, dev, "free_pages");
    p.n_ring = narrow(r.size(0), "the length of free_pages");
    p.cursor = vector<int64_t>(tensor(cursor, "cursor"), at::kLong, 2, dev, "cursor");
    p.shared = vector<int32_t>(s, at::kInt, s.dim() == 1 ? s.size(0) : -1, dev, "shared");
    p.n_pages = narrow(s.size(0), "the length of shared");
}

// release(held_lens, keep_lens, block_table, free_pages, cursor, shared,
//         page_size, window, sinks, out or None, status or None, stream)
PyObject *release(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        want(n_args, 12);
        const at::Tensor &held = tensor(a[0], "held_lens"), &table = tensor(a[2], "block_table");
        const int64_t dev = device_of(table, "block_table");
        const int64_t n = held.dim() == 1 ? held.size(0) : -1;
        dfc_release_args p;
        std::memset(&p, 0, sizeof(p));
        p.block_table = table_of(table, n, dev, p.table_stride, p.max_pages);
        p.n_requests = narrow(n, "requests");
        p.held_lens = vector<int32_t>(held, at::kInt, n, dev, "held_lens");
        p.keep_lens = vector<int32_t>(tensor(a[1], "keep_lens"), at::kInt, n, dev, "keep_lens");
        pool_of(a[3], a[4], a[5], dev, p);
        p.page_size = count(a[6], "page_size");
        p.window = count(a[7], "window");
        p.sinks = count(a[8], "sinks");
        p.status_dev = status_of(a[10], dev);
        // the workspace, and the new cursor before it
        const at::Tensor all = make({16 + DFC_RELEASE_WORKSPACE}, at::kByte, table);
        at::Tensor t[1];
        if (a[9] == Py_None)
            t[0] = part(all, at::kLong, 0, 2);
        else
            written(t[0] = tensor(a[9], "out"));
        p.cursor_out = vector<int64_t>(t[0], at::kLong, 2, dev, "out");
        p.workspace_dev = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(all.data_ptr()) + 16);
        written(table);
        written(tensor(a[3], "free_pages"));
        written(tensor(a[5], "shared"));
        return answer(call(g_release, &p, stream_of(a[11], dev)), t);
    });
}

// fork(context_lens, parents, block_table, free_pages, cursor, shared,
//      page_size, fork_lens or None, out or None, status or None, stream)
PyObject *fork(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        want(n_args, 11);
        const at::Tensor &context = tensor(a[0], "context_lens"), &table = tensor(a[2], "block_table");
        const int64_t dev = device_of(table, "block_table");
        const int64_t n = context.dim() == 1 ? context.size(0) : -1;
        dfc_fork_args p;
        std::memset(&p, 0, sizeof(p));
        p.block_table = table_of(table, n, dev, p.table_stride, p.max_pages);
        p.n_requests = narrow(n, "requests");
        p.context_lens = vector<int32_t>(context, at::kInt, n, dev, "context_lens");
        p.parents = vector<int32_t>(tensor(a[1], "parents"), at::kInt, n, dev, "parents");
        pool_of(a[3], a[4], a[5], dev, p);
        p.page_size = count(a[6], "page_size");
        if (a[7] != Py_None) p.fork_lens = vector<int32_t>(tensor(a[7], "fork_lens"), at::kInt, n, dev, "fork_lens");
        p.status_dev = status_of(a[9], dev);
        at::Tensor t[4];  // context_lens, src, dst, cursor
        if (a[8] == Py_None) {
            const at::Tensor all = make({16 + 12 * n}, at::kByte, table);
            t[3] = part(all, at::kLong, 0, 2);
            for (int i = 0; i < 3; ++i) t[i] = part(all, at::kInt, 4 + i * n, n);
        } else {
            if (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 4) type_error("out must be a PagedFork");
            for (int i = 0; i < 4; ++i) written(t[i] = tensor(PyTuple_GET_ITEM(a[8], i), "a field of out"));
        }
        p.context_out = vector<int32_t>(t[0], at::kInt, n, dev, "the fork's context_lens");
        p.src = vector<int32_t>(t[1], at::kInt, n, dev, "the fork's src");
        p.dst = vector<int32_t>(t[2], at::kInt, n, dev, "the fork's dst");
        p.cursor_out = vector<int64_t>(t[3], at::kLong, 2, dev, "the fork's cursor");
        written(table);
        written(tensor(a[5], "shared"));
        return answer(call(g_fork, &p, stream_of(a[10], dev)), t);
    });
}

// compact(context_lens, block_table, free_pages, cursor, shared, page_size,
//         out or None, status or None, stream)
PyObject *compact(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        want(n_args, 9);
        const at::Tensor &context = tensor(a[0], "context_lens"), &table = tensor(a[1], "block_table");
        const int64_t dev = device_of(table, "block_table");
        const int64_t n = context.dim() == 1 ? context.size(0) : -1;
        dfc_compact_args p;
        std::memset(&p, 0, sizeof(p));
        p.block_table = table_of(table, n, dev, p.table_stride, p.max_pages);
        p.n_requests = narrow(n, "requests");
        p.context_lens = vector<int32_t>(context, at::kInt, n, dev, "context_lens");
        pool_of(a[2], a[3], a[4], dev, p);
        p.page_size = count(a[5], "page_size");
        p.status_dev = status_of(a[7], dev);
        const int64_t half = p.n_pages / 2;
        at::Tensor t[3];  // src, dst, used
        if (a[6] == Py_None) {
            const at::Tensor all = make({2 * half + 1}, at::kInt, table);
            t[0] = part(all, at::kInt, 0, half);
            t[1] = part(all, at::kInt, half, half);
            t[2] = part(all, at::kInt, 2 * half, 1);
        } else {
            if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 3) type_error("out must be a PagedMoves");
            for (int i = 0; i < 3; ++i) written(t[i] = tensor(PyTuple_GET_ITEM(a[6], i), "a field of out"));
        }
        p.src = vector<int32_t>(t[0], at::kInt, half, dev, "the moves' src");
        p.dst = vector<int32_t>(t[1], at::kInt, half, dev, "the moves' dst");
        p.used = vector<int32_t>(t[2], at::kInt, 1, dev, "the moves' used");
        const at::Tensor work = make({int64_t(g_compact_workspace(p.n_pages))}, at::kByte, table);
        p.workspace_dev = static_cast<uint32_t *>(work.data_ptr());
        written(table);
        written(tensor(a[2], "free_pages"));
        written(tensor(a[4], "shared"));
        return answer(call(g_compact, &p, stream_of(a[8], dev)), t);
    });
}

// copy(caches, src, dst, status or None, stream): caches a sequence of pairs
PyObject *copy(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        want(n_args, 5);
        const at::Tensor &src = tensor(a[1], "src");
        const int64_t dev = device_of(src, "src");
        const int64_t n = src.dim() == 1 ? src.size(0) : -1;
        const int32_t *from = vector<int32_t>(src, at::kInt, n, dev, "src");
        const int32_t *to = vector<int32_t>(tensor(a[2], "dst"), at::kInt, n, dev, "dst");
        uint32_t *status = status_of(a[3], dev);
        struct Items {  // released however the call ends
            PyObject *of;
            ~Items() { Py_XDECREF(of); }
        };
        const Items all{PySequence_Fast(a[0], "caches must be a sequence of pairs (k_cache, v_cache)")};
        if (!all.of) throw Failed();
        std::vector<dfc_paged_cache> caches(size_t(PySequence_Fast_GET_SIZE(all.of)));
        std::vector<at::Tensor> tensors;
        for (size_t i = 0; i < caches.size(); ++i) {
            const Items pair{PySequence_Fast(PySequence_Fast_GET_ITEM(all.of, Py_ssize_t(i)),
                                             "a cache must be a pair (k_cache, v_cache)")};
            if (!pair.of) throw Failed();
            if (PySequence_Fast_GET_SIZE(pair.of) != 2) type_error("a cache must be a pair (k_cache, v_cache)");
            const at::Tensor &k = tensor(PySequence_Fast_GET_ITEM(pair.of, 0), "k_cache");
            const at::Tensor &v = tensor(PySequence_Fast_GET_ITEM(pair.of, 1), "v_cache");
            cache_of(k, v, dev, caches[i]);
            tensors.push_back(k);
            tensors.push_back(v);
        }
        for (const at::Tensor &t : tensors) written(t);
        const at::Tensor none[1];
        return answer(call(g_copy, caches.data(), uint32_t(caches.size()), from, to, narrow(n, "the length of src"), status,
                           stream_of(a[4], dev)),
                      none);
    });
}

uint32_t type_of(const at::Tensor &t, const char *name) {
    switch (t.scalar_type()) {
        case at::kFloat: return DFC_F32;
        case at::kBFloat16: return DFC_BF16;
        case at::kHalf: return DFC_F16;
        default: type_error("%s must be float32, bfloat16 or float16", name);
    }
}

// Rows of logits.
const void *logits_of(const at::Tensor &t, const char *name, int64_t dev, int64_t &stride) {
    if (t.dim() != 2 || !on(t, dev)) type_error("%s must be a tensor of shape (rows, vocabulary) on the call's device", name);
    if (t.stride(1) != 1 && t.size(1) > 1) value_error("the values of a row of %s must be contiguous", name);
    stride = t.size(0) > 1 ? t.stride(0) : t.size(1);  // a single row's stride says nothing
    return t.data_ptr();
}

void verify_sizes(const at::Tensor &logits, const at::Tensor &cu, dfc_verify_args &p) {
    if (logits.dim() != 2) type_error("logits must be a tensor of shape (rows, vocabulary)");
    if (cu.dim() != 1 || cu.size(0) < 1) type_error("cu_rows must be a one-dimensional tensor of requests + 1 elements");
    p.rows = uint64_t(logits.size(0));
    p.vocab = narrow(logits.size(1), "the vocabulary");
    p.n_requests = narrow(cu.size(0) - 1, "requests");
    p.dtype = type_of(logits, "logits");
}

// verify(logits, cu_rows, drafts, uniforms, draft_logits or None, temperature
//        or None, out or None, workspace or None, status or None, stream)
PyObject *verify(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        want(n_args, 10);
        const at::Tensor &logits = tensor(a[0], "logits"), &cu = tensor(a[1], "cu_rows");
        const int64_t dev = device_of(logits, "logits");
        dfc_verify_args p;
        std::memset(&p, 0, sizeof(p));
        verify_sizes(logits, cu, p);
        const int64_t rows = logits.size(0), n = p.n_requests;
        p.logits_dev = logits_of(logits, "logits", dev, p.logits_stride);
        if (a[4] != Py_None) {
            const at::Tensor &draft = tensor(a[4], "draft_logits");
            if (draft.scalar_type() != logits.scalar_type()) type_error("draft_logits must be of the type of logits");
            if (draft.dim() != 2 || draft.sizes() != logits.sizes()) value_error("draft_logits must have the shape of logits");
            p.draft_logits_dev = logits_of(draft, "draft_logits", dev, p.draft_stride);
        }
        p.cu_rows = vector<int32_t>(cu, at::kInt, n + 1, dev, "cu_rows");
        p.drafts = vector<int64_t>(tensor(a[2], "drafts"), at::kLong, rows, dev, "drafts");
        p.uniforms = vector<float>(tensor(a[3], "uniforms"), at::kFloat, rows, dev, "uniforms");
        if (a[5] != Py_None) p.temperature = vector<float>(tensor(a[5], "temperature"), at::kFloat, n, dev, "temperature");
        at::Tensor t[2];  // accepted, tokens
        if (a[6] == Py_None) {
            const at::Tensor all = make({12 * n}, at::kByte, logits);
            t[1] = part(all, at::kLong, 0, n);
            t[0] = part(all, at::kInt, 2 * n, n);
        } else {
            if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 2) type_error("out must be a Verified");
            for (int i = 0; i < 2; ++i) written(t[i] = tensor(PyTuple_GET_ITEM(a[6], i), "a field of out"));
        }
        p.accepted = vector<int32_t>(t[0], at::kInt, n, dev, "accepted");
        p.tokens = vector<int64_t>(t[1], at::kLong, n, dev, "tokens");
        at::Tensor work;
        if (a[7] == Py_None) {
            uint64_t bytes = 0;
            const dfc_status s = g_verify_workspace(&p, &bytes);
            if (s != DFC_OK) return answer(s, t);
            work = make({int64_t(bytes)}, at::kByte, logits);
        } else {
            work = tensor(a[7], "workspace");
            if (!on(work, dev) || !work.is_contiguous())
                type_error("workspace must be a contiguous tensor on the call's device");
            written(work);
        }
        p.workspace_dev = work.data_ptr();
        p.workspace_bytes = uint64_t(work.nbytes());
        p.status_dev = status_of(a[8], dev);
        return answer(call(g_verify, &p, stream_of(a[9], dev)), t);
    });
}

// verify_workspace(logits, cu_rows, draft_logits or None) -> (status, bytes)
PyObject *verify_workspace(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject * {
        want(n_args, 3);
        const at::Tensor &logits = tensor(a[0], "logits");
        dfc_verify_args p;
        std::memset(&p, 0, sizeof(p));
        verify_sizes(logits, tensor(a[1], "cu_rows"), p);
        if (a[2] != Py_None) p.draft_logits_dev = &p;  // (whether there are any)
        uint64_t bytes = 0;
        const dfc_status s = g_verify_workspace(&p, &bytes);
        return Py_BuildValue("iK", int(s), static_cast<unsigned long long>(bytes));
    });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<setup>("setup"),         method<plan>("plan"),       method<append>("append"),
                           method<attention>("attention"), method<workspace>("workspace"), method<release>("release"),
                           method<fork>("fork"),           method<compact>("compact"), method<copy>("copy"),
                           method<verify>("verify"),       method<verify_workspace>("verify_workspace"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() {
    PyObject *m = PyModule_Create(&g_module);
    // the torch whose structures are compiled in: another's may differ
    if (m && PyModule_AddStringConstant(m, "torch_version", DFC_TORCH) < 0) Py_CLEAR(m);
    return m;
}
