// native.cpp -- the Python side of the paged-cache entry points as a CPython module: it takes torch
// tensors, checks them and calls libdspark.  A decoding step makes these calls once a layer, and their
// kernels run for a few microseconds; checking a dozen tensors from Python costs more than that (a plan 10 us a
// call, here 4 us).  Shapes, types and layouts raise ValueError or TypeError before any address is
// taken; the library's own status is returned as a number (0 = ok).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>

#include "dspark.h"

namespace {

struct Refused {};  // the Python error is set

[[noreturn]] void refuse(PyObject* type, const char* text) {
    PyErr_SetString(type, text);
    throw Refused{};
}

const at::Tensor* tensor(PyObject* o) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "expected a torch tensor");
    return &THPVariable_Unpack(o);
}
const at::Tensor& needed(PyObject* o) {
    const at::Tensor* t = tensor(o);
    if (!t) refuse(PyExc_TypeError, "expected a torch tensor, got None");
    return *t;
}

// All of a call's tensors on one device, and that the current one: it is where the library launches.
void one_device(std::initializer_list<const at::Tensor*> tensors) {
    const at::Tensor* first = nullptr;
    for (const at::Tensor* t : tensors) {
        if (!t) continue;
        if (!first) first = t;
        if (t->device() != first->device()) refuse(PyExc_ValueError, "the tensors of a call are on one device");
    }
    if (first && first->is_cuda() && first->device().index() != c10::cuda::current_device())
        refuse(PyExc_ValueError, "the tensors are on another device than the current one");
}

void* address(const at::Tensor* t) {
    if (!t) return nullptr;
    if (!t->is_cuda()) refuse(PyExc_ValueError, "libdspark takes device tensors");
    if (!t->is_contiguous()) refuse(PyExc_ValueError, "libdspark takes contiguous tensors");
    return t->data_ptr();
}
// The last dimension dense; the other strides go along.
void* rows_address(const at::Tensor& t) {
    if (!t.is_cuda()) refuse(PyExc_ValueError, "libdspark takes device tensors");
    if (t.stride(-1) != 1 && t.size(-1) != 1) refuse(PyExc_ValueError, "the last dimension must be dense");
    return t.data_ptr();
}
template <typename T>
T* as(void* p) {
    return static_cast<T*>(p);
}

void want(const at::Tensor* t, at::ScalarType type, int64_t n, const char* text) {
    if (t && (t->scalar_type() != type || t->numel() != n)) refuse(PyExc_ValueError, text);
}

long long number(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}
int small(PyObject* o) {
    const long long v = number(o);
    if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_OverflowError, "a size past 32 bits");
    return (int)v;
}
int size32(int64_t v) {
    if (v > INT32_MAX) refuse(PyExc_OverflowError, "a size past 32 bits");
    return (int)v;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return (float)v;
}
// The stream given as its address, or torch's current stream of the tensors' device.
dspark_stream_t stream_of(PyObject* o, const at::Tensor& t) {
    if (o == Py_None) {
        if (!t.is_cuda()) refuse(PyExc_ValueError, "libdspark takes device tensors");
        return reinterpret_cast<dspark_stream_t>(c10::cuda::getCurrentCUDAStream(t.device().index()).stream());
    }
    return reinterpret_cast<dspark_stream_t>((uintptr_t)number(o));
}

// The caller's word for the first device error of its calls, or none.
int32_t* error_word(PyObject* o) {
    const at::Tensor* t = tensor(o);
    want(t, at::kInt, 1, "error is int32 [1]");
    return as<int32_t>(address(t));
}

int type_code(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return DSPARK_BF16;
        case at::kHalf: return DSPARK_F16;
        case at::kFloat8_e4m3fn: return DSPARK_E4M3;
        default: refuse(PyExc_TypeError, "the paged cache takes bf16, fp16 and e4m3");
    }
}

// Whether an index means the same element of both: one shape, and one stride wherever there is more than one index.
bool same_layout(const at::Tensor& x, const at::Tensor& y) {
    if (x.sizes() != y.sizes()) return false;
    for (int64_t i = 0; i < x.dim(); ++i)
        if (x.size(i) > 1 && x.stride(i) != y.stride(i)) return false;
    return true;
}

struct Pools {
    int pages, page_size, Hk, D;
    int64_t page, token, head;
};
Pools pools_of(const at::Tensor& k, const at::Tensor& v) {
    if (k.dim() != 4 || !same_layout(k, v))
        refuse(PyExc_ValueError, "k_pages and v_pages are [pages, page_size, Hk, D] of one shape and layout");
    if (k.scalar_type() != v.scalar_type()) refuse(PyExc_TypeError, "k_pages and v_pages are of one type");
    return {size32(k.size(0)), size32(k.size(1)), size32(k.size(2)), size32(k.size(3)), k.stride(0), k.stride(1), k.stride(2)};
}
void check_scales(const at::Tensor& pages, const at::Tensor* ks, const at::Tensor* vs, int Hk) {
    if ((ks || vs) && pages.scalar_type() != at::kFloat8_e4m3fn) refuse(PyExc_ValueError, "scales belong to an e4m3 cache");
    want(ks, at::kFloat, Hk, "a scale is fp32 [Hk]");
    want(vs, at::kFloat, Hk, "a scale is fp32 [Hk]");
}

// Pools of an int8 cache and the exponents of its blocks, [pages, Hk, page_size / block] uint8 each.
dspark_block_exponents exponents_of(const at::Tensor& kp, const Pools& x, const at::Tensor& ke, const at::Tensor& ve) {
    if (kp.scalar_type() != at::kChar) refuse(PyExc_TypeError, "k_pages and v_pages are int8");
    if (ke.scalar_type() != at::kByte || ve.scalar_type() != at::kByte || ke.dim() != 3 || !same_layout(ke, ve) ||
        ke.size(0) != x.pages || ke.size(1) != x.Hk || ke.size(2) < 1 || x.page_size % ke.size(2))
        refuse(PyExc_ValueError, "k_exp and v_exp are uint8 [pages, Hk, page_size / block] of one layout");
    if (!ke.is_cuda() || !ve.is_cuda()) refuse(PyExc_ValueError, "libdspark takes device tensors");
    return {static_cast<uint8_t*>(ke.data_ptr()), static_cast<uint8_t*>(ve.data_ptr()), (int)(x.page_size / ke.size(2)),
            ke.stride(0), ke.stride(2), ke.stride(1)};
}

// Runs a call's body; no C++ exception passes into Python.
template <typename F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}
void count_args(Py_ssize_t n, Py_ssize_t wanted) {
    if (n != wanted) refuse(PyExc_TypeError, "wrong number of arguments");
}

dspark_cache_params cache_params(const at::Tensor& cache_len, const at::Tensor& table, const at::Tensor& n_blocks,
                                 const at::Tensor& free_pages, const at::Tensor& n_free, PyObject* page_size,
                                 int max_tokens, PyObject* extra, PyObject* error) {
    if (cache_len.scalar_type() != at::kInt || free_pages.scalar_type() != at::kInt || table.scalar_type() != at::kInt)
        refuse(PyExc_ValueError, "cache_len, free_pages and block_table are int32");
    const int64_t B = cache_len.numel();
    want(&n_blocks, at::kInt, B, "n_blocks is int32 [B]");
    want(&n_free, at::kInt, 1, "n_free is int32 [1]");
    if (table.dim() != 2 || table.size(0) != B) refuse(PyExc_ValueError, "block_table is [B, max_blocks]");
    return {size32(B), small(page_size), size32(free_pages.numel()), size32(table.size(1)), max_tokens, small(extra), error_word(error), nullptr};
}

// cache_len, new_len, block_table, n_blocks, free_pages, n_free, page_size, max_tokens, extra,
// seq_len, offsets, slots, positions, n_blocks_out, n_free_out, workspace, stream, error
PyObject* cache_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        count_args(n, 18);
        const at::Tensor &cache_len = needed(a[0]), &table = needed(a[2]), &n_blocks = needed(a[3]), &free_pages = needed(a[4]),
                         &n_free = needed(a[5]), &seq = needed(a[9]), &off = needed(a[10]), &slots = needed(a[11]),
                         &n_blocks_out = needed(a[13]), &n_free_out = needed(a[14]), &ws = needed(a[15]);
        const at::Tensor *new_len = tensor(a[1]), *positions = tensor(a[12]);
        one_device({&cache_len, new_len, &table, &n_blocks, &free_pages, &n_free, &seq, &off, &slots, positions, &n_blocks_out,
                    &n_free_out, &ws, tensor(a[17])});
        const dspark_cache_params p = cache_params(cache_len, table, n_blocks, free_pages, n_free, a[6], small(a[7]), a[8], a[17]);
        want(new_len, at::kInt, p.B, "new_len is int32 [B]");
        want(&seq, at::kInt, p.B, "seq_len is int32 [B]");
        want(&off, at::kInt, (int64_t)p.B + 1, "offsets is int32 [B + 1]");
        want(&slots, at::kLong, p.max_tokens, "slots is int64 [max_tokens]");
        want(positions, at::kInt, p.max_tokens, "positions is int32 [max_tokens]");
        want(&n_blocks_out, at::kInt, p.B, "n_blocks is int32 [B]");
        want(&n_free_out, at::kInt, 1, "n_free is int32 [1]");
        return PyLong_FromLong(dspark_cache_plan(
            &p, as<int32_t>(address(&cache_len)), as<int32_t>(address(new_len)), as<int32_t>(address(&table)),
            as<int32_t>(address(&n_blocks)), as<int32_t>(address(&free_pages)), as<int32_t>(address(&n_free)),
            as<int32_t>(address(&seq)), as<int32_t>(address(&off)), as<int64_t>(address(&slots)),
            as<int32_t>(address(positions)), as<int32_t>(address(&n_blocks_out)), as<int32_t>(address(&n_free_out)),
            address(&ws), ws.nbytes(), stream_of(a[16], cache_len)));
    });
}

// cache_len, add_len, done, block_table, n_blocks, free_pages, n_free, page_size, extra, cache_len_out,
// n_blocks_out, n_free_out, workspace, stream, error, settled
PyObject* cache_commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        count_args(n, 16);
        const at::Tensor &cache_len = needed(a[0]), &table = needed(a[3]), &n_blocks = needed(a[4]), &free_pages = needed(a[5]),
                         &n_free = needed(a[6]), &len_out = needed(a[9]), &n_blocks_out = needed(a[10]),
                         &n_free_out = needed(a[11]), &ws = needed(a[12]);
        const at::Tensor *add_len = tensor(a[1]), *done = tensor(a[2]), *settled = tensor(a[15]);
        one_device({&cache_len, add_len, done, &table, &n_blocks, &free_pages, &n_free, &len_out, &n_blocks_out, &n_free_out, &ws,
                    tensor(a[14]), settled});
        dspark_cache_params p = cache_params(cache_len, table, n_blocks, free_pages, n_free, a[7], 0, a[8], a[14]);
        want(add_len, at::kInt, p.B, "add_len is int32 [B]");
        want(settled, at::kInt, 2 * (int64_t)p.B + 1, "settled is int32 [2 B + 1]");
        p.settled = as<int32_t>(address(settled));
        if (done && ((done->scalar_type() != at::kByte && done->scalar_type() != at::kBool) || done->numel() != p.B))
            refuse(PyExc_ValueError, "done is uint8 or bool [B]");
        want(&len_out, at::kInt, p.B, "cache_len is int32 [B]");
        want(&n_blocks_out, at::kInt, p.B, "n_blocks is int32 [B]");
        want(&n_free_out, at::kInt, 1, "n_free is int32 [1]");
        return PyLong_FromLong(dspark_cache_commit(
            &p, as<int32_t>(address(&cache_len)), as<int32_t>(address(add_len)), as<uint8_t>(address(done)),
            as<int32_t>(address(&table)), as<int32_t>(address(&n_blocks)), as<int32_t>(address(&free_pages)),
            as<int32_t>(address(&n_free)), as<int32_t>(address(&len_out)), as<int32_t>(address(&n_blocks_out)),
            as<int32_t>(address(&n_free_out)), address(&ws), ws.nbytes(), stream_of(a[13], cache_len)));
    });
}

// k, v, k_pages, v_pages, slots, k_scale, v_scale, stream
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        count_args(n, 8);
        const at::Tensor &k = needed(a[0]), &v = needed(a[1]), &kp = needed(a[2]), &vp = needed(a[3]), &slots = needed(a[4]);
        const at::Tensor *ks = tensor(a[5]), *vs = tensor(a[6]);
        one_device({&k, &v, &kp, &vp, &slots, ks, vs});
        const Pools x = pools_of(kp, vp);
        if (k.dim() != 3 || v.sizes() != k.sizes() || k.size(1) != x.Hk || k.size(2) != x.D ||
            k.scalar_type() != v.scalar_type())
            refuse(PyExc_ValueError, "k and v are [T, Hk, D] of one type");
        want(&slots, at::kLong, k.size(0), "slots is int64 [T]");
        check_scales(kp, ks, vs, x.Hk);
        const dspark_append_params p{size32(k.size(0)), x.Hk,        x.D,         x.page_size, x.pages,     type_code(k.scalar_type()),
                                     type_code(kp.scalar_type()),    k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                                     x.page,            x.token,     x.head};
        return PyLong_FromLong(dspark_cache_append(&p, rows_address(k), rows_address(v), rows_address(kp), rows_address(vp),
                                                   as<int64_t>(address(&slots)), as<float>(address(ks)),
                                                   as<float>(address(vs)), stream_of(a[7], k)));
    });
}

// k, v, k_pages, v_pages, k_exp, v_exp, slots, stream, error
PyObject* cache_append_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        count_args(n, 9);
        const at::Tensor &k = needed(a[0]), &v = needed(a[1]), &kp = needed(a[2]), &vp = needed(a[3]), &ke = needed(a[4]),
                         &ve = needed(a[5]), &slots = needed(a[6]);
        one_device({&k, &v, &kp, &vp, &ke, &ve, &slots, tensor(a[8])});
        const Pools x = pools_of(kp, vp);
        const dspark_block_exponents e = exponents_of(kp, x, ke, ve);
        if (k.dim() != 3 || v.sizes() != k.sizes() || k.size(1) != x.Hk || k.size(2) != x.D || k.scalar_type() != v.scalar_type())
            refuse(PyExc_ValueError, "k and v are [T, Hk, D] of one type");
        want(&slots, at::kLong, k.size(0), "slots is int64 [T]");
        const dspark_append_params p{size32(k.size(0)), x.Hk,     x.D,         x.page_size, x.pages,     type_code(k.scalar_type()),
                                     DSPARK_I8,         k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                                     x.page,            x.token,     x.head};
        return PyLong_FromLong(dspark_cache_append_i8(&p, &e, rows_address(k), rows_address(v), rows_address(kp), rows_address(vp),
                                                      as<int64_t>(address(&slots)), error_word(a[8]), stream_of(a[7], k)));
    });
}

// k_pages, v_pages, k_exp, v_exp, slots, k, v, stream
PyObject* cache_read_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        count_args(n, 8);
        const at::Tensor &kp = needed(a[0]), &vp = needed(a[1]), &ke = needed(a[2]), &ve = needed(a[3]), &slots = needed(a[4]),
                         &k = needed(a[5]), &v = needed(a[6]);
        one_device({&kp, &vp, &ke, &ve, &slots, &k, &v});
        const Pools x = pools_of(kp, vp);
        const dspark_block_exponents e = exponents_of(kp, x, ke, ve);
        const int64_t T = slots.numel();
        if (k.dim() != 3 || v.sizes() != k.sizes() || k.size(0) != T || k.size(1) != x.Hk || k.size(2) != x.D ||
            k.scalar_type() != v.scalar_type())
            refuse(PyExc_ValueError, "k and v are [slots, Hk, D] of one type");
        want(&slots, at::kLong, T, "slots is int64 [T]");
        const int64_t row = (int64_t)x.Hk * x.D;
        const dspark_append_params p{size32(T), x.Hk, x.D, x.page_size, x.pages, type_code(k.scalar_type()), DSPARK_I8,
                                     row,       x.D,  row, x.D,         x.page,  x.token,                    x.head};
        return PyLong_FromLong(dspark_cache_read_i8(&p, &e, rows_address(kp), rows_address(vp), as<int64_t>(address(&slots)),
                                                    address(&k), address(&v), stream_of(a[7], kp)));
    });
}

// q, k_pages, v_pages, block_table, seq_len, offsets, k_scale, v_scale, scale, softcap, causal, window,
// max_new, out, lse, workspace (or None: one is allocated), stream, error.  Returns (status, workspace).
// int8 pools: k_exp and v_exp in the scales' places.
template <bool I8>
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        count_args(n, 18);
        const at::Tensor &q = needed(a[0]), &kp = needed(a[1]), &vp = needed(a[2]), &table = needed(a[3]), &seq = needed(a[4]),
                         &out = needed(a[13]);
        const at::Tensor *off = tensor(a[5]), *ks = tensor(a[6]), *vs = tensor(a[7]), *lse = tensor(a[14]);
        one_device({&q, &kp, &vp, &table, &seq, off, ks, vs, &out, lse, tensor(a[15]), tensor(a[17])});
        const Pools x = pools_of(kp, vp);
        if (q.dim() != 3 || q.size(2) != x.D) refuse(PyExc_ValueError, "q is [T, Hq, D]");
        const int64_t T = q.size(0), B = seq.numel();
        if (seq.scalar_type() != at::kInt || table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != B)
            refuse(PyExc_ValueError, "block_table [B, max_blocks] and seq_len [B] are int32");
        want(off, at::kInt, B + 1, "offsets is int32 [B + 1]");
        dspark_block_exponents e{};
        if (I8)
            e = exponents_of(kp, x, needed(a[6]), needed(a[7]));
        else
            check_scales(kp, ks, vs, x.Hk);
        if (out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type())
            refuse(PyExc_ValueError, "out is [T, Hq, D] of q's type");
        if (lse && (lse->scalar_type() != at::kFloat || lse->dim() != 2 || lse->size(0) != T || lse->size(1) != q.size(1)))
            refuse(PyExc_ValueError, "lse is fp32 [T, Hq]");
        dspark_attention_params p;
        p.T = size32(T);
        p.B = size32(B);
        p.Hq = size32(q.size(1));
        p.Hk = x.Hk;
        p.D = x.D;
        p.page_size = x.page_size;
        p.num_pages = x.pages;
        p.max_blocks = size32(table.size(1));
        p.max_new = small(a[12]);
        p.dtype = type_code(q.scalar_type());
        p.kv_dtype = I8 ? (int)DSPARK_I8 : type_code(kp.scalar_type());
        p.causal = PyObject_IsTrue(a[10]);
        if (p.causal < 0) throw Refused{};
        p.window = small(a[11]);
        p.scale = real(a[8]);
        p.softcap = real(a[9]);
        p.q_token_stride = q.stride(0);
        p.q_head_stride = q.stride(1);
        p.kv_page_stride = x.page;
        p.kv_token_stride = x.token;
        p.kv_head_stride = x.head;
        p.error = error_word(a[17]);
        const dspark_stream_t s = stream_of(a[16], q);
        at::Tensor made;
        const at::Tensor* ws = tensor(a[15]);
        if (!ws) {  // 512-byte aligned, as torch's CUDA allocator gives it
            made = at::empty({(int64_t)dspark_paged_attention_workspace_size(&p) + 256}, q.options().dtype(at::kByte));
            ws = &made;
        }
        const dspark_status st =
            I8 ? dspark_paged_attention_i8(&p, &e, rows_address(q), rows_address(kp), rows_address(vp), as<int32_t>(address(&table)),
                                           as<int32_t>(address(&seq)), as<int32_t>(address(off)), address(&out),
                                           as<float>(address(lse)), address(ws), ws->nbytes(), s)
               : dspark_paged_attention(&p, rows_address(q), rows_address(kp), rows_address(vp), as<int32_t>(address(&table)),
                                        as<int32_t>(address(&seq)), as<int32_t>(address(off)), as<float>(address(ks)),
                                        as<float>(address(vs)), address(&out), as<float>(address(lse)), address(ws),
                                        ws->nbytes(), s);
        return Py_BuildValue("iN", (int)st, made.defined() ? THPVariable_Wrap(made) : (Py_INCREF(a[15]), a[15]));
    });
}

PyMethodDef methods[] = {
    {"cache_plan", (PyCFunction)(void (*)())cache_plan, METH_FASTCALL, nullptr},
    {"cache_commit", (PyCFunction)(void (*)())cache_commit, METH_FASTCALL, nullptr},
    {"cache_append", (PyCFunction)(void (*)())cache_append, METH_FASTCALL, nullptr},
    {"cache_append_i8", (PyCFunction)(void (*)())cache_append_i8, METH_FASTCALL, nullptr},
    {"cache_read_i8", (PyCFunction)(void (*)())cache_read_i8, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void (*)())paged_attention<false>, METH_FASTCALL, nullptr},
    {"paged_attention_i8", (PyCFunction)(void (*)())paged_attention<true>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
