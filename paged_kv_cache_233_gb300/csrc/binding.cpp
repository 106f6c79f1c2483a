// binding.cpp -- Python entry points of the 4-bit cache and of
// paged_kv_build_tables: tensors checked and unpacked in C++, then the C ABI.
//
// These are the calls of a decode step, which the GPU finishes in a few
// microseconds: with the checks in Python and the arguments through ctypes,
// paged_kv_build_tables spent 9.3 us on the host, here 2.6, most of it the launch.
#include <Python.h>

#include <ATen/core/TensorBase.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/pagedkv.h"

namespace {

PyObject *g_error = nullptr;   // PagedKVError

struct Raised {};              // a Python error is set

[[noreturn]] void fail(const char *message) {
    PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, message);
    throw Raised{};
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
        throw Raised{};
    }
    return THPVariable_Unpack(o);
}

int integer(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v > INT32_MAX || v < INT32_MIN) {
        PyErr_Format(g_error, "%s does not fit 32 bits", name);
        throw Raised{};
    }
    return int(v);
}

int narrow(int64_t v) {
    if (v > INT32_MAX) fail("a size does not fit 32 bits");
    return int(v);
}

int dtype_code(const at::Tensor &t) {
    switch (t.scalar_type()) {
        case at::kFloat: return PAGEDKV_F32;
        case at::kHalf: return PAGEDKV_F16;
        case at::kBFloat16: return PAGEDKV_BF16;
        default: fail("unsupported element type");
    }
}

// The current device, which every tensor of a call has to be on.
int device_of(const at::Tensor &t) {
    if (!t.is_cuda()) fail("expected CUDA tensors (the paged-KV path has no CPU fallback)");
    return c10::cuda::current_device();
}

void *on(int device, const at::Tensor &t, const char *name, at::ScalarType type) {
    if (!t.is_cuda() || t.get_device() != device) {
        PyErr_Format(g_error, "%s must be a CUDA tensor on the current device (cuda:%d)", name, device);
        throw Raised{};
    }
    if (t.scalar_type() != type) {
        PyErr_Format(g_error, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
        throw Raised{};
    }
    if (!t.is_contiguous()) {
        PyErr_Format(g_error, "%s must be contiguous", name);
        throw Raised{};
    }
    return t.data_ptr();
}

void *stream_of(PyObject *o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
    if (!h) throw Raised{};
    void *p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!p && PyErr_Occurred()) throw Raised{};
    return p;
}

PyObject *done(int status, const char *what) {
    if (status != PAGEDKV_OK) {
        PyErr_Format(g_error, "%s: %s (%d)", what, pagedkv_status_string(status), status);
        return nullptr;
    }
    Py_RETURN_NONE;
}

struct Pools {
    int blocks, heads, block;
};
Pools pools(const at::Tensor &k, const at::Tensor &v, int64_t dim) {
    if (k.dim() != 4 || v.sizes() != k.sizes() || k.size(3) * 8 != 5 * dim)
        fail("expected 4-bit pools [NB][Hkv][B][5 D / 8] for head_dim D");
    return {narrow(k.size(0)), narrow(k.size(1)), narrow(k.size(2))};
}

// A workspace tensor of any type, or None.
void *workspace_of(int device, PyObject *o, size_t *bytes) {
    *bytes = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, "workspace");
    *bytes = t.nbytes();
    return on(device, t, "workspace", t.scalar_type());
}

template <typename Body>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, Body body) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return nullptr;
    }
    try {
        return body();
    } catch (const Raised &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// rows (k, v, slot_mapping, k_cache, v_cache, stream), append or gather
PyObject *rows(PyObject *const *a, bool append) {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[2], "slot_mapping");
    const at::Tensor &kc = tensor(a[3], "k_cache"), &vc = tensor(a[4], "v_cache");
    if (k.dim() != 3 || v.sizes() != k.sizes() || slots.numel() != k.size(0))
        fail("expected k, v [T][Hkv][D] and one slot per token");
    const Pools p = pools(kc, vc, k.size(2));
    if (k.size(1) != p.heads) fail("token rows do not match the pools' kv heads");
    const int d = device_of(k), code = dtype_code(k), T = narrow(k.size(0)), D = narrow(k.size(2));
    void *kp = on(d, k, "k", k.scalar_type()), *vp = on(d, v, "v", k.scalar_type());
    const int64_t *sp = static_cast<const int64_t *>(on(d, slots, "slot_mapping", at::kLong));
    void *kcp = on(d, kc, "k_cache", at::kByte), *vcp = on(d, vc, "v_cache", at::kByte), *st = stream_of(a[5]);
    if (append)
        return done(paged_kv_append_q4(kp, vp, sp, kcp, vcp, T, p.blocks, p.block, p.heads, D, code, st),
                    "paged_kv_append_q4");
    return done(paged_kv_gather_q4(kcp, vcp, sp, kp, vp, T, p.blocks, p.block, p.heads, D, code, st),
                "paged_kv_gather_q4");
}

PyObject *append_q4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 6, [&] { return rows(a, true); });
}

PyObject *gather_q4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 6, [&] { return rows(a, false); });
}

// q, k_cache, v_cache, block_tables, context_lens, scale, out, partition_tokens, workspace, stream
PyObject *decode_q4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache");
        const at::Tensor &bt = tensor(a[3], "block_tables"), &lens = tensor(a[4], "context_lens");
        const at::Tensor &out = tensor(a[6], "out");
        if (q.dim() != 3 || out.sizes() != q.sizes() || bt.dim() != 2 || bt.size(0) != q.size(0) ||
            lens.numel() != q.size(0))
            fail("expected q/out [S][Hq][D], block_tables [S][max_blocks] and context_lens [S]");
        const Pools p = pools(kc, vc, q.size(2));
        const double scale = PyFloat_AsDouble(a[5]);
        if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
        const int part = integer(a[7], "partition_tokens"), d = device_of(q), code = dtype_code(q);
        size_t bytes;
        void *ws = workspace_of(d, a[8], &bytes);
        return done(paged_attention_decode_q4(
                        on(d, q, "q", q.scalar_type()), on(d, kc, "k_cache", at::kByte), on(d, vc, "v_cache", at::kByte),
                        static_cast<const int32_t *>(on(d, bt, "block_tables", at::kInt)),
                        static_cast<const int32_t *>(on(d, lens, "context_lens", at::kInt)), float(scale),
                        on(d, out, "out", q.scalar_type()), narrow(q.size(0)), narrow(q.size(1)), p.heads,
                        narrow(q.size(2)), p.blocks, p.block, narrow(bt.size(1)), part, ws, bytes, code,
                        stream_of(a[9])),
                    "paged_attention_decode_q4");
    });
}

// q, k_cache, v_cache, block_tables, query_start, context_lens, scale, out, max_query_len, workspace, key_parts, stream
PyObject *prefill_q4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 12, [&] {
        const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache");
        const at::Tensor &bt = tensor(a[3], "block_tables"), &start = tensor(a[4], "query_start");
        const at::Tensor &lens = tensor(a[5], "context_lens"), &out = tensor(a[7], "out");
        if (q.dim() != 3 || out.sizes() != q.sizes()) fail("q and out must be [num_tokens][n_q_heads][head_dim]");
        const int64_t S = lens.numel();
        if (start.numel() != S + 1 || bt.dim() != 2 || bt.size(0) != S)
            fail("query_start must hold num_seqs + 1 offsets, block_tables num_seqs rows");
        const Pools p = pools(kc, vc, q.size(2));
        const double scale = PyFloat_AsDouble(a[6]);
        if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
        const int most = integer(a[8], "max_query_len"), parts = integer(a[10], "key_parts");
        const int d = device_of(q), code = dtype_code(q);
        size_t bytes;
        void *ws = workspace_of(d, a[9], &bytes);
        return done(paged_attention_prefill_q4(
                        on(d, q, "q", q.scalar_type()), on(d, kc, "k_cache", at::kByte), on(d, vc, "v_cache", at::kByte),
                        static_cast<const int32_t *>(on(d, bt, "block_tables", at::kInt)),
                        static_cast<const int32_t *>(on(d, start, "query_start", at::kInt)),
                        static_cast<const int32_t *>(on(d, lens, "context_lens", at::kInt)), float(scale),
                        on(d, out, "out", q.scalar_type()), narrow(S), narrow(q.size(0)), most, narrow(q.size(1)),
                        p.heads, narrow(q.size(2)), p.blocks, p.block, narrow(bt.size(1)), code, parts, ws, bytes,
                        stream_of(a[11])),
                    "paged_attention_prefill_q4");
    });
}

// new_lens, context_lens, block_tables, free_blocks, free_count, block_size, num_blocks, query_start, token_seq,
// token_pos, slot_mapping, context_lens_out, free_count_out, stream
PyObject *build_tables(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 14, [&] {
        const at::Tensor &fresh = tensor(a[0], "new_lens"), &ctx = tensor(a[1], "context_lens");
        const at::Tensor &bt = tensor(a[2], "block_tables"), &free_blocks = tensor(a[3], "free_blocks");
        const at::Tensor &count = tensor(a[4], "free_count"), &start = tensor(a[7], "query_start");
        const at::Tensor &seq = tensor(a[8], "token_seq"), &pos = tensor(a[9], "token_pos");
        const at::Tensor *slots = a[10] == Py_None ? nullptr : &tensor(a[10], "slot_mapping");
        const at::Tensor &ctx_out = a[11] == Py_None ? ctx : tensor(a[11], "context_lens_out");
        const at::Tensor &count_out = a[12] == Py_None ? count : tensor(a[12], "free_count_out");
        const int64_t S = fresh.numel(), T = seq.numel();
        if (ctx.numel() != S || ctx_out.numel() != S || start.numel() != S + 1 || bt.dim() != 2 || bt.size(0) != S)
            fail("lengths, query_start and block_tables differ in their number of requests");
        if (pos.numel() != T || (slots && slots->numel() != T))
            fail("token_seq, token_pos and slot_mapping differ in length");
        if (count.numel() != 1 || count_out.numel() != 1) fail("free_count must hold one number");
        const int block = integer(a[5], "block_size"), blocks = integer(a[6], "num_blocks"), d = device_of(fresh);
        auto i32 = [&](const at::Tensor &t, const char *name) { return static_cast<int32_t *>(on(d, t, name, at::kInt)); };
        return done(paged_kv_build_tables(
                        i32(fresh, "new_lens"), i32(ctx, "context_lens"), i32(bt, "block_tables"),
                        i32(free_blocks, "free_blocks"), i32(count, "free_count"), i32(start, "query_start"),
                        i32(seq, "token_seq"), i32(pos, "token_pos"),
                        slots ? static_cast<int64_t *>(on(d, *slots, "slot_mapping", at::kLong)) : nullptr,
                        i32(ctx_out, "context_lens_out"), i32(count_out, "free_count_out"), narrow(S),
                        narrow(bt.size(1)), narrow(free_blocks.numel()), narrow(T), block, blocks, stream_of(a[13])),
                    "paged_kv_build_tables");
    });
}

PyObject *set_error(PyObject *, PyObject *cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"set_error", set_error, METH_O, "the class of the errors the others raise"},
    {"append_q4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append_q4)), METH_FASTCALL, nullptr},
    {"gather_q4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gather_q4)), METH_FASTCALL, nullptr},
    {"decode_q4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode_q4)), METH_FASTCALL, nullptr},
    {"prefill_q4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefill_q4)), METH_FASTCALL, nullptr},
    {"build_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(build_tables)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
