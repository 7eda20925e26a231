// CPython binding of the 8-bit cache, rotary cache write and cache read calls:
// what a decode step calls in its inner loop, where the host's time counts.
// A call checks its tensors (dense, type, shape, device), looks up the current
// stream and calls the C ABI, in 3 to 4 us, nearly all of it the launch; the
// same checks and a 24-argument ctypes call took 8 to 11 us in Python. The C
// functions come from the library that the package has loaded (bind()), so
// this file links against PyTorch only.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>
#include <string>

#include "pagedkv.h"

namespace {

// The entry points, by address.
struct Library {
    decltype(&paged_kv_cache_write_int8) write_int8;
    decltype(&paged_kv_cache_read) read;
    decltype(&paged_kv_rope_cache_write) rope;
    decltype(&paged_kv_rope_cache_write_fp8_scaled) rope_fp8_scaled;
    decltype(&paged_gqa_decode_attention_int8) decode;
    decltype(&paged_gqa_prefill_attention_int8) prefill;
} g_lib;

// A Python exception is set; caught at the entry of each call.
struct Raised {};

[[noreturn]] void raise(PyObject* kind, const std::string& what) {
    PyErr_SetString(kind, what.c_str());
    throw Raised{};
}

const char* type_name(at::ScalarType t) {
    switch (t) {
        case at::kHalf: return "float16";
        case at::kByte: return "uint8";
        case at::kFloat: return "float32";
        case at::kInt: return "int32";
        case at::kLong: return "int64";
        default: return c10::toString(t);
    }
}

std::string shape_text(c10::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// One call: the current device, and what its tensors are checked against.
struct Call {
    mutable int known = -1;
    int device() const {                 // looked up once a tensor on some GPU has been seen
        if (known < 0) known = c10::cuda::current_device();
        return known;
    }

    void* dense(const at::Tensor& t, const char* name, at::ScalarType type) const {
        if (!t.is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
        if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
        if (t.scalar_type() != type)
            raise(PyExc_TypeError, std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
        if (t.get_device() != device())
            raise(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
                                        ", but the current device is cuda:" + std::to_string(device()));
        return t.data_ptr();
    }
    // The address of a dense tensor of this type and shape on the current device.
    void* take(PyObject* o, const char* name, at::ScalarType type, c10::IntArrayRef shape) const {
        const at::Tensor& t = tensor(o, name);
        void* p = dense(t, name, type);
        if (t.sizes() != shape)
            raise(PyExc_ValueError, std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
        return p;
    }
    void* take(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) const {
        return take(o, name, type, c10::IntArrayRef(shape.begin(), shape.size()));
    }
    // None: the current stream; else an integer handle or an object with cuda_stream.
    void* stream(PyObject* o) const {
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device()).stream();
        if (PyLong_Check(o)) {
            void* p = PyLong_AsVoidPtr(o);
            if (!p && PyErr_Occurred()) throw Raised{};          // an integer that is no address
            return p;
        }
        PyObject* handle = PyObject_GetAttrString(o, "cuda_stream");
        if (!handle) throw Raised{};
        void* p = PyLong_AsVoidPtr(handle);
        Py_DECREF(handle);
        if (PyErr_Occurred()) throw Raised{};
        return p;
    }
};

int32_t int32(int64_t v, const char* name) {
    if (v < INT32_MIN || v > INT32_MAX) raise(PyExc_ValueError, std::string(name) + " is out of range");
    return (int32_t)v;
}
int32_t integer(PyObject* o, const char* name) {
    PyObject* n = PyNumber_Index(o);
    if (!n) throw Raised{};
    const long long v = PyLong_AsLongLong(n);
    Py_DECREF(n);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return int32(v, name);
}
float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)v;
}

// A scale of the whole cache. Not a CUDA tensor: its value would have to be copied to the host first, which waits
// for the stream and cannot be captured.
float scale_number(PyObject* o, const char* name) {
    if (THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda())
        raise(PyExc_TypeError, std::string(name) + " must be a number here, not a CUDA tensor");
    return number(o);
}

// A paged cache of any type.
struct Cache {
    void *k, *v;
    float* scales = nullptr;
    int32_t blocks, rows, heads, dim;

    Cache(const Call& c, PyObject* k_cache, PyObject* v_cache, PyObject* kv_scales, int code) {
        const at::Tensor& t = tensor(k_cache, "k_cache");
        const at::ScalarType type = code == PKV_KV_F16 ? at::kHalf : at::kByte;
        k = c.dense(t, "k_cache", type);
        if (t.dim() != 4) raise(PyExc_ValueError, "k_cache must be [num_blocks, block_size, num_kv_heads, head_dim]");
        v = c.take(v_cache, "v_cache", type, t.sizes());
        blocks = int32(t.size(0), "num_blocks");
        rows = int32(t.size(1), "block_size");
        heads = int32(t.size(2), "num_kv_heads");
        dim = int32(t.size(3), "head_dim");
        if (code == PKV_KV_INT8) {
            if (kv_scales == Py_None) raise(PyExc_ValueError, "an int8 cache needs kv_scales");
            scales = (float*)c.take(kv_scales, "kv_scales", at::kFloat, {blocks, heads, 2, rows});
        } else if (kv_scales != Py_None) {
            raise(PyExc_ValueError, "kv_scales belongs to an int8 cache");
        }
    }
};

void arguments(Py_ssize_t have, Py_ssize_t want) {
    if (have != want) raise(PyExc_TypeError, "expected " + std::to_string(want) + " arguments, got " + std::to_string(have));
}

// Runs `f` (which returns a status) and turns its exceptions into Python's.
template <typename F>
PyObject* guarded(F f) {
    try {
        return PyLong_FromLong((long)f());
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <typename F>
pkv_status unlocked(F f) {
    pkv_status s;
    Py_BEGIN_ALLOW_THREADS s = f();
    Py_END_ALLOW_THREADS return s;
}

// cache_write_int8(k_new, v_new, k_cache, v_cache, kv_scales, slot_mapping, stream)
PyObject* cache_write_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arguments(n, 7);
        const Call c;
        const Cache cache(c, a[2], a[3], a[4], PKV_KV_INT8);
        const at::Tensor& slots = tensor(a[5], "slot_mapping");
        auto* sm = (const int64_t*)c.dense(slots, "slot_mapping", at::kLong);
        const int32_t T = int32(slots.numel(), "slot_mapping");
        void* k = c.take(a[0], "k_new", at::kHalf, {T, cache.heads, cache.dim});
        void* v = c.take(a[1], "v_new", at::kHalf, {T, cache.heads, cache.dim});
        void* st = c.stream(a[6]);
        return unlocked([&] {
            return g_lib.write_int8(k, v, cache.k, cache.v, cache.scales, sm, T, cache.heads, cache.dim, cache.blocks,
                                    cache.rows, st);
        });
    });
}

// cache_read(k_out, v_out, k_cache, v_cache, slot_mapping, code, kv_scales, k_scale, v_scale, stream)
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arguments(n, 10);
        const Call c;
        const int code = integer(a[5], "kv_dtype");
        const Cache cache(c, a[2], a[3], a[6], code);
        const at::Tensor& slots = tensor(a[4], "slot_mapping");
        auto* sm = (const int64_t*)c.dense(slots, "slot_mapping", at::kLong);
        const int32_t T = int32(slots.numel(), "slot_mapping");
        void* k = c.take(a[0], "k_out", at::kHalf, {T, cache.heads, cache.dim});
        void* v = c.take(a[1], "v_out", at::kHalf, {T, cache.heads, cache.dim});
        const float ks = scale_number(a[7], "k_scale"), vs = scale_number(a[8], "v_scale");
        void* st = c.stream(a[9]);
        return unlocked([&] {
            return g_lib.read(k, v, cache.k, cache.v, cache.scales, sm, T, cache.heads, cache.dim, cache.blocks, cache.rows,
                              code, ks, vs, st);
        });
    });
}

// rope_cache_write(q_out, q, k_new, v_new, k_cache, v_cache, slot_mapping, positions, inv_freq, sections, flags, code,
//                  kv_scales, k_scale, v_scale, stream); k_scale and v_scale: numbers, or tensors (FP8)
PyObject* rope_cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arguments(n, 16);
        const Call c;
        const int code = integer(a[11], "kv_dtype");
        const Cache cache(c, a[4], a[5], a[12], code);
        const at::Tensor &slots = tensor(a[6], "slot_mapping"), &pos = tensor(a[7], "positions"),
                         &freq = tensor(a[8], "inv_freq"), &q = tensor(a[1], "q");
        auto* sm = (const int64_t*)c.dense(slots, "slot_mapping", at::kLong);
        auto* ps = (const int64_t*)c.dense(pos, "positions", at::kLong);
        auto* fr = (const float*)c.dense(freq, "inv_freq", at::kFloat);
        const int32_t T = int32(slots.numel(), "slot_mapping");
        if ((pos.dim() != 1 && pos.dim() != 2) || pos.size(-1) != T)
            raise(PyExc_ValueError, "positions must be [" + std::to_string(T) + "] or [axes, " + std::to_string(T) +
                                        "], got " + shape_text(pos.sizes()));
        const int32_t axes = pos.dim() == 2 ? int32(pos.size(0), "axes") : 1;
        const int32_t half = int32(freq.numel(), "inv_freq");
        if (half > (1 << 20)) raise(PyExc_ValueError, "inv_freq is too long");
        int32_t sections[16];
        if (a[9] == Py_None) {
            if (axes != 1) raise(PyExc_ValueError, "1 sections for " + std::to_string(axes) + " position axes");
            sections[0] = half;
        } else {
            PyObject* s = PySequence_Fast(a[9], "sections must be a sequence");
            if (!s) throw Raised{};
            const Py_ssize_t len = PySequence_Fast_GET_SIZE(s);
            bool bad = len != axes || len > 16;
            for (Py_ssize_t i = 0; !bad && i < len; ++i) {
                PyObject* count = PyNumber_Index(PySequence_Fast_GET_ITEM(s, i));    // (NumPy's integers too)
                const long v = count ? PyLong_AsLong(count) : -1;
                Py_XDECREF(count);
                bad = v < 0 || v > half;
                sections[i] = (int32_t)v;
            }
            Py_DECREF(s);
            PyErr_Clear();
            if (bad)
                raise(PyExc_ValueError, "sections must be " + std::to_string(axes) + " counts, one per position axis, of 0 to " +
                                            std::to_string(half));
        }
        if (q.dim() != 3) raise(PyExc_ValueError, "q must be [T, num_q_heads, head_dim]");
        const int32_t Hq = int32(q.size(1), "num_q_heads");
        void* qi = c.take(a[1], "q", at::kHalf, {T, Hq, cache.dim});
        void* qo = c.take(a[0], "q_out", at::kHalf, {T, Hq, cache.dim});
        void* k = c.take(a[2], "k_new", at::kHalf, {T, cache.heads, cache.dim});
        void* v = c.take(a[3], "v_new", at::kHalf, {T, cache.heads, cache.dim});
        const uint32_t flags = (uint32_t)integer(a[10], "flags");
        void* st = c.stream(a[15]);
        if (code == PKV_KV_FP8_E4M3 && THPVariable_Check(a[13])) {
            const at::Tensor &kt = tensor(a[13], "k_scales"), &vt = tensor(a[14], "v_scales");
            auto* ks = (const float*)c.dense(kt, "k_scales", at::kFloat);
            auto* vs = (const float*)c.dense(vt, "v_scales", at::kFloat);
            if (kt.numel() != vt.numel() || (kt.numel() != 1 && kt.numel() != cache.heads))
                raise(PyExc_ValueError, "k_scales and v_scales need 1 (per tensor) or num_kv_heads (per head) elements");
            const int32_t per_head = kt.numel() == cache.heads && cache.heads > 1;
            return unlocked([&] {
                return g_lib.rope_fp8_scaled(qo, qi, k, v, cache.k, cache.v, sm, ps, fr, T, Hq, cache.heads, cache.dim,
                                             2 * half, axes, sections, cache.blocks, cache.rows, ks, vs, per_head, flags, st);
            });
        }
        const float ks = scale_number(a[13], "k_scale"), vs = scale_number(a[14], "v_scale");
        return unlocked([&] {
            return g_lib.rope(qo, qi, k, v, cache.k, cache.v, cache.scales, sm, ps, fr, T, Hq, cache.heads, cache.dim,
                              2 * half, axes, sections, cache.blocks, cache.rows, code, ks, vs, flags, st);
        });
    });
}

// What decode and chunk attention share: out, q, k_cache, v_cache, kv_scales, block_tables, context_lens, workspace.
struct Attention {
    Cache cache;
    void *out, *q, *ws;
    const int32_t *tables, *lens;
    int32_t total, heads, batch, width;
    size_t ws_bytes;

    Attention(const Call& c, PyObject* const* a, PyObject* workspace) : cache(c, a[2], a[3], a[4], PKV_KV_INT8) {
        const at::Tensor &qt = tensor(a[1], "q"), &bt = tensor(a[5], "block_tables"), &w = tensor(workspace, "workspace");
        if (qt.dim() != 3 || bt.dim() != 2)
            raise(PyExc_ValueError, "q must be [rows, num_q_heads, head_dim] and block_tables [batch, max_blocks]");
        total = int32(qt.size(0), "q");
        heads = int32(qt.size(1), "num_q_heads");
        batch = int32(bt.size(0), "batch");
        width = int32(bt.size(1), "max_blocks");
        q = c.take(a[1], "q", at::kHalf, {total, heads, cache.dim});
        out = c.take(a[0], "out", at::kHalf, {total, heads, cache.dim});
        tables = (const int32_t*)c.dense(bt, "block_tables", at::kInt);
        lens = (const int32_t*)c.take(a[6], "context_lens", at::kInt, {batch});
        const at::ScalarType type = w.scalar_type();
        if (type != at::kByte && type != at::kFloat && type != at::kInt)
            raise(PyExc_TypeError, std::string("workspace must be uint8 or float32 or int32, got ") + type_name(type));
        ws = c.dense(w, "workspace", type);
        ws_bytes = (size_t)w.nbytes();
    }
};

// decode_attention_int8(out, q, k_cache, v_cache, kv_scales, block_tables, context_lens, max_context_len,
//                       softmax_scale, workspace, stream)
PyObject* decode_attention_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arguments(n, 11);
        const Call c;
        const Attention t(c, a, a[9]);
        if (t.total != t.batch)
            raise(PyExc_ValueError, std::to_string(t.total) + " query rows for " + std::to_string(t.batch) + " sequences");
        const int32_t longest = integer(a[7], "max_context_len");
        const float scale = number(a[8]);
        void* st = c.stream(a[10]);
        return unlocked([&] {
            return g_lib.decode(t.out, t.q, t.cache.k, t.cache.v, t.cache.scales, t.tables, t.lens, t.batch, t.heads,
                                t.cache.heads, t.cache.dim, t.cache.rows, t.width, t.cache.blocks, longest, scale, t.ws,
                                t.ws_bytes, st);
        });
    });
}

// prefill_attention_int8(out, q, k_cache, v_cache, kv_scales, block_tables, context_lens, query_start, max_query_len,
//                        max_context_len, softmax_scale, workspace, stream)
PyObject* prefill_attention_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arguments(n, 13);
        const Call c;
        const Attention t(c, a, a[11]);
        auto* qs = (const int32_t*)c.take(a[7], "query_start", at::kInt, {(int64_t)t.batch + 1});
        const int32_t most = integer(a[8], "max_query_len"), longest = integer(a[9], "max_context_len");
        const float scale = number(a[10]);
        void* st = c.stream(a[12]);
        return unlocked([&] {
            return g_lib.prefill(t.out, t.q, t.cache.k, t.cache.v, t.cache.scales, t.tables, t.lens, qs, t.batch, t.total,
                                 most, t.heads, t.cache.heads, t.cache.dim, t.cache.rows, t.width, t.cache.blocks, longest,
                                 scale, t.ws, t.ws_bytes, st);
        });
    });
}

// bind(addresses): the C functions' addresses, in the order of Library.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        arguments(n, 6);
        void* at[6];
        for (int i = 0; i < 6; ++i) {
            at[i] = PyLong_AsVoidPtr(a[i]);
            if (PyErr_Occurred()) throw Raised{};
        }
        g_lib.write_int8 = reinterpret_cast<decltype(g_lib.write_int8)>(at[0]);
        g_lib.read = reinterpret_cast<decltype(g_lib.read)>(at[1]);
        g_lib.rope = reinterpret_cast<decltype(g_lib.rope)>(at[2]);
        g_lib.rope_fp8_scaled = reinterpret_cast<decltype(g_lib.rope_fp8_scaled)>(at[3]);
        g_lib.decode = reinterpret_cast<decltype(g_lib.decode)>(at[4]);
        g_lib.prefill = reinterpret_cast<decltype(g_lib.prefill)>(at[5]);
        return PKV_OK;
    });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FAST(bind), FAST(cache_write_int8), FAST(cache_read), FAST(rope_cache_write),
                          FAST(decode_attention_int8), FAST(prefill_attention_int8), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
