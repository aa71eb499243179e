// torch_args.cpp - arguments of the serving calls from torch tensors, as a CPython extension.
//
// A decoding step calls fa2_rope, fa2_kv_append and fa2_decode on tensors so small that the host
// sets the pace: reading shapes, types, strides and pointers of a dozen tensors from Python took
// 3.4 us (rope) to 7.3 us (append) of a call, the launch itself about 2 us. Here the same checks
// read the tensors' fields directly. The computation stays behind the C ABI: this file calls the
// library's entry points, whose addresses binding.py hands over.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fa2.h"

namespace {

decltype(&fa2_rope) g_rope = nullptr;
decltype(&fa2_rope_backward) g_rope_backward = nullptr;
decltype(&fa2_kv_append) g_kv_append = nullptr;
decltype(&fa2_kv_read) g_kv_read = nullptr;
decltype(&fa2_decode) g_decode = nullptr;

// A Python exception is set: unwinds to the entry point.
struct Raised {};

template <typename... A>
[[noreturn]] void refuse(PyObject* type, const char* format, A... args) {
    PyErr_Format(type, format, args...);
    throw Raised{};
}

// A tensor argument; null for None where that is allowed.
struct Arg {
    const at::Tensor* t = nullptr;
    const char* name;
    Arg(PyObject* o, const char* n, bool optional = false) : name(n) {
        if (optional && o == Py_None) return;
        if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor, got %s", n, Py_TYPE(o)->tp_name);
        t = &THPVariable_Unpack(o);
    }
    explicit operator bool() const { return t != nullptr; }
    int64_t dim() const { return t->dim(); }
    int64_t size(int i) const { return t->sizes()[i]; }
    int64_t stride(int i) const { return t->strides()[i]; }
    at::ScalarType type() const { return t->scalar_type(); }
};

struct Call {
    const char* where;
    int device = 0;
    void* stream = nullptr;

    [[noreturn]] void value_error(const char* what) const { refuse(PyExc_ValueError, "%s: %s", where, what); }

    void type(const Arg& a, at::ScalarType want) const {
        if (a && a.type() != want)
            refuse(PyExc_TypeError, "%s: %s must be %s, got %s", where, a.name, c10::toString(want), c10::toString(a.type()));
    }
    void same_type(const Arg& ref, const Arg& a) const {
        if (a.type() != ref.type())
            refuse(PyExc_TypeError, "%s: %s is %s, expected %s like the other tensors", where, a.name, c10::toString(a.type()),
                   c10::toString(ref.type()));
    }
    fa2_dtype code(const Arg& a) const {
        switch (a.type()) {
            case at::kFloat: return FA2_DTYPE_F32;
            case at::kHalf: return FA2_DTYPE_F16;
            case at::kBFloat16: return FA2_DTYPE_BF16;
            default: refuse(PyExc_TypeError, "unsupported dtype %s", c10::toString(a.type()));
        }
    }
    // The current device and the stream given, or torch's current one there; `a` is a tensor of the call.
    void begin(const Arg& a, PyObject* given) {
        if (!a.t->is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", a.name);
        device = c10::cuda::current_device();
        if (given == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
            return;
        }
        PyObject* raw = PyObject_GetAttrString(given, "cuda_stream");
        if (!raw) throw Raised{};
        stream = PyLong_AsVoidPtr(raw);
        Py_DECREF(raw);
        if (PyErr_Occurred()) throw Raised{};
    }
    void here(const Arg& a) const {
        if (!a.t->is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", a.name);
        const int at = a.t->get_device();
        // the library launches on the current device; another device's memory is not its to read
        if (at != device)
            refuse(PyExc_ValueError, "%s is on cuda:%d, but the current device is cuda:%d", a.name, at, device);
    }
    void* whole(const Arg& a) const {  // a contiguous tensor
        here(a);
        if (!a.t->is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", a.name);
        return a.t->data_ptr();
    }
    void* rows(const Arg& a) const {  // its last dimension contiguous, the others as they are
        here(a);
        const int64_t last = a.dim() - 1;
        if (a.size((int)last) > 1 && a.stride((int)last) != 1)
            refuse(PyExc_ValueError, "%s's last dimension must be contiguous", a.name);
        return a.t->data_ptr();
    }
};

bool same_sizes(const Arg& a, const Arg& b) { return a.t->sizes() == b.t->sizes(); }

// The stride of a dimension of one element means nothing.
bool same_strides(const Arg& a, const Arg& b) {
    for (int64_t i = 0; i < a.dim(); ++i)
        if (a.size((int)i) > 1 && a.stride((int)i) != b.stride((int)i)) return false;
    return true;
}

bool sizes_are(const Arg& a, std::initializer_list<int64_t> want) { return a.t->sizes() == at::IntArrayRef(want); }

// The paged cache, the block table and the lengths of a call: checks in the constructor, pointers
// once the device is known.
struct Paged {
    const Call& call;
    Arg k, v, k_exp, v_exp, table, lens;
    fa2_kv_cache cache{};
    int64_t batch, heads, d, per_seq, table_stride;

    Paged(const Call& c, PyObject* kp, PyObject* vp, PyObject* ke, PyObject* ve, PyObject* tab, PyObject* len, const Arg& row)
        : call(c), k(kp, "k_pages"), v(vp, "v_pages"), k_exp(ke, "k_exp", true), v_exp(ve, "v_exp", true),
          table(tab, "block_table"), lens(len, "seq_lens") {
        if (k.dim() != 4 || !same_sizes(k, v))
            c.value_error("k_pages and v_pages are [num_pages, n_kv_heads, page_size, d], both of one shape");
        if (!same_strides(k, v)) c.value_error("k_pages and v_pages must have the same strides");
        c.same_type(k, v);
        heads = k.size(1);
        d = k.size(3);
        if (k.type() == at::kFloat8_e4m3fn) {
            if (!k_exp || !v_exp) c.value_error("an e4m3 cache has scale bytes, k_exp and v_exp");
            c.type(k_exp, at::kByte);
            c.type(v_exp, at::kByte);
            for (const Arg* e : {&k_exp, &v_exp})
                if (!sizes_are(*e, {k.size(0), heads, k.size(2)}))
                    c.value_error("k_exp and v_exp must be [num_pages, n_kv_heads, page_size]");
            cache.type = FA2_CACHE_E4M3;
        } else {
            if (k_exp || v_exp) c.value_error("k_exp and v_exp belong to an e4m3 cache");
            if (k.type() != row.type())
                refuse(PyExc_TypeError, "%s: the pages are %s, expected %s or Float8_e4m3fn", c.where, c10::toString(k.type()),
                       c10::toString(row.type()));
            cache.type = FA2_CACHE_SAME;
        }
        c.type(table, at::kInt);
        c.type(lens, at::kInt);
        if (table.dim() != 2 || !sizes_are(lens, {table.size(0)}))
            c.value_error("block_table is [batch, pages_per_seq] and seq_lens [batch]");
        batch = table.size(0);
        per_seq = table.size(1);
        table_stride = batch > 1 ? table.stride(0) : per_seq;
        for (int i = 0; i < 3; ++i)
            if (k.size(i) > INT32_MAX) c.value_error("a dimension of the pages is past 2^31 - 1");
        cache.num_pages = k.size(0);
        cache.n_kv_heads = (int32_t)heads;
        cache.page_size = (int32_t)k.size(2);
        cache.head_dim = (int32_t)(d > INT32_MAX ? INT32_MAX : d);
        cache.page_stride = k.stride(0);
        cache.head_stride = k.stride(1);
        cache.slot_stride = k.stride(2);
    }
    const fa2_kv_cache* pools() {
        cache.k = call.rows(k);
        cache.v = call.rows(v);
        if (cache.type == FA2_CACHE_E4M3) {
            cache.k_exp = static_cast<uint8_t*>(call.whole(k_exp));
            cache.v_exp = static_cast<uint8_t*>(call.whole(v_exp));
        }
        return &cache;
    }
    const int32_t* table_at() const { return static_cast<const int32_t*>(call.rows(table)); }
    const int32_t* lens_at() const { return static_cast<const int32_t*>(call.whole(lens)); }
};

PyObject* result(fa2_status st) { return PyLong_FromLong((long)st); }

// Runs an entry point's body: a Python exception for whatever it throws, and for a missing library.
template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t want, F body) {
    if (given != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, got %zd", want, given);
        return nullptr;
    }
    try {
        if (!g_decode) refuse(PyExc_RuntimeError, "%s", "the library's entry points are not set");
        return result(body());
    } catch (const Raised&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}

// x, y, inv_freq, positions | None, interleaved, magnitude, stream | None, backward
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 8, [&] {
        const bool backward = a[7] == Py_True;
        Call c{backward ? "fa2_rope_backward" : "fa2_rope"};
        const Arg x(a[0], backward ? "dy" : "x"), y(a[1], backward ? "dx" : "y"), f(a[2], "inv_freq"), pos(a[3], "positions", true);
        if (x.dim() != 4 || !same_sizes(x, y)) c.value_error("the tensors are [B, H, N, d], both of one shape");
        c.same_type(x, y);
        c.type(f, at::kDouble);
        if (f.dim() != 1) c.value_error("inv_freq must be [rot_dim / 2]");
        const int64_t b = x.size(0), h = x.size(1), n = x.size(2), d = x.size(3);
        int64_t step = 0;
        if (pos) {
            c.type(pos, at::kInt);
            if (!sizes_are(pos, {n}) && !sizes_are(pos, {1, n}) && !sizes_are(pos, {b, n}))
                c.value_error("positions must be [N], [1, N] or [B, N]");
            if (pos.dim() == 2 && pos.size(0) > 1) step = pos.stride(0);
        }
        const fa2_dtype code = c.code(x);
        const int interleaved = PyObject_IsTrue(a[4]);
        if (interleaved < 0) throw Raised{};
        const float magnitude = (float)number(a[5]);
        c.begin(x, a[6]);
        const int64_t xs[3] = {x.stride(0), x.stride(1), x.stride(2)}, ys[3] = {y.stride(0), y.stride(1), y.stride(2)};
        const void* xp = c.rows(x);
        void* yp = c.rows(y);
        const int32_t* pp = pos ? static_cast<const int32_t*>(c.rows(pos)) : nullptr;
        const double* fp = static_cast<const double*>(c.whole(f));
        const int64_t rot = 2 * f.size(0);
        const int32_t d32 = (int32_t)(d > INT32_MAX ? INT32_MAX : d), r32 = (int32_t)(rot > INT32_MAX ? INT32_MAX : rot);
        fa2_status st;
        Py_BEGIN_ALLOW_THREADS
        st = (backward ? g_rope_backward : g_rope)(xp, yp, pp, step, fp, b, h, n, d32, r32, xs, ys, interleaved, magnitude, code,
                                                   c.stream);
        Py_END_ALLOW_THREADS
        return st;
    });
}

// k_pages, v_pages, k, v, block_table, seq_lens, cu_new | None, k_exp | None, v_exp | None, stream | None
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 10, [&] {
        Call c{"fa2_kv_append"};
        const Arg k(a[2], "k"), v(a[3], "v"), cu(a[6], "cu_new", true);
        Paged p(c, a[0], a[1], a[7], a[8], a[4], a[5], k);
        if (k.dim() != 3 || !same_sizes(k, v) || k.size(1) != p.heads || k.size(2) != p.d)
            c.value_error("k and v are [tokens, n_kv_heads, d]");
        c.same_type(k, v);
        c.type(cu, at::kInt);
        if (cu && !sizes_are(cu, {p.batch + 1})) c.value_error("cu_new must be [batch + 1]");
        const fa2_dtype code = c.code(k);
        c.begin(k, a[9]);
        const fa2_kv_cache* cache = p.pools();
        const void *kp = c.rows(k), *vp = c.rows(v);
        const int64_t ks[2] = {k.stride(0), k.stride(1)}, vs[2] = {v.stride(0), v.stride(1)};
        const int32_t *table = p.table_at(), *lens = p.lens_at(), *cp = cu ? static_cast<const int32_t*>(c.whole(cu)) : nullptr;
        const int64_t tokens = k.size(0);
        fa2_status st;
        Py_BEGIN_ALLOW_THREADS
        st = g_kv_append(cache, kp, vp, ks, vs, table, p.table_stride, p.per_seq, cp, lens, p.batch, tokens, code, c.stream);
        Py_END_ALLOW_THREADS
        return st;
    });
}

// k_pages, v_pages, k_out, v_out, block_table, seq_lens, k_exp | None, v_exp | None, stream | None
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 9, [&] {
        Call c{"fa2_kv_read"};
        const Arg k(a[2], "k_out"), v(a[3], "v_out");
        Paged p(c, a[0], a[1], a[6], a[7], a[4], a[5], k);
        if (k.dim() != 4 || !same_sizes(k, v) || k.size(0) != p.batch || k.size(1) != p.heads || k.size(3) != p.d)
            c.value_error("k_out and v_out are [batch, n_kv_heads, max_len, d]");
        if (!same_strides(k, v)) c.value_error("k_out and v_out must have the same strides");
        c.same_type(k, v);
        const fa2_dtype code = c.code(k);
        c.begin(k, a[8]);
        const fa2_kv_cache* cache = p.pools();
        void *kp = c.rows(k), *vp = c.rows(v);
        const int64_t strides[3] = {k.stride(0), k.stride(1), k.stride(2)}, longest = k.size(2);
        const int32_t *table = p.table_at(), *lens = p.lens_at();
        fa2_status st;
        Py_BEGIN_ALLOW_THREADS
        st = g_kv_read(cache, kp, vp, strides, table, p.table_stride, p.per_seq, lens, p.batch, longest, code, c.stream);
        Py_END_ALLOW_THREADS
        return st;
    });
}

// q, k_pages, v_pages, o, lse, block_table, seq_lens, workspace, softmax_scale, window, k_exp | None, v_exp | None,
// stream | None
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 13, [&] {
        Call c{"fa2_decode"};
        const Arg q(a[0], "q"), o(a[3], "o"), lse(a[4], "lse"), ws(a[7], "workspace");
        Paged p(c, a[1], a[2], a[10], a[11], a[5], a[6], q);
        if (q.dim() != 3 || q.size(0) != p.batch || q.size(2) != p.d || !same_sizes(q, o) ||
            !sizes_are(lse, {q.size(0), q.size(1)}))
            c.value_error("q and o are [batch, n_heads, d], lse [batch, n_heads]");
        if (q.size(1) > INT32_MAX) c.value_error("n_heads is past 2^31 - 1");
        c.same_type(q, o);
        c.type(lse, at::kFloat);
        const fa2_dtype code = c.code(q);
        const float scale = (float)number(a[8]);
        const int64_t window = PyLong_AsLongLong(a[9]);
        if (window == -1 && PyErr_Occurred()) throw Raised{};
        c.begin(q, a[12]);
        const fa2_kv_cache* cache = p.pools();
        const void* qp = c.rows(q);
        void *op = c.whole(o), *wp = c.whole(ws);
        float* lp = static_cast<float*>(c.whole(lse));
        const int64_t qs[2] = {q.stride(0), q.stride(1)};
        const size_t bytes = (size_t)ws.t->numel() * ws.t->element_size();
        const int32_t *table = p.table_at(), *lens = p.lens_at();
        const int32_t heads = (int32_t)q.size(1);
        fa2_status st;
        Py_BEGIN_ALLOW_THREADS
        st = g_decode(qp, qs, cache, op, lp, table, p.table_stride, p.per_seq, lens, p.batch, heads, window, wp, bytes, code, scale, c.stream);
        Py_END_ALLOW_THREADS
        return st;
    });
}

// The addresses of fa2_rope, fa2_rope_backward, fa2_kv_append, fa2_kv_read and fa2_decode.
PyObject* set_entry_points(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (n_args != 5) {
        PyErr_SetString(PyExc_TypeError, "five addresses are wanted");
        return nullptr;
    }
    void* p[5];
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_rope = reinterpret_cast<decltype(g_rope)>(p[0]);
    g_rope_backward = reinterpret_cast<decltype(g_rope_backward)>(p[1]);
    g_kv_append = reinterpret_cast<decltype(g_kv_append)>(p[2]);
    g_kv_read = reinterpret_cast<decltype(g_kv_read)>(p[3]);
    g_decode = reinterpret_cast<decltype(g_decode)>(p[4]);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<rope>("rope"), method<kv_append>("kv_append"), method<kv_read>("kv_read"),
                           method<decode>("decode"), method<set_entry_points>("set_entry_points"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fa2_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa2_torch() { return PyModule_Create(&g_module); }
