// The Python binding's calls that a serving loop makes every step, in C++: rotation,
// append, tree attention, accepted paths and forks.  Each checks its tensors (type,
// device, layout, sizes that belong together), makes the outputs that were not given,
// and calls the C ABI on the device's current stream, as the calls in __init__.py do;
// in Python these checks took longer than most of the calls' work on the GPU (an
// accepted path 14.7 us, here 4.3).
//
// The library is not linked: bind() is given the addresses of its functions.

#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "swiattn.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refused {   // a ValueError
    std::string text;
};
struct Raised {};   // Python's error is set

[[noreturn]] void refuse(const char* format, ...) {
    char text[400];
    va_list list;
    va_start(list, format);
    vsnprintf(text, sizeof(text), format, list);
    va_end(list);
    throw Refused{text};
}

PyObject* g_error;   // SwiAttnError

struct Library {
    decltype(&swiattn_rope) rope, rope_backward;
    decltype(&swiattn_rope_axes) rope_axes, rope_axes_backward;
    decltype(&swiattn_append_paged) append_paged;
    decltype(&swiattn_append_paged_at) append_paged_at;
    decltype(&swiattn_decode_tree) decode_tree;
    decltype(&swiattn_decode_tree_workspace) decode_tree_workspace;
    decltype(&swiattn_accept_tree) accept_tree;
    decltype(&swiattn_fork_paged) fork_paged;
} g_lib;

template <typename F>
void address(PyObject* dict, const char* name, F& f) {
    PyObject* o = PyDict_GetItemString(dict, name);   // borrowed
    void* p = o ? PyLong_AsVoidPtr(o) : nullptr;
    if (!p) refuse("no address for %s", name);
    f = reinterpret_cast<F>(p);
}

// ---- arguments ---------------------------------------------------------------
bool is_none(PyObject* o) { return o == Py_None; }

int whole(PyObject* o, const char* name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v > INT_MAX || v < INT_MIN) refuse("%s does not fit 32 bits: %ld", name, v);
    return static_cast<int>(v);
}
float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return static_cast<float>(v);
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}

std::string sizes_of(const Tensor& t) {
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "]";
}

// The first tensor of a call, whose device is the call's.
const Tensor& first(PyObject* o, const char* name) {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) refuse("%s must be a CUDA tensor", name);
    return THPVariable_Unpack(o);
}
// A further one: contiguous, on the same device, of a type.
const Tensor& same(PyObject* o, const char* name, int index) {
    const Tensor& t = first(o, name);
    if (!t.is_contiguous()) refuse("%s must be contiguous", name);
    if (t.get_device() != index) refuse("%s is on cuda:%d, expected cuda:%d", name, static_cast<int>(t.get_device()), index);
    return t;
}
const Tensor& same(PyObject* o, const char* name, int index, ScalarType type) {
    const Tensor& t = same(o, name, index);
    if (t.scalar_type() != type) refuse("%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
    return t;
}
const int32_t* ints(PyObject* o, const char* name, int index, int64_t count) {
    const Tensor& t = same(o, name, index, at::kInt);
    if (t.numel() != count) refuse("%s must hold %lld values, got %lld", name, static_cast<long long>(count), static_cast<long long>(t.numel()));
    return static_cast<const int32_t*>(t.data_ptr());
}

int kind_of(const Tensor& t) {
    if (t.scalar_type() == at::kFloat) return SWIATTN_F32;
    if (t.scalar_type() == at::kBFloat16) return SWIATTN_BF16;
    refuse("dtype must be torch.float32 or torch.bfloat16, got %s", c10::toString(t.scalar_type()));
}

// q, k or v of a call, [lead..., heads, d]: packed heads, one distance between tokens (a
// view of a fused projection is fine).
struct Tokens {
    const Tensor* t;
    int heads, d;
    int64_t step;
};
Tokens tokens(PyObject* o, const char* name, c10::IntArrayRef lead, int index, ScalarType type) {
    const Tensor& t = first(o, name);
    if (t.get_device() != index) refuse("%s must be a tensor on cuda:%d", name, index);
    if (t.scalar_type() != type) refuse("%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
    const int64_t n = static_cast<int64_t>(lead.size());
    bool fits = t.dim() == n + 2;
    for (int64_t i = 0; fits && i < n; ++i) fits = t.size(i) == lead[i];
    if (!fits) refuse("%s must have the call's tokens, then [heads, d], got %s", name, sizes_of(t).c_str());
    const int64_t heads = t.size(n), d = t.size(n + 1);
    if (heads > INT_MAX || d > INT_MAX) refuse("%s is too large", name);
    Tokens r{&t, static_cast<int>(heads), static_cast<int>(d), heads * d};
    if (t.is_contiguous()) return r;
    if (t.stride(n + 1) != 1 || (heads > 1 && t.stride(n) != d)) refuse("%s: heads and their elements must be contiguous", name);
    int64_t count = 1;
    for (int64_t i = n - 1; i >= 0; --i) {
        if (t.size(i) <= 1) continue;   // dimensions of size 1 may have any stride
        if (count == 1) r.step = t.stride(i);
        else if (t.stride(i) != count * r.step) refuse("%s: tokens must be evenly spaced", name);
        count *= t.size(i);
    }
    return r;
}

// Page pools [num_pages, page_size, Hkv, d], or of several layers.
struct Pools {
    void *k, *v;
    uint8_t *k_exp, *v_exp;
    int layers, num_pages, page_size, Hkv, d, kind;
};
uint8_t* exponents(PyObject* o, const char* name, int index, const Tensor& pages) {
    const Tensor& t = same(o, name, index);
    if (t.scalar_type() != at::kByte && t.scalar_type() != at::kFloat8_e8m0fnu) refuse("%s must be uint8 or float8_e8m0fnu", name);
    const int64_t n = pages.dim();
    bool fits = t.dim() == n - 1;
    for (int64_t i = 0; fits && i < n - 3; ++i) fits = t.size(i) == pages.size(i);
    if (!fits || t.size(n - 3) != pages.size(n - 2) || t.size(n - 2) != pages.size(n - 3)) refuse("%s must be [..., num_pages, Hkv, page_size], got %s", name, sizes_of(t).c_str());
    return static_cast<uint8_t*>(t.data_ptr());
}
Pools pools(PyObject* k_pages, PyObject* v_pages, PyObject* k_exp, PyObject* v_exp, int index, bool layered) {
    const Tensor& k = same(k_pages, "k_pages", index);
    const Tensor& v = same(v_pages, "v_pages", index, k.scalar_type());
    const int64_t n = k.dim();
    if (v.sizes() != k.sizes() || !(n == 4 || (layered && n == 5)))
        refuse("k_pages and v_pages must both be %s[num_pages, page_size, Hkv, d]", layered ? "[layers, num_pages, page_size, Hkv, d] or " : "");
    for (int64_t i = 0; i < n; ++i)
        if (k.size(i) > INT_MAX) refuse("k_pages is too large");
    Pools p{};
    p.k = k.data_ptr();
    p.v = v.data_ptr();
    p.layers = n == 5 ? static_cast<int>(k.size(0)) : 1;
    p.num_pages = static_cast<int>(k.size(n - 4));
    p.page_size = static_cast<int>(k.size(n - 3));
    p.Hkv = static_cast<int>(k.size(n - 2));
    p.d = static_cast<int>(k.size(n - 1));
    if (k.scalar_type() == at::kFloat8_e4m3fn) {
        p.kind = SWIATTN_E4M3;
        p.k_exp = exponents(k_exp, "k_exp", index, k);
        p.v_exp = exponents(v_exp, "v_exp", index, k);
    } else if (k.scalar_type() == at::kFloat || k.scalar_type() == at::kBFloat16) {
        p.kind = kind_of(k);
    } else {
        refuse("pages must be float32, bfloat16 or float8_e4m3fn, got %s", c10::toString(k.scalar_type()));
    }
    return p;
}

struct Sequences {
    const int32_t *table, *lens;
    int B, max_pages;
};
Sequences sequences(PyObject* block_table, PyObject* seq_lens, int index) {
    const Tensor& lens = same(seq_lens, "seq_lens", index, at::kInt);
    const Tensor& table = same(block_table, "block_table", index, at::kInt);
    if (table.dim() != 2 || table.size(0) != lens.numel() || table.size(1) > INT_MAX || lens.numel() > INT_MAX)
        refuse("block_table must be [%lld, max_pages]", static_cast<long long>(lens.numel()));
    return {static_cast<const int32_t*>(table.data_ptr()), static_cast<const int32_t*>(lens.data_ptr()), static_cast<int>(lens.numel()),
            static_cast<int>(table.size(1))};
}

const int32_t* parents_of(PyObject* o, int index, int64_t& count) {
    if (is_none(o)) return nullptr;
    const Tensor& t = same(o, "parents", index, at::kInt);
    if (t.dim() != 1) refuse("parents must be [T]");
    count = t.numel();
    return static_cast<const int32_t*>(t.data_ptr());
}

// Axes as bytes, or none.
const uint8_t* axes_of(PyObject* o, int64_t half) {
    if (is_none(o)) return nullptr;
    if (PyBytes_GET_SIZE(o) != half)
        refuse("axes must hold %lld values, one for each frequency, got %lld", static_cast<long long>(half), static_cast<long long>(PyBytes_GET_SIZE(o)));
    return reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(o));
}

Tensor fresh(c10::IntArrayRef sizes, const Tensor& like, ScalarType type) { return at::empty(sizes, like.options().dtype(type)); }

// Makes a call with its device current, on the device's current stream, and without
// the interpreter's lock.
template <typename F>
void call(const char* where, int index, F f) {
    const c10::cuda::OptionalCUDAGuard guard(static_cast<c10::DeviceIndex>(index));
    void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = f(stream);
    Py_END_ALLOW_THREADS
    if (status == SWIATTN_OK) return;
    PyObject* error = PyObject_CallFunction(g_error, "is", status, where);
    if (error) {
        PyErr_SetObject(g_error, error);
        Py_DECREF(error);
    }
    throw Raised{};
}

template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
    HANDLE_TH_ERRORS
    try {
        if (given != wanted) refuse("%zd arguments, expected %zd", given, wanted);
        return f();
    } catch (const Refused& r) {
        PyErr_SetString(PyExc_ValueError, r.text.c_str());
        return nullptr;
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject* new_ref(PyObject* o) {
    Py_INCREF(o);
    return o;
}
PyObject* pair(PyObject* a, PyObject* b) {   // of references that it takes over
    if (!a || !b) {
        Py_XDECREF(a);
        Py_XDECREF(b);
        throw Raised{};
    }
    PyObject* t = PyTuple_New(2);
    if (!t) throw Raised{};
    PyTuple_SET_ITEM(t, 0, a);
    PyTuple_SET_ITEM(t, 1, b);
    return t;
}

// ---- the calls ---------------------------------------------------------------
// backward, q, k, inv_freq, positions, interleaved, factor, q_out, k_out, axes
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject* {
        const bool backward = truth(a[0]);
        PyObject* const x[2] = {a[1], a[2]};
        PyObject* const out[2] = {a[7], a[8]};
        const Tensor& some = first(is_none(x[0]) ? x[1] : x[0], "q and k");
        const int index = some.get_device();
        if (some.dim() != 4) refuse("q and k must be [B, N, heads, d], got %s", sizes_of(some).c_str());
        const int64_t B = some.size(0), N = some.size(1), d = some.size(3);
        if (B > INT_MAX || N > INT_MAX) refuse("too many tokens");
        const int kind = kind_of(some);
        Tokens in[2] = {}, to[2] = {};
        Tensor made[2];
        for (int i = 0; i < 2; ++i) {
            const char* name = i ? "k" : "q";
            if (is_none(x[i])) {
                if (!is_none(out[i])) refuse("out for %s, which is None", name);
                continue;
            }
            in[i] = tokens(x[i], name, some.sizes().slice(0, 2), index, some.scalar_type());
            if (in[i].d != d) refuse("q and k must have one head size");
            if (is_none(out[i])) {
                made[i] = fresh(in[i].t->sizes(), some, some.scalar_type());
                to[i] = {&made[i], in[i].heads, in[i].d, static_cast<int64_t>(in[i].heads) * in[i].d};
            } else {
                to[i] = tokens(out[i], i ? "out for k" : "out for q", some.sizes().slice(0, 2), index, some.scalar_type());
                if (to[i].heads != in[i].heads || to[i].d != d) refuse("out for %s must be %s, got %s", name, sizes_of(*in[i].t).c_str(), sizes_of(*to[i].t).c_str());
            }
        }
        const Tensor& freq = same(a[3], "inv_freq", index, at::kDouble);
        if (freq.numel() > INT_MAX / 2) refuse("inv_freq is too large");   // any other wrong size is the library's to refuse
        const int32_t* positions = nullptr;
        int n_axes = 0;
        const uint8_t* axes = axes_of(a[9], freq.numel());
        if (axes) {
            if (is_none(a[4])) refuse("axes without positions");
            const Tensor& p = same(a[4], "positions", index, at::kInt);
            if (p.dim() != 3 || p.size(1) != B || p.size(2) != N || p.size(0) > INT_MAX)
                refuse("positions must be [axes, %lld, %lld], got %s", static_cast<long long>(B), static_cast<long long>(N), sizes_of(p).c_str());
            positions = static_cast<const int32_t*>(p.data_ptr());
            n_axes = static_cast<int>(p.size(0));
        } else if (!is_none(a[4])) {
            positions = ints(a[4], "positions", index, B * N);
        }
        const bool interleaved = truth(a[5]);
        const float factor = number(a[6]);
        // A tensor without elements (no tokens, no heads) has nothing to rotate; the other may.
        const auto held = [](const Tokens& t) { return t.t && t.t->numel() > 0; };
        if (held(in[0]) || held(in[1])) {
            const int rot = 2 * static_cast<int>(freq.numel());
            const auto ptr = [&](const Tokens& t) { return held(t) ? t.t->data_ptr() : nullptr; };
            const double* w = static_cast<const double*>(freq.data_ptr());
            const char* where = axes ? (backward ? "swiattn_rope_axes_backward" : "swiattn_rope_axes") : backward ? "swiattn_rope_backward" : "swiattn_rope";
            call(where, index, [&](void* stream) {
                const int b = static_cast<int>(B), s = static_cast<int>(N), h = static_cast<int>(d);
                if (axes)
                    return (backward ? g_lib.rope_axes_backward : g_lib.rope_axes)(ptr(in[0]), ptr(in[1]), positions, axes, n_axes, w, ptr(to[0]), ptr(to[1]), b, s, in[0].heads,
                                                                                  in[1].heads, h, rot, interleaved, factor, in[0].step, in[1].step, to[0].step, to[1].step, kind, stream);
                return (backward ? g_lib.rope_backward : g_lib.rope)(ptr(in[0]), ptr(in[1]), positions, w, ptr(to[0]), ptr(to[1]), b, s, in[0].heads, in[1].heads, h, rot, interleaved,
                                                                    factor, in[0].step, in[1].step, to[0].step, to[1].step, kind, stream);
            });
        }
        PyObject* r[2];
        for (int i = 0; i < 2; ++i) r[i] = is_none(x[i]) || !is_none(out[i]) ? new_ref(out[i]) : THPVariable_Wrap(made[i]);
        return pair(r[0], r[1]);
    });
}

// q, k, v, k_pages, v_pages, block_table, seq_lens, inv_freq, starts, interleaved, factor, k_exp, v_exp, out, positions, axes
PyObject* append_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 16, [&]() -> PyObject* {
        const Tensor& k0 = first(a[1], "k");
        const int index = k0.get_device();
        if (k0.dim() != 3) refuse("k must be [T, Hkv, d], got %s", sizes_of(k0).c_str());
        const int kind = kind_of(k0);
        const ScalarType type = k0.scalar_type();
        const auto lead = k0.sizes().slice(0, 1);
        const int64_t T = lead[0];
        if (T > INT_MAX) refuse("too many tokens");
        const Tokens k = tokens(a[1], "k", lead, index, type), v = tokens(a[2], "v", lead, index, type);
        if (v.heads != k.heads || v.d != k.d) refuse("k and v must have one shape");
        Tokens q = {};
        Tensor made;
        void* q_out = nullptr;
        PyObject* out = a[13];
        if (!is_none(a[0])) {
            q = tokens(a[0], "q", lead, index, type);
            if (q.d != k.d) refuse("q and k must have one head size");
            if (is_none(out)) {
                made = fresh(q.t->sizes(), k0, type);
                q_out = made.data_ptr();
            } else {
                const Tensor& o = same(out, "out", index, type);
                if (o.sizes() != q.t->sizes()) refuse("out must be %s, got %s", sizes_of(*q.t).c_str(), sizes_of(o).c_str());
                q_out = o.data_ptr();
            }
        } else if (!is_none(out)) {
            refuse("out without q");
        }
        const Tensor& pages = same(a[3], "k_pages", index);
        if (pages.scalar_type() != type && pages.scalar_type() != at::kFloat8_e4m3fn)
            refuse("pages must be %s or float8_e4m3fn, got %s", c10::toString(type), c10::toString(pages.scalar_type()));
        const Pools p = pools(a[3], a[4], a[11], a[12], index, false);
        if (p.Hkv != k.heads || p.d != k.d) refuse("k_pages and v_pages must be [num_pages, page_size, Hkv, d]");
        const Sequences s = sequences(a[5], a[6], index);
        const int32_t* starts = is_none(a[8]) ? nullptr : ints(a[8], "starts", index, s.B + int64_t(1));
        const double* freq = nullptr;
        int64_t half = 0;
        if (!is_none(a[7])) {
            const Tensor& f = same(a[7], "inv_freq", index, at::kDouble);
            freq = static_cast<const double*>(f.data_ptr());
            half = f.numel();
            if (half > INT_MAX / 2) refuse("inv_freq is too large");
        }
        const int32_t* positions = nullptr;
        const uint8_t* axes = nullptr;
        int n_axes = 1;
        if (!is_none(a[14]) || !is_none(a[15])) {
            if (is_none(a[7]) || is_none(a[14])) refuse("positions turn by inv_freq, and axes are of positions");
            const Tensor& given = same(a[14], "positions", index, at::kInt);
            axes = axes_of(a[15], half);
            if (given.dim() != (axes ? 2 : 1) || given.size(given.dim() - 1) != T || given.size(0) > INT_MAX)
                refuse("positions must be [%lld], or [axes, %lld] with axes, got %s", static_cast<long long>(T), static_cast<long long>(T), sizes_of(given).c_str());
            positions = static_cast<const int32_t*>(given.data_ptr());
            if (axes) n_axes = static_cast<int>(given.size(0));
        }
        const bool interleaved = truth(a[9]);
        const float factor = number(a[10]);
        const int rot = 2 * static_cast<int>(half), t = static_cast<int>(T);
        const void* q_in = q.t ? q.t->data_ptr() : nullptr;
        const bool at_positions = !is_none(a[14]);
        call(at_positions ? "swiattn_append_paged_at" : "swiattn_append_paged", index, [&](void* stream) {
            if (at_positions)
                return g_lib.append_paged_at(q_in, k.t->data_ptr(), v.t->data_ptr(), starts, s.lens, s.table, positions, axes, n_axes, freq, q_out, p.k, p.v, p.k_exp, p.v_exp, t, s.B,
                                             s.max_pages, p.page_size, p.num_pages, q.heads, k.heads, k.d, rot, interleaved, factor, q.step, k.step, v.step, kind, p.kind, stream);
            return g_lib.append_paged(q_in, k.t->data_ptr(), v.t->data_ptr(), starts, s.lens, s.table, freq, q_out, p.k, p.v, p.k_exp, p.v_exp, t, s.B, s.max_pages, p.page_size, p.num_pages,
                                      q.heads, k.heads, k.d, rot, interleaved, factor, q.step, k.step, v.step, kind, p.kind, stream);
        });
        if (!q.t || !is_none(out)) return new_ref(out);
        return THPVariable_Wrap(made);
    });
}

// q, k_pages, v_pages, block_table, seq_lens, starts, parents, gate, W, scale, out, want_lse, workspace, n_anchor, k_exp, v_exp
PyObject* decode_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 16, [&]() -> PyObject* {
        const Tensor& q0 = first(a[0], "q");
        const int index = q0.get_device();
        const Tensor& q = same(a[0], "q", index);
        if (q.dim() != 3) refuse("q must be [T, Hq, d], got %s", sizes_of(q).c_str());
        const int kind = kind_of(q);
        const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2);
        if (T > INT_MAX || Hq > INT_MAX || d > INT_MAX) refuse("q is too large");
        const Pools p = pools(a[1], a[2], a[14], a[15], index, false);
        if (p.d != d) refuse("k_pages and v_pages must be [num_pages, page_size, Hkv, d]");
        const Sequences s = sequences(a[3], a[4], index);
        const int32_t* starts = ints(a[5], "starts", index, s.B + int64_t(1));
        int64_t count = T;
        const int32_t* parents = parents_of(a[6], index, count);
        const Tensor& gate = same(a[7], "gate", index, at::kByte);
        if (count != T || gate.numel() != T) refuse("parents and gate must hold %lld values", static_cast<long long>(T));
        const int W = whole(a[8], "W"), n_anchor = whole(a[13], "n_anchor");
        const float scale = is_none(a[9]) ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(d))) : number(a[9]);
        Tensor made, lse, ws;
        void* o;
        if (is_none(a[10])) {
            made = fresh(q.sizes(), q, q.scalar_type());
            o = made.data_ptr();
        } else {
            const Tensor& out = same(a[10], "out", index, q.scalar_type());
            if (out.sizes() != q.sizes()) refuse("out must be %s, got %s", sizes_of(q).c_str(), sizes_of(out).c_str());
            o = out.data_ptr();
        }
        const bool want_lse = truth(a[11]);
        if (want_lse) lse = fresh({T, Hq}, q, at::kFloat);
        if (is_none(a[12])) {
            const size_t bytes = g_lib.decode_tree_workspace(static_cast<int>(T), s.B, static_cast<int>(Hq), p.Hkv, static_cast<int>(d), kind);
            ws = fresh({static_cast<int64_t>(bytes < 256 ? 256 : bytes)}, q, at::kByte);
        } else {
            ws = same(a[12], "workspace", index, at::kByte);
        }
        const uint8_t* gates = static_cast<const uint8_t*>(gate.data_ptr());
        float* l = want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr;
        call("swiattn_decode_tree", index, [&](void* stream) {
            return g_lib.decode_tree(q.data_ptr(), p.k, p.v, p.k_exp, p.v_exp, s.table, s.lens, starts, parents, gates, o, l, static_cast<int>(T), s.B, s.max_pages, p.page_size, p.num_pages,
                                     static_cast<int>(Hq), p.Hkv, static_cast<int>(d), W, n_anchor, scale, kind, p.kind, ws.data_ptr(), static_cast<size_t>(ws.numel()), stream);
        });
        PyObject* r = is_none(a[10]) ? THPVariable_Wrap(made) : new_ref(a[10]);
        return want_lse ? pair(r, THPVariable_Wrap(lse)) : r;
    });
}

// k_pages, v_pages, block_table, seq_lens, starts, parents, leaf, k_exp, v_exp, out
PyObject* accept_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject* {
        const Tensor& pages = first(a[0], "k_pages");
        const int index = pages.get_device();
        const Pools p = pools(a[0], a[1], a[7], a[8], index, true);
        const Sequences s = sequences(a[2], a[3], index);
        const int32_t* starts = ints(a[4], "starts", index, s.B + int64_t(1));
        int64_t T = INT_MAX;
        const int32_t* parents = parents_of(a[5], index, T);
        if (T > INT_MAX) refuse("too many tokens");
        const int32_t* leaf = ints(a[6], "leaf", index, s.B);
        Tensor made;
        int32_t* lens;
        if (is_none(a[9])) {
            made = fresh({s.B}, pages, at::kInt);
            lens = static_cast<int32_t*>(made.data_ptr());
        } else {
            lens = const_cast<int32_t*>(ints(a[9], "out", index, s.B));
        }
        call("swiattn_accept_tree", index, [&](void* stream) {
            return g_lib.accept_tree(p.k, p.v, p.k_exp, p.v_exp, s.table, s.lens, starts, parents, leaf, lens, p.layers, static_cast<int>(T), s.B, s.max_pages, p.page_size, p.num_pages, p.Hkv,
                                     p.d, p.kind, stream);
        });
        return is_none(a[9]) ? THPVariable_Wrap(made) : new_ref(a[9]);
    });
}

// k_pages, v_pages, block_table, seq_lens, source, new_page, k_exp, v_exp, table_out, lens_out
PyObject* fork_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject* {
        const Tensor& pages = first(a[0], "k_pages");
        const int index = pages.get_device();
        const Pools p = pools(a[0], a[1], a[6], a[7], index, true);
        const Sequences s = sequences(a[2], a[3], index);
        const Tensor& source = same(a[4], "source", index, at::kInt);
        const int64_t C = source.numel();
        if (C > INT_MAX) refuse("too many children");
        const int32_t* new_page = ints(a[5], "new_page", index, C);
        Tensor table, lens;
        int32_t *table_to, *lens_to;
        const bool make = is_none(a[8]) && is_none(a[9]);
        if (make) {
            table = fresh({C, s.max_pages}, pages, at::kInt);
            lens = fresh({C}, pages, at::kInt);
            table_to = static_cast<int32_t*>(table.data_ptr());
            lens_to = static_cast<int32_t*>(lens.data_ptr());
        } else {
            const Tensor& t = same(a[8], "out", index, at::kInt);
            if (t.dim() != 2 || t.size(0) != C || t.size(1) != s.max_pages) refuse("out must be [%lld, %d] and [%lld]", static_cast<long long>(C), s.max_pages, static_cast<long long>(C));
            table_to = static_cast<int32_t*>(t.data_ptr());
            lens_to = const_cast<int32_t*>(ints(a[9], "out", index, C));
        }
        const int32_t* from = static_cast<const int32_t*>(source.data_ptr());
        call("swiattn_fork_paged", index, [&](void* stream) {
            return g_lib.fork_paged(p.k, p.v, p.k_exp, p.v_exp, s.table, s.lens, from, new_page, table_to, lens_to, p.layers, s.B, static_cast<int>(C), s.max_pages, p.page_size, p.num_pages,
                                    p.Hkv, p.d, p.kind, stream);
        });
        if (!make) return pair(new_ref(a[8]), new_ref(a[9]));
        return pair(THPVariable_Wrap(table), THPVariable_Wrap(lens));
    });
}

// {name: address}, SwiAttnError
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 2, [&]() -> PyObject* {
        address(a[0], "swiattn_rope", g_lib.rope);
        address(a[0], "swiattn_rope_backward", g_lib.rope_backward);
        address(a[0], "swiattn_rope_axes", g_lib.rope_axes);
        address(a[0], "swiattn_rope_axes_backward", g_lib.rope_axes_backward);
        address(a[0], "swiattn_append_paged", g_lib.append_paged);
        address(a[0], "swiattn_append_paged_at", g_lib.append_paged_at);
        address(a[0], "swiattn_decode_tree", g_lib.decode_tree);
        address(a[0], "swiattn_decode_tree_workspace", g_lib.decode_tree_workspace);
        address(a[0], "swiattn_accept_tree", g_lib.accept_tree);
        address(a[0], "swiattn_fork_paged", g_lib.fork_paged);
        Py_XDECREF(g_error);
        g_error = new_ref(a[1]);
        Py_RETURN_NONE;
    });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(bind), FAST(rope), FAST(append_paged), FAST(decode_tree), FAST(accept_tree), FAST(fork_paged), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
