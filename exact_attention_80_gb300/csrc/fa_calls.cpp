// fa_calls.cpp — the Python module `_calls`: rope, kv_append_fp8,
// attention_paged_fp8, attention_window and attention_window_backward for plain
// arguments, from the tensors' checks to the launch.
//
// A call on a few tokens takes the GPU a few microseconds, so the interpreter's
// share of it counts (one call after the other, us, with ctypes and here: 8
// rotated tokens 15 and 5.2, 128 appended ones 19 and 4.4, one token decoded over
// 516 keys 20 and 7.4). A call that is not plain (a tensor of another type, shape, layout or
// device than the operator takes, a subclass, an argument that is not a number)
// returns None before anything happened: the Python form of the same call then
// says what is wrong, or handles it. A status other than FA_OK is returned as a
// number.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <cstring>

#include "fa.h"

namespace {

// The library's entry points, handed over by init().
struct {
    decltype(&::fa_rope) rope;
    decltype(&::fa_kv_append_fp8) append;
    decltype(&::fa_fwd_paged_fp8) paged;
    decltype(&::fa_paged_num_splits) num_splits;
    decltype(&::fa_paged_workspace_bytes) workspace_bytes;
    decltype(&::fa_fwd_window) window;
    decltype(&::fa_bwd_window) window_backward;
    decltype(&::fa_bwd_window_workspace_bytes) window_workspace;
    decltype(&::fa_window_num_splits) window_splits;
    decltype(&::fa_fwd_window_splitkv) window_splitkv;
    decltype(&::fa_combine) combine;
} lib;

bool tensor(PyObject* o, const at::Tensor** t) {
    if (!THPVariable_CheckExact(o)) return false;
    *t = &THPVariable_Unpack(o);
    return true;
}
bool number(PyObject* o, int* out) {
    if (!PyLong_CheckExact(o)) return false;
    int overflow = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &overflow);
    if (overflow || x < INT_MIN || x > INT_MAX) return false;
    *out = static_cast<int>(x);
    return true;
}
bool flag(PyObject* o, int* out) {
    if (o != Py_True && o != Py_False) return false;
    *out = o == Py_True;
    return true;
}

// A bf16 tensor [B, H, N, d] or [N, H, d] on device `index` with contiguous columns.
struct Heads {
    long long B, H, N, d, sb, sh, sn;
};
bool heads(const at::Tensor& t, int index, Heads* v) {
    if (t.layout() != at::kStrided || t.scalar_type() != at::kBFloat16 || !t.is_cuda() || t.get_device() != index ||
        t.numel() == 0)
        return false;
    const auto n = t.sizes(), s = t.strides();
    if (t.dim() == 4) {
        *v = {n[0], n[1], n[2], n[3], n[0] > 1 ? s[0] : 0, n[1] > 1 ? s[1] : 0, n[2] > 1 ? s[2] : 0};
        return s[3] == 1 && n[0] <= INT_MAX && n[1] <= INT_MAX && n[2] <= INT_MAX && n[3] <= INT_MAX;
    }
    if (t.dim() == 3) {
        *v = {1, n[1], n[0], n[2], 0, n[1] > 1 ? s[1] : 0, n[0] > 1 ? s[0] : 0};
        return s[2] == 1 && n[0] <= INT_MAX && n[1] <= INT_MAX && n[2] <= INT_MAX;
    }
    return false;
}
// A packed bf16 tensor [tokens, heads, d] whose heads and columns are contiguous.
struct Tokens {
    long long n, h, d, stride;
};
bool tokens(const at::Tensor& t, int index, Tokens* v) {
    if (t.layout() != at::kStrided || t.scalar_type() != at::kBFloat16 || !t.is_cuda() || t.get_device() != index ||
        t.dim() != 3 || t.numel() == 0)
        return false;
    const auto n = t.sizes(), s = t.strides();
    *v = {n[0], n[1], n[2], n[0] > 1 ? s[0] : n[1] * n[2]};
    return s[2] == 1 && (n[1] == 1 || s[1] == n[2]) && n[0] <= INT_MAX && n[1] <= INT_MAX && n[2] <= INT_MAX;
}
bool array(const at::Tensor& t, at::ScalarType type, int index) {
    return t.layout() == at::kStrided && t.scalar_type() == type && t.is_cuda() && t.get_device() == index &&
           t.is_contiguous();
}

// fa_rotation of a table and of `axes` rows of positions (null: none) for tokens
// [B, N] (`dense`) or [N].
bool rotation(const at::Tensor& table, const at::Tensor* positions, long long axes, PyObject* sections,
              int interleaved, bool dense, long long B, long long N, int index, fa_rotation* r) {
    if (!array(table, at::kFloat, index) || table.dim() != 2 || table.size(0) > INT_MAX || table.size(1) > INT_MAX)
        return false;
    if (axes < 1 || axes > FA_MAX_AXES) return false;
    std::memset(r, 0, sizeof(*r));
    if (positions) {
        if (!array(*positions, at::kInt, index)) return false;
        const auto n = positions->sizes();
        const size_t dim = n.size(), tokens = dense ? 2 : 1;  // dimensions of the tokens
        const bool fits = (dim == tokens || dim == tokens + 1) && n[dim - 1] == N && (!dense || n[dim - 2] == B);
        // (One axis of [B, N] tokens may come flat.)
        if (!fits && !(dense && axes == 1 && positions->numel() == B * N && (dim == 1 || (dim == 2 && n[0] == 1))))
            return false;
        r->positions = static_cast<const int*>(positions->data_ptr());
    }
    r->table = static_cast<const float*>(table.data_ptr());
    r->max_pos = static_cast<int>(table.size(0));
    r->rot = static_cast<int>(table.size(1));
    r->axes = static_cast<int>(axes);
    r->interleaved = interleaved;
    if (sections == Py_None) {
        if (axes != 1) return false;
        r->sections[0] = r->rot / 2;
        return true;
    }
    const bool list = PyList_CheckExact(sections);
    if (!list && !PyTuple_CheckExact(sections)) return false;
    if ((list ? PyList_GET_SIZE(sections) : PyTuple_GET_SIZE(sections)) != axes) return false;
    for (long long a = 0; a < axes; ++a)
        if (!number(list ? PyList_GET_ITEM(sections, a) : PyTuple_GET_ITEM(sections, a), &r->sections[a])) return false;
    return true;
}

// The cache's four tensors and the batch's three.
struct Paged {
    fa_paged_cache cache;
    const int *table, *cu, *lens;
    int B, max_pages;
};
bool paged(PyObject* const* a, int index, Paged* p) {
    const at::Tensor* t[7];
    for (int i = 0; i < 7; ++i)
        if (!tensor(a[i], &t[i])) return false;
    if (t[0]->dim() != 4 || t[0]->sizes() != t[1]->sizes()) return false;
    const auto n = t[0]->sizes();
    for (int i = 0; i < 2; ++i) {
        const at::ScalarType type = t[i]->scalar_type();
        if ((type != at::kByte && type != at::kFloat8_e4m3fn) || !array(*t[i], type, index)) return false;
        const at::Tensor& s = *t[2 + i];
        if (!array(s, at::kFloat, index) || s.dim() != 2 || s.size(0) != n[0] || s.size(1) != n[1]) return false;
    }
    for (int i = 0; i < 4; ++i)
        if (n[i] > INT_MAX) return false;
    for (int i = 4; i < 7; ++i)
        if (!array(*t[i], at::kInt, index)) return false;
    if (t[4]->dim() != 2 || t[5]->dim() != 1 || t[6]->dim() != 1) return false;
    const long long B = t[4]->size(0), width = t[4]->size(1);
    if (B < 1 || B >= INT_MAX || width > INT_MAX || t[5]->size(0) != B + 1 || t[6]->size(0) != B) return false;
    p->cache = {t[0]->data_ptr(), t[1]->data_ptr(), static_cast<float*>(t[2]->data_ptr()),
                static_cast<float*>(t[3]->data_ptr()), static_cast<int>(n[0]), static_cast<int>(n[1]),
                static_cast<int>(n[2]), static_cast<int>(n[3])};
    p->table = static_cast<const int*>(t[4]->data_ptr());
    p->cu = static_cast<const int*>(t[5]->data_ptr());
    p->lens = static_cast<const int*>(t[6]->data_ptr());
    p->B = static_cast<int>(B);
    p->max_pages = static_cast<int>(width);
    return true;
}

// q [B, H, Nq, d], k and v [B, Hkv, Nk, d] of a dense call, contiguous.
struct Dense {
    int B, H, Hkv, Nq, Nk, d;
};
bool dense(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, int index, Dense* c) {
    if (!array(q, at::kBFloat16, index) || !array(k, at::kBFloat16, index) || !array(v, at::kBFloat16, index))
        return false;
    if (q.dim() != 4 || k.dim() != 4 || v.sizes() != k.sizes()) return false;
    const auto n = q.sizes(), m = k.sizes();
    if (m[0] != n[0] || m[3] != n[3]) return false;
    for (int i = 0; i < 4; ++i)
        if (n[i] > INT_MAX || m[i] > INT_MAX) return false;
    *c = {static_cast<int>(n[0]), static_cast<int>(n[1]), static_cast<int>(m[1]),
          static_cast<int>(n[2]), static_cast<int>(m[2]), static_cast<int>(n[3])};
    return true;
}
// A scale argument: None is 1 / sqrt(d), rounded once to fp32.
bool scale_of(PyObject* o, int d, float* scale) {
    if (o != Py_None && !PyFloat_CheckExact(o)) return false;
    *scale = static_cast<float>(o == Py_None ? std::pow(static_cast<double>(d), -0.5) : PyFloat_AS_DOUBLE(o));
    return true;
}
// A tuple of new tensors.
PyObject* tuple_of(at::Tensor* t, int n) {
    PyObject* all = PyTuple_New(n);
    for (int i = 0; all && i < n; ++i) {
        PyObject* x = THPVariable_Wrap(std::move(t[i]));
        if (!x) {
            Py_DECREF(all);
            return nullptr;
        }
        PyTuple_SET_ITEM(all, i, x);
    }
    return all;
}

// The index of a CUDA tensor's device if it is the current one, else -1.
int current_index(const at::Tensor& t) {
    if (!t.is_cuda()) return -1;
    const int index = t.get_device();
    return index == c10::cuda::current_device() ? index : -1;
}
template <typename F>
fa_status launch(int index, F&& call) {
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
    fa_status s;
    Py_BEGIN_ALLOW_THREADS
    s = call(stream);
    Py_END_ALLOW_THREADS
    return s;
}

#define NOT_PLAIN_UNLESS(x) \
    if (!(x)) Py_RETURN_NONE

// rope(q, k or None, table, positions, sections, interleaved, inverse) -> q_out or (q_out, k_out)
PyObject* call_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *t[2] = {nullptr, nullptr}, *table, *positions;
    NOT_PLAIN_UNLESS(n == 7 && tensor(a[0], &t[0]) && (a[1] == Py_None || tensor(a[1], &t[1])) &&
                     tensor(a[2], &table) && tensor(a[3], &positions));
    int interleaved, inverse;
    NOT_PLAIN_UNLESS(flag(a[5], &interleaved) && flag(a[6], &inverse));
    const int index = current_index(*t[0]);
    Heads v[2];
    NOT_PLAIN_UNLESS(index >= 0 && heads(*t[0], index, &v[0]));
    if (t[1]) {
        NOT_PLAIN_UNLESS(t[1]->dim() == t[0]->dim() && heads(*t[1], index, &v[1]) && v[1].B == v[0].B &&
                         v[1].N == v[0].N && v[1].d == v[0].d);
    }
    const long long axes = positions->dim() == t[0]->dim() - 1 ? positions->size(0) : 1;
    fa_rotation r;
    NOT_PLAIN_UNLESS(rotation(*table, positions, axes, a[4], interleaved, t[0]->dim() == 4, v[0].B, v[0].N, index, &r));
    at::Tensor out[2];
    fa_rope_tensor x[2];
    for (int i = 0; i < (t[1] ? 2 : 1); ++i) {
        const Heads& w = v[i];
        out[i] = at::empty(t[i]->sizes(), t[i]->options());
        const bool packed = t[i]->dim() == 3;
        x[i] = {t[i]->data_ptr(), out[i].data_ptr(), static_cast<int>(w.H), {w.sb, w.sh, w.sn},
                {packed ? 0 : w.H * w.N * w.d, packed ? w.d : w.N * w.d, packed ? w.H * w.d : w.d}};
    }
    const fa_status s = launch(index, [&](cudaStream_t stream) {
        return lib.rope(&x[0], t[1] ? &x[1] : nullptr, &r, static_cast<int>(v[0].B), static_cast<int>(v[0].N),
                        static_cast<int>(v[0].d), inverse, stream);
    });
    if (s != FA_OK) return PyLong_FromLong(s);
    return t[1] ? tuple_of(out, 2) : THPVariable_Wrap(std::move(out[0]));
    END_HANDLE_TH_ERRORS
}

// append(q or None, k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, seqlens_k, max_seqlen, table or
// None, positions or None, sections, interleaved) -> q_out, or True without queries
PyObject* call_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *q = nullptr, *k, *v, *table = nullptr, *positions = nullptr;
    NOT_PLAIN_UNLESS(n == 15 && (a[0] == Py_None || tensor(a[0], &q)) && tensor(a[1], &k) && tensor(a[2], &v) &&
                     (a[11] == Py_None || tensor(a[11], &table)) && (a[12] == Py_None || tensor(a[12], &positions)));
    int max_new, interleaved;
    NOT_PLAIN_UNLESS(number(a[10], &max_new) && flag(a[14], &interleaved) && (table || !positions));
    const int index = current_index(*k);
    Tokens kt, vt, qt = {0, 0, 0, 0};
    Paged p;
    NOT_PLAIN_UNLESS(index >= 0 && tokens(*k, index, &kt) && tokens(*v, index, &vt) && paged(a + 3, index, &p));
    NOT_PLAIN_UNLESS(vt.n == kt.n && vt.h == kt.h && vt.d == kt.d && p.cache.Hkv == kt.h && p.cache.d == kt.d);
    if (q) {
        NOT_PLAIN_UNLESS(tokens(*q, index, &qt) && qt.n == kt.n && qt.d == kt.d);
    }
    fa_rotation r;
    if (table) {
        const long long axes = positions && positions->dim() == 2 ? positions->size(0) : 1;
        NOT_PLAIN_UNLESS(rotation(*table, positions, axes, a[13], interleaved, false, 1, kt.n, index, &r));
    }
    at::Tensor out;
    if (q) out = at::empty({qt.n, qt.h, qt.d}, q->options());
    const fa_status s = launch(index, [&](cudaStream_t stream) {
        return lib.append(q ? q->data_ptr() : nullptr, k->data_ptr(), v->data_ptr(), q ? out.data_ptr() : nullptr,
                          table ? &r : nullptr, &p.cache, p.table, p.cu, p.lens, p.B, static_cast<int>(qt.h),
                          static_cast<int>(kt.n), max_new, p.max_pages, qt.stride, kt.stride, vt.stride, stream);
    });
    if (s != FA_OK) return PyLong_FromLong(s);
    if (!q) Py_RETURN_TRUE;
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// paged(q, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens_q, seqlens_k, max_seqlen_q, max_seqlen_k, window,
// sinks, scale or None, num_splits or None) -> (o, lse)
PyObject* call_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor* q;
    int max_q, max_k, window, sinks, splits = 0;
    NOT_PLAIN_UNLESS(n == 14 && tensor(a[0], &q) && number(a[8], &max_q) && number(a[9], &max_k) &&
                     number(a[10], &window) && number(a[11], &sinks) && (a[13] == Py_None || number(a[13], &splits)));
    const int index = current_index(*q);
    Tokens t;
    Paged p;
    NOT_PLAIN_UNLESS(index >= 0 && tokens(*q, index, &t) && t.stride == t.h * t.d && paged(a + 1, index, &p) &&
                     p.cache.d == t.d);
    const int H = static_cast<int>(t.h), total = static_cast<int>(t.n), d = static_cast<int>(t.d);
    if (a[13] == Py_None) {
        splits = lib.num_splits(p.B, H, p.cache.Hkv, max_q, max_k, d, window, sinks);
        if (splits < 1) splits = 1;
    }
    float scale;
    NOT_PLAIN_UNLESS(scale_of(a[12], d, &scale));
    at::Tensor o = at::empty({t.n, t.h, t.d}, q->options());
    at::Tensor lse = at::empty({t.h, t.n}, q->options().dtype(at::kFloat));
    at::Tensor workspace;
    if (splits > 1)
        workspace = at::empty({static_cast<int64_t>(lib.workspace_bytes(total, H, d, splits) / 4)},
                              q->options().dtype(at::kFloat));
    const fa_status s = launch(index, [&](cudaStream_t stream) {
        return lib.paged(q->data_ptr(), &p.cache, p.table, p.cu, p.lens, o.data_ptr(),
                         static_cast<float*>(lse.data_ptr()), splits > 1 ? workspace.data_ptr() : nullptr, p.B, H,
                         total, max_q, max_k, p.max_pages, scale, window, sinks, splits, stream);
    });
    if (s != FA_OK) return PyLong_FromLong(s);
    at::Tensor out[2] = {std::move(o), std::move(lse)};
    return tuple_of(out, 2);
    END_HANDLE_TH_ERRORS
}

// window(q, k, v, window, sinks, scale or None, num_splits or None) -> (o, lse)
PyObject* call_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *q, *k, *v;
    int window, sinks, splits = 0;
    NOT_PLAIN_UNLESS(n == 7 && tensor(a[0], &q) && tensor(a[1], &k) && tensor(a[2], &v) && number(a[3], &window) &&
                     number(a[4], &sinks) && (a[6] == Py_None || (number(a[6], &splits) && splits >= 1 &&
                                                                 splits <= FA_MAX_SPLITS)));
    const int index = current_index(*q);
    Dense c;
    float scale;
    NOT_PLAIN_UNLESS(index >= 0 && dense(*q, *k, *v, index, &c) && scale_of(a[5], c.d, &scale));
    at::Tensor out[2] = {at::empty(q->sizes(), q->options()),
                         at::empty({c.B, c.H, c.Nq}, q->options().dtype(at::kFloat))};
    if (a[6] == Py_None) splits = lib.window_splits(c.B, c.H, c.Hkv, c.Nq, c.Nk, c.d, window, sinks);
    at::Tensor workspace;
    if (splits > 1)
        workspace = at::empty({static_cast<int64_t>(splits) * c.B * c.H * c.Nq * (c.d + 2)},
                              q->options().dtype(at::kFloat));
    const fa_status s = launch(index, [&](cudaStream_t stream) {
        if (splits > 1) {
            const fa_status first = lib.window_splitkv(q->data_ptr(), k->data_ptr(), v->data_ptr(),
                                                       workspace.data_ptr(), c.B, c.H, c.Hkv, c.Nq, c.Nk, c.d, scale,
                                                       window, sinks, splits, stream);
            if (first != FA_OK) return first;
            return lib.combine(workspace.data_ptr(), out[0].data_ptr(), static_cast<float*>(out[1].data_ptr()), c.B,
                               c.H, c.Nq, c.d, splits, stream);
        }
        return lib.window(q->data_ptr(), k->data_ptr(), v->data_ptr(), out[0].data_ptr(),
                          static_cast<float*>(out[1].data_ptr()), c.B, c.H, c.Hkv, c.Nq, c.Nk, c.d, scale, window,
                          sinks, stream);
    });
    return s == FA_OK ? tuple_of(out, 2) : PyLong_FromLong(s);
    END_HANDLE_TH_ERRORS
}

// window_backward(q, k, v, o, lse, dout, window, sinks, scale or None) -> (dq, dk, dv)
PyObject* call_window_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *q, *k, *v, *o, *lse, *dout;
    int window, sinks;
    NOT_PLAIN_UNLESS(n == 9 && tensor(a[0], &q) && tensor(a[1], &k) && tensor(a[2], &v) && tensor(a[3], &o) &&
                     tensor(a[4], &lse) && tensor(a[5], &dout) && number(a[6], &window) && number(a[7], &sinks));
    const int index = current_index(*q);
    Dense c;
    float scale;
    NOT_PLAIN_UNLESS(index >= 0 && dense(*q, *k, *v, index, &c) && scale_of(a[8], c.d, &scale));
    NOT_PLAIN_UNLESS(array(*o, at::kBFloat16, index) && o->sizes() == q->sizes() &&
                     array(*dout, at::kBFloat16, index) && dout->sizes() == q->sizes() &&
                     array(*lse, at::kFloat, index) && lse->sizes() == q->sizes().slice(0, 3));
    at::Tensor out[3] = {at::empty(q->sizes(), q->options()), at::empty(k->sizes(), k->options()),
                         at::empty(k->sizes(), k->options())};
    const size_t bytes = lib.window_workspace(c.B, c.H, c.Hkv, c.Nq, c.Nk, c.d, window, sinks);
    at::Tensor workspace = at::empty({static_cast<int64_t>(bytes < 4 ? 1 : bytes / 4)}, q->options().dtype(at::kFloat));
    const fa_status s = launch(index, [&](cudaStream_t stream) {
        return lib.window_backward(q->data_ptr(), k->data_ptr(), v->data_ptr(), o->data_ptr(), dout->data_ptr(),
                                   static_cast<const float*>(lse->data_ptr()), out[0].data_ptr(), out[1].data_ptr(),
                                   out[2].data_ptr(), workspace.data_ptr(), c.B, c.H, c.Hkv, c.Nq, c.Nk, c.d, scale,
                                   window, sinks, stream);
    });
    return s == FA_OK ? tuple_of(out, 3) : PyLong_FromLong(s);
    END_HANDLE_TH_ERRORS
}

// init: addresses of the library's entry points, in the order of `lib`.
PyObject* call_init(PyObject*, PyObject* args) {
    unsigned long long f[11];
    if (!PyArg_ParseTuple(args, "KKKKKKKKKKK", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &f[7], &f[8], &f[9],
                          &f[10]))
        return nullptr;
    lib.rope = reinterpret_cast<decltype(lib.rope)>(static_cast<uintptr_t>(f[0]));
    lib.append = reinterpret_cast<decltype(lib.append)>(static_cast<uintptr_t>(f[1]));
    lib.paged = reinterpret_cast<decltype(lib.paged)>(static_cast<uintptr_t>(f[2]));
    lib.num_splits = reinterpret_cast<decltype(lib.num_splits)>(static_cast<uintptr_t>(f[3]));
    lib.workspace_bytes = reinterpret_cast<decltype(lib.workspace_bytes)>(static_cast<uintptr_t>(f[4]));
    lib.window = reinterpret_cast<decltype(lib.window)>(static_cast<uintptr_t>(f[5]));
    lib.window_backward = reinterpret_cast<decltype(lib.window_backward)>(static_cast<uintptr_t>(f[6]));
    lib.window_workspace = reinterpret_cast<decltype(lib.window_workspace)>(static_cast<uintptr_t>(f[7]));
    lib.window_splits = reinterpret_cast<decltype(lib.window_splits)>(static_cast<uintptr_t>(f[8]));
    lib.window_splitkv = reinterpret_cast<decltype(lib.window_splitkv)>(static_cast<uintptr_t>(f[9]));
    lib.combine = reinterpret_cast<decltype(lib.combine)>(static_cast<uintptr_t>(f[10]));
    Py_RETURN_NONE;
}

// A fast-call function as the method table takes it.
PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"init", call_init, METH_VARARGS, nullptr},
    {"rope", fast(call_rope), METH_FASTCALL, nullptr},
    {"append", fast(call_append), METH_FASTCALL, nullptr},
    {"paged", fast(call_paged), METH_FASTCALL, nullptr},
    {"window", fast(call_window), METH_FASTCALL, nullptr},
    {"window_backward", fast(call_window_backward), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
    PyObject* m = PyModule_Create(&module);
    // Tensors are read through the headers of the PyTorch that this was built
    // against: the binding takes the module with no other.
    if (m && PyModule_AddStringConstant(m, "torch_version", FA_TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
