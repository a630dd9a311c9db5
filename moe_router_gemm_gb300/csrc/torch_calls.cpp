// torch_calls.cpp — the usual calls of the operators around the linear, marshalled in
// C++: a call that makes its own outputs and runs on the current stream.
//
// The kernels of a decode step take two to ten microseconds; a Python wrapper that
// checks five tensors, makes two and calls through ctypes takes fifteen.  These do the
// same checks on the tensors themselves and give None for anything they do not take
// (wrong types, shapes or devices, another current device): the Python wrapper then
// goes its own way, which says what is wrong or handles it.  They give the status as
// an int where the library refuses.  The library's entry points are handed in by
// address (bind), so there is one library, the one the wrapper has loaded.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "bf16_linear.h"

namespace {

decltype(&bf16_rmsnorm) g_rmsnorm;
decltype(&bf16_route) g_route;
decltype(&bf16_quant_mxfp4) g_quant;
decltype(&bf16_dequant_mxfp4) g_dequant;
decltype(&bf16_linear_mxfp4) g_linear;
decltype(&bf16_linear_mxfp4_dynamic) g_dynamic;
decltype(&bf16_linear_mxfp4_dynamic_workspace) g_workspace;
decltype(&bf16_group_rows) g_group;
decltype(&bf16_linear_grouped) g_grouped;
decltype(&bf16_combine_rows) g_combine;
decltype(&bf16_linear_lora) g_lora;
decltype(&bf16_linear_lora_workspace) g_lora_workspace;
decltype(&bf16_linear_grouped_workspace) g_grouped_workspace;

using at::Tensor;

// A defined CUDA tensor on the current device, or nothing.
const Tensor *cuda_tensor(PyObject *o) {
    if (!THPVariable_Check(o)) return nullptr;
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided || t.device().index() != c10::cuda::current_device())
        return nullptr;
    return &t;
}

// ... contiguous, of this type and shape.
const Tensor *dense(PyObject *o, at::ScalarType type, int64_t rows, int64_t cols) {
    const Tensor *t = cuda_tensor(o);
    if (!t || t->scalar_type() != type || t->dim() != 2 || t->size(0) != rows || t->size(1) != cols || !t->is_contiguous())
        return nullptr;
    return t;
}
const Tensor *dense(PyObject *o, at::ScalarType type, int64_t planes, int64_t rows, int64_t cols) {
    const Tensor *t = cuda_tensor(o);
    if (!t || t->scalar_type() != type || t->dim() != 3 || t->size(0) != planes || t->size(1) != rows ||
        t->size(2) != cols || !t->is_contiguous())
        return nullptr;
    return t;
}
const Tensor *dense(PyObject *o, at::ScalarType type, int64_t n) {
    const Tensor *t = cuda_tensor(o);
    if (!t || t->scalar_type() != type || t->dim() != 1 || t->size(0) != n || !t->is_contiguous()) return nullptr;
    return t;
}

// Elements between the rows of a 2-D tensor whose rows are contiguous, or -1.
int64_t pitch(const Tensor &t) {
    const int64_t rows = t.size(0), cols = t.size(1), ld = t.stride(0);
    if ((t.stride(1) != 1 && cols > 1) || (ld < cols && rows > 1)) return -1;
    return ld > cols ? ld : cols;
}

Tensor make(const Tensor &like, at::ScalarType type, at::IntArrayRef shape) {
    return at::empty(shape, like.options().dtype(type));
}

// A dense tensor of `base`'s type inside its memory, from element `first` (an allocation takes over a microsecond, this 0.2).
Tensor part_of(const Tensor &base, int64_t first, at::IntArrayRef shape) {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(), base.dtype());
    impl->set_sizes_contiguous(shape);
    impl->set_storage_offset(first);
    return Tensor(std::move(impl));
}

bf16l_stream_t stream_of(const Tensor &t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

PyObject *none() { Py_RETURN_NONE; }

PyObject *item(Tensor t) {
    if (t.defined()) return THPVariable_Wrap(std::move(t));
    Py_RETURN_NONE;
}

PyObject *pack(std::initializer_list<Tensor> list) {
    PyObject *r = PyTuple_New((Py_ssize_t)list.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor &t : list) {
        PyObject *o = item(t);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// The C ABI's int and flags of a Python number; `wide` where it does not fit (the wrapper then refuses it).
int as_int(PyObject *o, bool &wide) {
    int over = 0;
    const long v = PyLong_AsLongAndOverflow(o, &over);
    if (over || v < INT32_MIN || v > INT32_MAX) wide = true;
    return (int)v;
}
uint32_t as_flags(PyObject *o, bool &wide) {
    int over = 0;
    const long v = PyLong_AsLongAndOverflow(o, &over);
    if (over || v < 0 || v > (long)UINT32_MAX) wide = true;
    return (uint32_t)v;
}

// The interpreter is free while this lives: an allocation may wait for the device, and a launch waits where the stream has
// as many as it takes, maybe behind a host function that needs the interpreter.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

bool wrong_count(Py_ssize_t got, Py_ssize_t want) {
    if (got == want) return false;
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd are wanted", got, want);
    return true;
}

// rmsnorm(x, weight, residual, eps, quant, scale, bf16_out, flags)
PyObject *rmsnorm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (wrong_count(n, 8)) return nullptr;
    const double eps = PyFloat_AsDouble(args[3]);
    bool wide = false;
    const int quant = as_int(args[4], wide), want = PyObject_IsTrue(args[6]);
    const uint32_t flags = as_flags(args[7], wide);
    if (PyErr_Occurred() || want < 0) return nullptr;
    if (wide) return none();
    const Tensor *x = cuda_tensor(args[0]);
    if (!x || x->scalar_type() != at::kBFloat16 || x->dim() != 2) return none();
    const int64_t rows = x->size(0), H = x->size(1), ld = pitch(*x);
    const Tensor *w = dense(args[1], at::kBFloat16, H), *r = nullptr, *s = nullptr;
    const bool mx = quant == BF16L_QUANT_MXFP8 || quant == BF16L_QUANT_MXFP4;
    if (ld < 0 || !w || H > INT32_MAX || (!want && quant == BF16L_QUANT_NONE)) return none();
    if (args[2] != Py_None && !(r = dense(args[2], at::kBFloat16, rows, H))) return none();
    if (quant == BF16L_QUANT_FP8 ? !(s = dense(args[5], at::kFloat, 1)) : args[5] != Py_None) return none();
    Tensor out, sum, codes, scales;
    int st;
    {
        const Unlocked unlocked;
        if (r) sum = make(*x, at::kBFloat16, {rows, H});
        if (want) out = make(*x, at::kBFloat16, {rows, H});
        if (quant != BF16L_QUANT_NONE) codes = make(*x, at::kByte, {rows, quant == BF16L_QUANT_MXFP4 ? H / 2 : H});
        if (mx) scales = make(*x, at::kByte, {rows, H / 32});
        st = g_rmsnorm(x->const_data_ptr(), ld, r ? r->const_data_ptr() : nullptr, w->const_data_ptr(),
                       out.defined() ? out.data_ptr() : nullptr, sum.defined() ? sum.data_ptr() : nullptr,
                       codes.defined() ? codes.data_ptr() : nullptr, scales.defined() ? scales.data_ptr() : nullptr,
                       s ? static_cast<const float *>(s->const_data_ptr()) : nullptr, rows, (int)H, (float)eps, quant,
                       flags, stream_of(*x));
    }
    return st ? PyLong_FromLong(st) : pack({out, sum, codes, scales});
    END_HANDLE_TH_ERRORS
}

// route(logits, k, scoring, bias, groups, top_groups, group_best, renormalize, scale, flags)
PyObject *route(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (wrong_count(n, 10)) return nullptr;
    bool wide = false;
    const int k = as_int(args[1], wide), scoring = as_int(args[2], wide), groups = as_int(args[4], wide),
              top = as_int(args[5], wide), best = as_int(args[6], wide);
    const uint32_t flags = as_flags(args[9], wide);
    const int renorm = PyObject_IsTrue(args[7]);
    const double scale = PyFloat_AsDouble(args[8]);
    if (PyErr_Occurred() || renorm < 0) return nullptr;
    if (wide) return none();
    const Tensor *l = cuda_tensor(args[0]), *b = nullptr;
    if (!l || l->dim() != 2 || (l->scalar_type() != at::kFloat && l->scalar_type() != at::kBFloat16)) return none();
    const int64_t T = l->size(0), E = l->size(1), ld = pitch(*l);
    if (ld < 0 || E > INT32_MAX || k < 1 || k > 1024) return none();
    if (args[3] != Py_None && !(b = dense(args[3], at::kFloat, E))) return none();
    Tensor w, ids;
    int st;
    {
        const Unlocked unlocked;
        w = make(*l, at::kFloat, {T, k});
        ids = make(*l, at::kInt, {T, k});
        st = g_route(l->const_data_ptr(), ld, b ? static_cast<const float *>(b->const_data_ptr()) : nullptr,
                     static_cast<float *>(w.data_ptr()), static_cast<int32_t *>(ids.data_ptr()), T, (int)E, k, scoring,
                     groups, top, best, renorm, (float)scale, l->scalar_type() == at::kBFloat16, flags, stream_of(*l));
    }
    return st ? PyLong_FromLong(st) : pack({w, ids});
    END_HANDLE_TH_ERRORS
}

// quant_mxfp4(x, flags)
PyObject *quant_mxfp4(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (wrong_count(n, 2)) return nullptr;
    bool wide = false;
    const uint32_t flags = as_flags(args[1], wide);
    if (PyErr_Occurred()) return nullptr;
    if (wide) return none();
    const Tensor *x = cuda_tensor(args[0]);
    if (!x || x->dim() != 2 || x->scalar_type() != at::kBFloat16 || !x->is_contiguous()) return none();
    const int64_t rows = x->size(0), K = x->size(1);
    if (K > INT32_MAX) return none();
    Tensor q, s;
    int st;
    {
        const Unlocked unlocked;
        q = make(*x, at::kByte, {rows, K / 2});
        s = make(*x, at::kByte, {rows, K / 32});
        st = g_quant(x->const_data_ptr(), rows, (int)K, q.data_ptr(), s.data_ptr(), flags, stream_of(*x));
    }
    return st ? PyLong_FromLong(st) : pack({q, s});
    END_HANDLE_TH_ERRORS
}

// dequant_mxfp4(codes, scales, flags)
PyObject *dequant_mxfp4(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (wrong_count(n, 3)) return nullptr;
    bool wide = false;
    const uint32_t flags = as_flags(args[2], wide);
    if (PyErr_Occurred()) return nullptr;
    if (wide) return none();
    const Tensor *q = cuda_tensor(args[0]);
    if (!q || q->dim() != 2 || q->scalar_type() != at::kByte || !q->is_contiguous()) return none();
    const int64_t rows = q->size(0), h = q->size(1);
    const Tensor *s = dense(args[1], at::kByte, rows, h / 16);
    if (!s || 2 * h > INT32_MAX) return none();
    Tensor out;
    int st;
    {
        const Unlocked unlocked;
        out = make(*q, at::kBFloat16, {rows, 2 * h});
        st = g_dequant(q->const_data_ptr(), s->const_data_ptr(), rows, (int)(2 * h), out.data_ptr(), flags, stream_of(*q));
    }
    return st ? PyLong_FromLong(st) : item(out);
    END_HANDLE_TH_ERRORS
}

// linear_mxfp4(x, xs, wq, ws, bias, flags): xs None for a bf16 x that the call quantises
PyObject *linear_mxfp4(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (wrong_count(n, 6)) return nullptr;
    bool wide = false;
    const uint32_t flags = as_flags(args[5], wide);
    if (PyErr_Occurred()) return nullptr;
    if (wide) return none();
    const bool dynamic = args[1] == Py_None;
    const Tensor *x = cuda_tensor(args[0]), *wq = cuda_tensor(args[2]), *xs = nullptr, *b = nullptr;
    if (!x || !wq || x->dim() != 2 || wq->dim() != 2 || !x->is_contiguous() ||
        x->scalar_type() != (dynamic ? at::kBFloat16 : at::kByte))
        return none();
    const int64_t M = x->size(0), K = dynamic ? x->size(1) : 2 * x->size(1), N = wq->size(0);
    const Tensor *ws = dense(args[3], at::kByte, N, K / 32);
    if (!ws || !dense(args[2], at::kByte, N, K / 2) || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return none();
    if (!dynamic && !(xs = dense(args[1], at::kByte, M, K / 32))) return none();
    if (args[4] != Py_None && !(b = dense(args[4], at::kBFloat16, N))) return none();
    Tensor out;
    const void *bias = b ? b->const_data_ptr() : nullptr;
    int st;
    {
        const Unlocked unlocked;
        out = make(*x, at::kBFloat16, {M, N});
        if (dynamic) {
            Tensor space;  // freed on return, to this stream's own memory
            const size_t need = g_workspace((int)M, (int)N, (int)K);
            if (need) space = make(*x, at::kByte, {(int64_t)need});
            st = g_dynamic(x->const_data_ptr(), wq->const_data_ptr(), ws->const_data_ptr(), bias, out.data_ptr(), (int)M,
                           (int)N, (int)K, need ? space.data_ptr() : nullptr, need, flags, stream_of(*x));
        } else {
            st = g_linear(x->const_data_ptr(), xs->const_data_ptr(), wq->const_data_ptr(), ws->const_data_ptr(), bias,
                          out.data_ptr(), (int)M, (int)N, (int)K, flags, stream_of(*x));
        }
    }
    return st ? PyLong_FromLong(st) : item(out);
    END_HANDLE_TH_ERRORS
}

// group_rows(ids, groups, flags)
PyObject *group_rows(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (wrong_count(n, 3)) return nullptr;
    bool wide = false;
    const int groups = as_int(args[1], wide);
    const uint32_t flags = as_flags(args[2], wide);
    if (PyErr_Occurred()) return nullptr;
    if (wide || groups < 1 || groups > 65536) return none();
    const Tensor *ids = cuda_tensor(args[0]);
    if (!ids || ids->scalar_type() != at::kInt || ids->dim() < 1 || ids->dim() > 2 || !ids->is_contiguous()) return none();
    const int64_t T = ids->size(0), k = ids->dim() == 2 ? ids->size(1) : 1;
    if (k < 1 || k > INT32_MAX) return none();
    Tensor offsets, rows, place;
    int st;
    {
        const Unlocked unlocked;
        const int64_t rows_at = (groups + 1 + 63) / 64 * 64, place_at = rows_at + (T * k + 63) / 64 * 64;  // (256 bytes)
        const Tensor all = make(*ids, at::kInt, {place_at + T * k});
        offsets = part_of(all, 0, {groups + 1});
        rows = part_of(all, rows_at, {T * k});
        place = part_of(all, place_at, ids->sizes());
        st = g_group(static_cast<const int32_t *>(ids->const_data_ptr()), T, (int)k, groups,
                     static_cast<int32_t *>(offsets.data_ptr()), static_cast<int32_t *>(rows.data_ptr()),
                     static_cast<int32_t *>(place.data_ptr()), flags, stream_of(*ids));
    }
    return st ? PyLong_FromLong(st) : pack({offsets, rows, place});
    END_HANDLE_TH_ERRORS
}

// linear_grouped(x, w, offsets, bias, rows, swiglu, flags)
PyObject *linear_grouped(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (wrong_count(n, 7)) return nullptr;
    bool wide = false;
    const int swiglu = PyObject_IsTrue(args[5]);
    const uint32_t flags = as_flags(args[6], wide);
    if (PyErr_Occurred() || swiglu < 0) return nullptr;
    if (wide) return none();
    const Tensor *x = cuda_tensor(args[0]), *w = cuda_tensor(args[1]), *rows = nullptr, *bias = nullptr;
    if (!x || !w || x->scalar_type() != at::kBFloat16 || w->scalar_type() != at::kBFloat16 || x->dim() != 2 ||
        w->dim() != 3 || !x->is_contiguous() || !w->is_contiguous() || w->size(2) != x->size(1))
        return none();
    const int64_t G = w->size(0), W = w->size(1), K = x->size(1), N = swiglu ? W / 2 : W;
    if (G > INT32_MAX || W > INT32_MAX || K > INT32_MAX || (swiglu && W % 2)) return none();
    const Tensor *offsets = dense(args[2], at::kInt, G + 1);
    if (!offsets || (args[3] != Py_None && !(bias = dense(args[3], at::kBFloat16, G, W)))) return none();
    if (args[4] != Py_None) {
        rows = cuda_tensor(args[4]);
        if (!rows || rows->scalar_type() != at::kInt || rows->dim() != 1 || !rows->is_contiguous()) return none();
    }
    const int64_t P = rows ? rows->size(0) : x->size(0);
    Tensor out;
    int st;
    {
        const Unlocked unlocked;
        out = make(*x, at::kBFloat16, {P, N});
        Tensor space;  // freed on return, to this stream's own memory
        const size_t need = g_grouped_workspace(P, (int)G, (int)N, (int)K, swiglu);
        if (need) space = make(*x, at::kByte, {(int64_t)need});
        st = g_grouped(x->const_data_ptr(), x->size(0), w->const_data_ptr(), bias ? bias->const_data_ptr() : nullptr,
                       static_cast<const int32_t *>(offsets->const_data_ptr()),
                       rows ? static_cast<const int32_t *>(rows->const_data_ptr()) : nullptr, out.data_ptr(), P, (int)G,
                       (int)N, (int)K, swiglu, need ? space.data_ptr() : nullptr, need, flags, stream_of(*x));
    }
    return st ? PyLong_FromLong(st) : item(out);
    END_HANDLE_TH_ERRORS
}

// combine_rows(y, place, weights, addend, flags)
PyObject *combine_rows(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (wrong_count(n, 5)) return nullptr;
    bool wide = false;
    const uint32_t flags = as_flags(args[4], wide);
    if (PyErr_Occurred()) return nullptr;
    if (wide) return none();
    const Tensor *y = cuda_tensor(args[0]), *place = cuda_tensor(args[1]), *weights = nullptr, *addend = nullptr;
    if (!y || !place || y->scalar_type() != at::kBFloat16 || y->dim() != 2 || !y->is_contiguous() ||
        place->scalar_type() != at::kInt || place->dim() != 2 || !place->is_contiguous())
        return none();
    const int64_t T = place->size(0), k = place->size(1), H = y->size(1);
    if (k > INT32_MAX || H > INT32_MAX) return none();
    if (args[2] != Py_None && !(weights = dense(args[2], at::kFloat, T, k))) return none();
    if (args[3] != Py_None && !(addend = dense(args[3], at::kBFloat16, T, H))) return none();
    Tensor out;
    int st;
    {
        const Unlocked unlocked;
        out = make(*y, at::kBFloat16, {T, H});
        st = g_combine(y->const_data_ptr(), y->size(0), static_cast<const int32_t *>(place->const_data_ptr()),
                       weights ? static_cast<const float *>(weights->const_data_ptr()) : nullptr,
                       addend ? addend->const_data_ptr() : nullptr, out.data_ptr(), T, (int)k, (int)H, flags,
                       stream_of(*y));
    }
    return st ? PyLong_FromLong(st) : item(out);
    END_HANDLE_TH_ERRORS
}

// linear_lora(x, w, a, b, ids, bias, scale, flags)
PyObject *linear_lora(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (wrong_count(n, 8)) return nullptr;
    bool wide = false;
    const uint32_t flags = as_flags(args[7], wide);
    if (PyErr_Occurred()) return nullptr;
    if (wide) return none();
    const Tensor *x = cuda_tensor(args[0]), *w = cuda_tensor(args[1]), *a = cuda_tensor(args[2]), *bias = nullptr,
                 *scale = nullptr;
    if (!x || !w || !a || x->dim() != 2 || w->dim() != 2 || a->dim() != 3) return none();
    const int64_t M = x->size(0), K = x->size(1), N = w->size(0), L = a->size(0), R = a->size(1);
    const Tensor *b = dense(args[3], at::kBFloat16, L, N, R), *ids = dense(args[4], at::kInt, M);
    if (!dense(args[0], at::kBFloat16, M, K) || !dense(args[1], at::kBFloat16, N, K) ||
        !dense(args[2], at::kBFloat16, L, R, K) || !b || !ids || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX ||
        L > INT32_MAX || R > INT32_MAX)
        return none();
    if (args[5] != Py_None && !(bias = dense(args[5], at::kBFloat16, N))) return none();
    if (args[6] != Py_None && !(scale = dense(args[6], at::kFloat, L))) return none();
    Tensor out;
    int st;
    {
        const Unlocked unlocked;
        out = make(*x, at::kBFloat16, {M, N});
        Tensor space;  // freed on return, to this stream's own memory
        const size_t need = g_lora_workspace((int)M, (int)N, (int)K, (int)R, (int)L);
        if (need) space = make(*x, at::kByte, {(int64_t)need});
        st = g_lora(x->const_data_ptr(), w->const_data_ptr(), bias ? bias->const_data_ptr() : nullptr, a->const_data_ptr(),
                    b->const_data_ptr(), scale ? static_cast<const float *>(scale->const_data_ptr()) : nullptr,
                    static_cast<const int32_t *>(ids->const_data_ptr()), out.data_ptr(), (int)M, (int)N, (int)K, (int)R,
                    (int)L, need ? space.data_ptr() : nullptr, need, flags, stream_of(*x));
    }
    return st ? PyLong_FromLong(st) : item(out);
    END_HANDLE_TH_ERRORS
}

// bind(addresses of the entry points, in the order of the declarations above)
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (wrong_count(n, 13)) return nullptr;
    void *p[13];
    for (int i = 0; i < 13; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_rmsnorm = reinterpret_cast<decltype(g_rmsnorm)>(p[0]);
    g_route = reinterpret_cast<decltype(g_route)>(p[1]);
    g_quant = reinterpret_cast<decltype(g_quant)>(p[2]);
    g_dequant = reinterpret_cast<decltype(g_dequant)>(p[3]);
    g_linear = reinterpret_cast<decltype(g_linear)>(p[4]);
    g_dynamic = reinterpret_cast<decltype(g_dynamic)>(p[5]);
    g_workspace = reinterpret_cast<decltype(g_workspace)>(p[6]);
    g_group = reinterpret_cast<decltype(g_group)>(p[7]);
    g_grouped = reinterpret_cast<decltype(g_grouped)>(p[8]);
    g_combine = reinterpret_cast<decltype(g_combine)>(p[9]);
    g_lora = reinterpret_cast<decltype(g_lora)>(p[10]);
    g_lora_workspace = reinterpret_cast<decltype(g_lora_workspace)>(p[11]);
    g_grouped_workspace = reinterpret_cast<decltype(g_grouped_workspace)>(p[12]);
    Py_RETURN_NONE;
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {CALL(rmsnorm),       CALL(route),        CALL(quant_mxfp4),
                           CALL(dequant_mxfp4), CALL(linear_mxfp4), CALL(group_rows),
                           CALL(linear_grouped), CALL(combine_rows), CALL(linear_lora), CALL(bind),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls(void) { return PyModule_Create(&g_module); }
