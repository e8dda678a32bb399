// binding.cpp -- the hot path of the decoder operators' Python binding.
//
// A decode step's kernels run for a few microseconds, less than the interpreter needs
// to look at the dozen tensors of a call.  This module does what decoder.py's checks do
// (types, shapes, strides, devices), allocates what the caller left out, and makes the
// C call on the current stream.  It holds no state but the addresses of the library's
// functions, and computes nothing.  A call that it does not accept returns None, having
// done nothing: decoder.py then finds the reason and raises it.  A status other than 0 is
// returned as an integer.
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>

#include "lowbit.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct {
    decltype(&lowbit_kv_append_ex) kv_append;
    decltype(&lowbit_kv_append4) kv_append4;
    decltype(&lowbit_attention) attention;
    decltype(&lowbit_attention4) attention4;
    decltype(&lowbit_attention_workspace) workspace;
    decltype(&lowbit_attention4_workspace) workspace4;
    decltype(&lowbit_cache_values) values;
    decltype(&lowbit_cache4_values) values4;
    decltype(&lowbit_sample) sample;
} fn;

// The tensor behind an argument, or null.
const Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool is(const Tensor *t, ScalarType type, int dev, int64_t dims) {
    return t != nullptr && t->is_cuda() && t->get_device() == dev && t->scalar_type() == type && t->dim() == dims;
}

// A contiguous tensor of n values; its address in *at.
template <typename T>
bool vector(PyObject *o, ScalarType type, int dev, int64_t n, T *at) {
    const Tensor *t = tensor(o);
    if (!is(t, type, dev, 1) || t->size(0) != n || (n > 1 && t->stride(0) != 1)) return false;
    *at = static_cast<T>(t->data_ptr());
    return true;
}

// bf16 [T, H, D] with contiguous values of a head.
struct Rows { uint16_t *at; int64_t token, head; };
bool rows(const Tensor *t, int dev, int64_t T, int64_t H, int64_t D, Rows *r) {
    if (!is(t, ScalarType::BFloat16, dev, 3) || t->size(0) != T || t->size(1) != H || t->size(2) != D || t->stride(2) != 1) return false;
    *r = {static_cast<uint16_t *>(t->data_ptr()), t->stride(0), t->stride(1)};
    return true;
}

// Whether torch has something to say about new tensors beside `like`: a mode or a subclass that sees what is
// called, or deterministic algorithms, which fill them.
bool watched(const Tensor &like) {
    return at::globalContext().deterministicAlgorithms() || c10::impl::TorchDispatchModeTLS::any_modes_set() ||
           like.key_set().has(c10::DispatchKey::Python);
}
// A new contiguous tensor beside `like`.  (Through the dispatcher it costs a microsecond more.)
Tensor fresh(at::IntArrayRef sizes, ScalarType type, const Tensor &like) {
    if (watched(like)) return at::empty(sizes, at::TensorOptions().dtype(type).device(like.device()));
    return Tensor(at::detail::empty_cuda(sizes, type, like.device(), std::nullopt));
}
// at::empty_like of rows [T, H, D].
Tensor fresh_rows(const Tensor &q) {
    if (!watched(q) && q.stride(2) == 1 && q.stride(1) >= q.size(2) && q.stride(0) >= q.stride(1))
        return fresh(q.sizes(), ScalarType::BFloat16, q);
    return at::empty_like(q);
}

bool small(int64_t n) { return n >= 0 && n <= INT32_MAX; }

// A cache of either kind.
struct Cache {
    bool four;
    lowbit_cache c8;
    lowbit_cache4 c4;
    int32_t kv_heads() const { return four ? c4.kv_heads : c8.kv_heads; }
};

// Two tensors [pages, heads, page, n] of the same strides, each head's page contiguous.
bool pages_of(const Tensor *k, const Tensor *v, int dev, ScalarType type, int64_t n) {
    for (const Tensor *t : {k, v})
        if (t == nullptr || !t->is_cuda() || t->get_device() != dev || t->dim() != 4 ||
            (t->scalar_type() != type && t->scalar_type() != ScalarType::Byte))
            return false;
    if (k->sizes() != v->sizes() || k->strides() != v->strides() || k->size(3) != n) return false;
    if (k->numel() > 0 && (k->stride(2) != n || k->stride(3) != 1)) return false;
    return small(k->size(0)) && small(k->size(1)) && small(k->size(2));
}

template <typename T>
T *at(const Tensor *t) { return static_cast<T *>(t->data_ptr()); }

bool cache_of(PyObject *const *a, int dev, int64_t dim, Cache *c) {
    const Tensor *k = tensor(a[0]), *v = tensor(a[1]), *e[2] = {tensor(a[2]), tensor(a[3])};
    *c = {};
    c->four = e[0] != nullptr && e[0]->dim() == 4;
    if (c->four) {                               // the 4-bit kind: a scale for each 32 values
        if (dim % 32 != 0 || !pages_of(k, v, dev, ScalarType::Byte, dim / 2) || !pages_of(e[0], e[1], dev, ScalarType::Float8_e5m2, dim / 32))
            return false;
        if (k->size(0) != e[0]->size(0) || k->size(1) != e[0]->size(1) || k->size(2) != e[0]->size(2)) return false;
        c->c4.k = at<uint8_t>(k), c->c4.v = at<uint8_t>(v), c->c4.k_scale = at<uint8_t>(e[0]), c->c4.v_scale = at<uint8_t>(e[1]);
        c->c4.page_stride = k->stride(0), c->c4.head_stride = k->stride(1);
        c->c4.scale_page_stride = e[0]->stride(0), c->c4.scale_head_stride = e[0]->stride(1);
        c->c4.pages = (int32_t)k->size(0), c->c4.kv_heads = (int32_t)k->size(1), c->c4.page = (int32_t)k->size(2);
        c->c4.head_dim = (int32_t)dim;
        return true;
    }
    if (!pages_of(k, v, dev, ScalarType::Float8_e4m3fn, dim)) return false;
    for (const Tensor *t : e)
        if (!is(t, ScalarType::Char, dev, 2) || t->size(0) != k->size(0) || t->size(1) != k->size(1) || !t->is_contiguous()) return false;
    c->c8.k = at<uint8_t>(k), c->c8.v = at<uint8_t>(v), c->c8.k_exp = at<int8_t>(e[0]), c->c8.v_exp = at<int8_t>(e[1]);
    c->c8.page_stride = k->stride(0), c->c8.head_stride = k->stride(1);
    c->c8.pages = (int32_t)k->size(0), c->c8.kv_heads = (int32_t)k->size(1), c->c8.page = (int32_t)k->size(2), c->c8.head_dim = (int32_t)dim;
    return true;
}

// a: page_table, lens, cu_q, max_q.
bool sequences_of(PyObject *const *a, int dev, int64_t tokens, lowbit_sequences *s) {
    const Tensor *table = tensor(a[0]);
    if (!is(table, ScalarType::Int, dev, 2)) return false;
    const int64_t batch = table->size(0), width = table->size(1);
    if ((table->stride(1) != 1 && width > 1) || (table->stride(0) < width && batch > 1) || !small(batch) || !small(width) || !small(tokens))
        return false;
    *s = {};
    if (!vector(a[1], ScalarType::Int, dev, batch, &s->lens)) return false;
    if (a[2] == Py_None) {
        if (batch > 0 && tokens % batch != 0) return false;
        s->max_q = batch > 0 ? (int32_t)(tokens / batch) : 0;
    } else {
        if (!vector(a[2], ScalarType::Int, dev, batch + 1, &s->cu_q)) return false;
        if (a[3] == Py_None) {
            s->max_q = (int32_t)tokens;
        } else {
            const long n = PyLong_AsLong(a[3]);
            if (PyErr_Occurred() || n < INT32_MIN || n > INT32_MAX) return PyErr_Clear(), false;
            s->max_q = (int32_t)n;
        }
    }
    s->page_table = static_cast<int32_t *>(table->data_ptr());
    s->table_stride = std::max(table->stride(0), width);
    s->width = (int32_t)width, s->batch = (int32_t)batch, s->tokens = (int32_t)tokens;
    return true;
}

// A float argument: a number that is not a tensor.
bool number(PyObject *o, float *x) {
    const double d = PyFloat_AsDouble(o);
    if (d == -1.0 && PyErr_Occurred()) return PyErr_Clear(), false;
    *x = (float)d;
    return true;
}
bool integer(PyObject *o, int32_t *x) {
    const long n = PyLong_AsLong(o);
    if (n == -1 && PyErr_Occurred()) return PyErr_Clear(), false;
    if (n < INT32_MIN || n > INT32_MAX) return false;
    *x = (int32_t)n;
    return true;
}

PyObject *refuse() { Py_RETURN_NONE; }
PyObject *result(lowbit_status st, const Tensor &out) { return st != LOWBIT_OK ? PyLong_FromLong(st) : THPVariable_Wrap(out); }
lowbit_stream_t stream(int dev) { return reinterpret_cast<lowbit_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream()); }

// What stands before the write; a: q_norm, k_norm, eps, positions, axes.
bool prologue_of(PyObject *const *a, int dev, int64_t T, int64_t D, int64_t pairs, lowbit_kv_prologue *b) {
    *b = {};
    const Tensor *first = nullptr;
    const void **norms[2] = {&b->q_norm, &b->k_norm};
    for (int i = 0; i < 2; ++i) {
        if (a[i] == Py_None) continue;
        const Tensor *w = tensor(a[i]);
        if (w == nullptr || (first != nullptr && w->scalar_type() != first->scalar_type()) || !vector(a[i], w->scalar_type(), dev, D, norms[i]))
            return false;
        switch (w->scalar_type()) {
            case ScalarType::Float: b->norm_dtype = LOWBIT_DTYPE_F32; break;
            case ScalarType::BFloat16: b->norm_dtype = LOWBIT_DTYPE_BF16; break;
            case ScalarType::Half: b->norm_dtype = LOWBIT_DTYPE_F16; break;
            default: return false;
        }
        first = w;
    }
    if (!number(a[2], &b->eps)) return false;
    if (a[3] == Py_None) return a[4] == Py_None;
    const Tensor *p = tensor(a[3]);
    if (p == nullptr || p->dim() < 1 || !is(p, ScalarType::Int, dev, p->dim() == 1 ? 1 : 2) || p->size(0) != T) return false;
    const int64_t axes = p->dim() == 1 ? 1 : p->size(1);
    if (axes < 1 || axes > 255 || (axes > 1 && (p->stride(1) != 1 || a[4] == Py_None))) return false;
    if (a[4] != Py_None && !vector(a[4], ScalarType::Byte, dev, pairs, &b->axis)) return false;
    b->positions = at<int32_t>(p), b->positions_token = p->stride(0), b->axes = (int32_t)axes;
    // An empty tensor has no address: nothing of it is read, but positions they are.
    return b->positions != nullptr || T == 0;
}

// q, k, v, k_cache, v_cache, k_exp, v_exp, page_table, lens, cu_q, max_q, turns, interleaved, factor, out[, q_norm, k_norm,
// eps, positions, axes]
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 15 && n != 20) return refuse();
    const Tensor *q = tensor(a[0]);
    if (q == nullptr || !q->is_cuda() || q->dim() != 3) return refuse();
    const int dev = q->get_device();
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2);
    Rows rq, rk, rv, ro;
    Cache c;
    lowbit_sequences s;
    lowbit_kv_prologue before = {};
    lowbit_kv_append_args args = {};
    if (!small(H) || !small(D) || !rows(q, dev, T, H, D, &rq) || !cache_of(a + 3, dev, D, &c) || !rows(tensor(a[1]), dev, T, c.kv_heads(), D, &rk) ||
        !rows(tensor(a[2]), dev, T, c.kv_heads(), D, &rv) || !sequences_of(a + 7, dev, T, &s) || !number(a[13], &args.factor))
        return refuse();
    if (a[11] != Py_None) {
        const Tensor *t = tensor(a[11]);
        if (t == nullptr || t->dim() != 1 || t->size(0) > 4096 || !vector(a[11], ScalarType::Long, dev, t->size(0), &args.turns)) return refuse();
        args.rotary_dim = 2 * (int32_t)t->size(0);
    }
    if (n == 20 && !prologue_of(a + 15, dev, T, D, args.rotary_dim / 2, &before)) return refuse();
    const int interleaved = PyObject_IsTrue(a[12]);
    if (interleaved < 0) return PyErr_Clear(), refuse();
    const c10::cuda::OptionalCUDAGuard guard(q->device());
    const Tensor out = a[14] == Py_None ? fresh_rows(*q) : (tensor(a[14]) != nullptr ? *tensor(a[14]) : Tensor());
    if (!out.defined() || !rows(&out, dev, T, H, D, &ro)) return refuse();
    args.q = rq.at, args.k = rk.at, args.v = rv.at, args.q_out = ro.at;
    args.q_token = rq.token, args.q_head = rq.head, args.k_token = rk.token, args.k_head = rk.head;
    args.v_token = rv.token, args.v_head = rv.head, args.o_token = ro.token, args.o_head = ro.head;
    args.heads = (int32_t)H, args.interleaved = interleaved;
    return result(c.four ? fn.kv_append4(&args, &before, &c.c4, &s, stream(dev)) : fn.kv_append(&args, &before, &c.c8, &s, stream(dev)), out);
}

// q, k_cache, v_cache, k_exp, v_exp, page_table, lens, cu_q, max_q, scale, window, out, lse, workspace
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 14) return refuse();
    const Tensor *q = tensor(a[0]);
    if (q == nullptr || !q->is_cuda() || q->dim() != 3) return refuse();
    const int dev = q->get_device();
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2);
    Rows rq, ro;
    Cache c;
    lowbit_sequences s;
    lowbit_attention_args args = {};
    if (!small(H) || !small(D) || !rows(q, dev, T, H, D, &rq) || !cache_of(a + 1, dev, D, &c) || !sequences_of(a + 5, dev, T, &s) ||
        !integer(a[10], &args.window))
        return refuse();
    args.scale = 1.f / std::sqrt((float)D);
    if (a[9] != Py_None && !number(a[9], &args.scale)) return refuse();
    if (a[12] != Py_None) {
        const Tensor *lse = tensor(a[12]);
        if (!is(lse, ScalarType::Float, dev, 2) || lse->size(0) != T || lse->size(1) != H || (H > 1 && lse->stride(1) != 1)) return refuse();
        args.lse = static_cast<float *>(lse->data_ptr()), args.lse_token = lse->stride(0);
    }
    const c10::cuda::OptionalCUDAGuard guard(q->device());
    const Tensor out = a[11] == Py_None ? fresh_rows(*q) : (tensor(a[11]) != nullptr ? *tensor(a[11]) : Tensor());
    if (!out.defined() || !rows(&out, dev, T, H, D, &ro)) return refuse();
    c10::DataPtr own;                            // like a tensor of the current stream that goes after the launch
    Tensor seen;                                 // or one
    if (a[13] == Py_None) {
        const size_t bytes = c.four ? fn.workspace4((int32_t)H, &c.c4, &s) : fn.workspace((int32_t)H, &c.c8, &s);
        if (watched(*q)) seen = fresh({(int64_t)bytes}, ScalarType::Byte, *q);
        else own = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
        args.workspace = seen.defined() ? seen.data_ptr() : own.get(), args.workspace_bytes = bytes;
    } else {
        const Tensor *w = tensor(a[13]);
        if (!is(w, ScalarType::Byte, dev, 1) || !w->is_contiguous()) return refuse();
        args.workspace = w->data_ptr(), args.workspace_bytes = (size_t)w->numel();
    }
    args.q = rq.at, args.out = ro.at;
    args.q_token = rq.token, args.q_head = rq.head, args.o_token = ro.token, args.o_head = ro.head;
    args.heads = (int32_t)H;
    return result(c.four ? fn.attention4(&args, &c.c4, &s, stream(dev)) : fn.attention(&args, &c.c8, &s, stream(dev)), out);
}

// k_cache, v_cache, k_exp, v_exp, k_out, v_out
PyObject *cache_values(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 6) return refuse();
    const Tensor *k = tensor(a[0]), *e = tensor(a[2]);
    if (k == nullptr || !k->is_cuda() || k->dim() != 4 || e == nullptr || !small(k->size(3))) return refuse();
    const int dev = k->get_device();
    const int64_t D = k->size(3) * (e->dim() == 4 ? 2 : 1);
    Cache c;
    if (!cache_of(a, dev, D, &c)) return refuse();
    const c10::cuda::OptionalCUDAGuard guard(k->device());
    Tensor out[2];
    for (int i = 0; i < 2; ++i) {
        if (a[4 + i] == Py_None) {
            out[i] = fresh({k->size(0), k->size(1), k->size(2), D}, ScalarType::BFloat16, *k);
            continue;
        }
        const Tensor *t = tensor(a[4 + i]);
        if (!is(t, ScalarType::BFloat16, dev, 4) || t->size(0) != k->size(0) || t->size(1) != k->size(1) || t->size(2) != k->size(2) ||
            t->size(3) != D || !t->is_contiguous())
            return refuse();
        out[i] = *t;
    }
    uint16_t *ko = at<uint16_t>(&out[0]), *vo = at<uint16_t>(&out[1]);
    const lowbit_status st = c.four ? fn.values4(&c.c4, ko, vo, stream(dev)) : fn.values(&c.c8, ko, vo, stream(dev));
    if (st != LOWBIT_OK) return PyLong_FromLong(st);
    PyObject *pair = PyTuple_New(2);
    for (int i = 0; i < 2 && pair != nullptr; ++i) {
        PyObject *o = THPVariable_Wrap(out[i]);
        if (o == nullptr) Py_CLEAR(pair);
        else PyTuple_SET_ITEM(pair, i, o);
    }
    return pair;
}

// logits, u, temperature, top_k, top_p, min_p, out, logprob
PyObject *sample(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 8) return refuse();
    const Tensor *x = tensor(a[0]);
    if (x == nullptr || !x->is_cuda() || x->dim() != 2) return refuse();
    const int dev = x->get_device();
    const int64_t B = x->size(0), V = x->size(1);
    lowbit_sample_args args = {};
    switch (x->scalar_type()) {
        case ScalarType::Float: args.dtype = LOWBIT_DTYPE_F32; break;
        case ScalarType::BFloat16: args.dtype = LOWBIT_DTYPE_BF16; break;
        case ScalarType::Half: args.dtype = LOWBIT_DTYPE_F16; break;
        default: return refuse();
    }
    if ((x->stride(1) != 1 && V > 1) || !small(B) || !small(V) || !vector(a[1], ScalarType::Float, dev, B, &args.u)) return refuse();
    // A setting: one number for all rows, or one a row.
    auto setting = [&](PyObject *o, const float **each, float *all, float unset) {
        if (!THPVariable_Check(o)) return number(o, all);
        *all = unset;
        return vector(o, ScalarType::Float, dev, B, each);
    };
    if (!setting(a[2], &args.temperature, &args.temperature_all, 1.f) || !setting(a[4], &args.top_p, &args.top_p_all, 1.f) ||
        !setting(a[5], &args.min_p, &args.min_p_all, 0.f))
        return refuse();
    if (THPVariable_Check(a[3]) ? !vector(a[3], ScalarType::Int, dev, B, &args.top_k) : !integer(a[3], &args.top_k_all)) return refuse();
    if (a[7] != Py_None && !vector(a[7], ScalarType::Float, dev, B, &args.logprob)) return refuse();
    const c10::cuda::OptionalCUDAGuard guard(x->device());
    const Tensor out = a[6] == Py_None ? fresh({B}, ScalarType::Long, *x) : (tensor(a[6]) != nullptr ? *tensor(a[6]) : Tensor());
    if (!out.defined() || !is(&out, ScalarType::Long, dev, 1) || out.size(0) != B || (B > 1 && out.stride(0) != 1)) return refuse();
    args.token = static_cast<int64_t *>(out.data_ptr());
    args.logits = x->data_ptr(), args.row_stride = x->stride(0), args.rows = (int32_t)B, args.vocab = (int32_t)V;
    return result(fn.sample(&args, stream(dev)), out);
}

// The addresses of the library's functions, in the order of `fn`.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    constexpr int kFunctions = 9;
    void *p[kFunctions];
    if (n != kFunctions) return PyErr_SetString(PyExc_TypeError, "bind takes nine addresses"), nullptr;
    for (int i = 0; i < kFunctions; ++i)
        if ((p[i] = PyLong_AsVoidPtr(a[i])) == nullptr) return PyErr_Occurred() ? nullptr : (PyErr_SetString(PyExc_ValueError, "null address"), nullptr);
    int i = 0;
    auto next = [&](auto &f) { f = reinterpret_cast<std::decay_t<decltype(f)>>(p[i++]); };
    next(fn.kv_append), next(fn.kv_append4), next(fn.attention), next(fn.attention4), next(fn.workspace), next(fn.workspace4);
    next(fn.values), next(fn.values4), next(fn.sample);
    Py_RETURN_NONE;
}

// C++ exceptions (an allocation that fails) become Python's.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    return F(self, a, n);
    END_HANDLE_TH_ERRORS
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(kv_append), METHOD(attention), METHOD(cache_values), METHOD(sample), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lowbit_torch", "Hot path of the decoder operators' binding.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lowbit_torch() { return PyModule_Create(&module); }
