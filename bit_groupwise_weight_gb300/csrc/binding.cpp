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

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
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
    decltype(&lowbit_kv_append) kv_append;
    decltype(&lowbit_attention) attention;
    decltype(&lowbit_attention_workspace) workspace;
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

bool small(int64_t n) { return n >= 0 && n <= INT32_MAX; }

bool cache_of(PyObject *const *a, int dev, int64_t dim, lowbit_cache *c) {
    const Tensor *k = tensor(a[0]), *v = tensor(a[1]), *e[2] = {tensor(a[2]), tensor(a[3])};
    for (const Tensor *t : {k, v})
        if (t == nullptr || !t->is_cuda() || t->get_device() != dev || t->dim() != 4 ||
            (t->scalar_type() != ScalarType::Float8_e4m3fn && t->scalar_type() != ScalarType::Byte))
            return false;
    if (k->sizes() != v->sizes() || k->strides() != v->strides() || k->size(3) != dim) return false;
    if (k->numel() > 0 && (k->stride(2) != dim || k->stride(3) != 1)) return false;
    if (!small(k->size(0)) || !small(k->size(1)) || !small(k->size(2))) return false;
    for (const Tensor *t : e)
        if (!is(t, ScalarType::Char, dev, 2) || t->size(0) != k->size(0) || t->size(1) != k->size(1) || !t->is_contiguous()) return false;
    *c = {};
    c->k = static_cast<uint8_t *>(k->data_ptr()), c->v = static_cast<uint8_t *>(v->data_ptr());
    c->k_exp = static_cast<int8_t *>(e[0]->data_ptr()), c->v_exp = static_cast<int8_t *>(e[1]->data_ptr());
    c->page_stride = k->stride(0), c->head_stride = k->stride(1);
    c->pages = (int32_t)k->size(0), c->kv_heads = (int32_t)k->size(1), c->page = (int32_t)k->size(2), c->head_dim = (int32_t)dim;
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

// q, k, v, k_cache, v_cache, k_exp, v_exp, page_table, lens, cu_q, max_q, turns, interleaved, factor, out
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 15) return refuse();
    const Tensor *q = tensor(a[0]);
    if (q == nullptr || !q->is_cuda() || q->dim() != 3) return refuse();
    const int dev = q->get_device();
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2);
    Rows rq, rk, rv, ro;
    lowbit_cache c;
    lowbit_sequences s;
    lowbit_kv_append_args args = {};
    if (!small(H) || !small(D) || !rows(q, dev, T, H, D, &rq) || !cache_of(a + 3, dev, D, &c) || !rows(tensor(a[1]), dev, T, c.kv_heads, D, &rk) ||
        !rows(tensor(a[2]), dev, T, c.kv_heads, D, &rv) || !sequences_of(a + 7, dev, T, &s) || !number(a[13], &args.factor))
        return refuse();
    if (a[11] != Py_None) {
        const Tensor *t = tensor(a[11]);
        if (t == nullptr || t->dim() != 1 || t->size(0) > 4096 || !vector(a[11], ScalarType::Long, dev, t->size(0), &args.turns)) return refuse();
        args.rotary_dim = 2 * (int32_t)t->size(0);
    }
    const int interleaved = PyObject_IsTrue(a[12]);
    if (interleaved < 0) return PyErr_Clear(), refuse();
    const c10::cuda::OptionalCUDAGuard guard(q->device());
    const Tensor out = a[14] == Py_None ? at::empty_like(*q) : (tensor(a[14]) != nullptr ? *tensor(a[14]) : Tensor());
    if (!out.defined() || !rows(&out, dev, T, H, D, &ro)) return refuse();
    args.q = rq.at, args.k = rk.at, args.v = rv.at, args.q_out = ro.at;
    args.q_token = rq.token, args.q_head = rq.head, args.k_token = rk.token, args.k_head = rk.head;
    args.v_token = rv.token, args.v_head = rv.head, args.o_token = ro.token, args.o_head = ro.head;
    args.heads = (int32_t)H, args.interleaved = interleaved;
    return result(fn.kv_append(&args, &c, &s, stream(dev)), out);
}

// q, k_cache, v_cache, k_exp, v_exp, page_table, lens, cu_q, max_q, scale, window, out, lse, workspace
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 14) return refuse();
    const Tensor *q = tensor(a[0]);
    if (q == nullptr || !q->is_cuda() || q->dim() != 3) return refuse();
    const int dev = q->get_device();
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2);
    Rows rq, ro;
    lowbit_cache c;
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
    const Tensor out = a[11] == Py_None ? at::empty_like(*q) : (tensor(a[11]) != nullptr ? *tensor(a[11]) : Tensor());
    if (!out.defined() || !rows(&out, dev, T, H, D, &ro)) return refuse();
    Tensor own;
    if (a[13] == Py_None) {
        own = at::empty({(int64_t)fn.workspace((int32_t)H, &c, &s)}, q->options().dtype(at::kByte));
        args.workspace = own.data_ptr(), args.workspace_bytes = (size_t)own.numel();
    } else {
        const Tensor *w = tensor(a[13]);
        if (!is(w, ScalarType::Byte, dev, 1) || !w->is_contiguous()) return refuse();
        args.workspace = w->data_ptr(), args.workspace_bytes = (size_t)w->numel();
    }
    args.q = rq.at, args.out = ro.at;
    args.q_token = rq.token, args.q_head = rq.head, args.o_token = ro.token, args.o_head = ro.head;
    args.heads = (int32_t)H;
    return result(fn.attention(&args, &c, &s, stream(dev)), out);
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
    const Tensor out = a[6] == Py_None ? at::empty({B}, x->options().dtype(at::kLong)) : (tensor(a[6]) != nullptr ? *tensor(a[6]) : Tensor());
    if (!out.defined() || !is(&out, ScalarType::Long, dev, 1) || out.size(0) != B || (B > 1 && out.stride(0) != 1)) return refuse();
    args.token = static_cast<int64_t *>(out.data_ptr());
    args.logits = x->data_ptr(), args.row_stride = x->stride(0), args.rows = (int32_t)B, args.vocab = (int32_t)V;
    return result(fn.sample(&args, stream(dev)), out);
}

// The addresses of lowbit_kv_append, _attention, _attention_workspace and _sample.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *p[4];
    if (n != 4) return PyErr_SetString(PyExc_TypeError, "bind takes four addresses"), nullptr;
    for (int i = 0; i < 4; ++i)
        if ((p[i] = PyLong_AsVoidPtr(a[i])) == nullptr) return PyErr_Occurred() ? nullptr : (PyErr_SetString(PyExc_ValueError, "null address"), nullptr);
    fn = {reinterpret_cast<decltype(fn.kv_append)>(p[0]), reinterpret_cast<decltype(fn.attention)>(p[1]),
          reinterpret_cast<decltype(fn.workspace)>(p[2]), reinterpret_cast<decltype(fn.sample)>(p[3])};
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
PyMethodDef methods[] = {METHOD(bind), METHOD(kv_append), METHOD(attention), METHOD(sample), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lowbit_torch", "Hot path of the decoder operators' binding.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lowbit_torch() { return PyModule_Create(&module); }
