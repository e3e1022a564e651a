// Python entry to the 4-bit and the training operators for the calls that are all in order:
// plain torch tensors on the current device, outputs to be allocated.  It
// checks, allocates, fetches the current stream and calls the C ABI in one
// step, which takes the host 6 us where the same through ctypes takes 10
// (one token quantized); the kernels of short calls run 2 to 3.  Anything else
// returns None, and the Python code takes the call: it names what is wrong, or
// handles what is rare.  A C ABI status other than 0 is returned as an int.
#include <Python.h>

#include <ATen/ops/empty_strided.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>

#include "fp8mi.h"

namespace {

const at::Tensor* plain(PyObject* o)
{
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.layout() == at::kStrided ? &t : nullptr;
}
// On the GPU that kernels are launched on.
bool here(const at::Tensor& t) { return t.is_cuda() && t.get_device() == c10::hip::current_device(); }

// A matrix whose rows lie `ld` apart (a single row's stride may be anything).
bool matrix(const at::Tensor& t, int64_t& ld)
{
    if (t.dim() != 2 || t.numel() == 0 || (t.size(1) > 1 && t.stride(1) != 1)) return false;
    ld = t.size(0) > 1 ? t.stride(0) : std::max(t.stride(0), t.size(1));
    return true;
}

at::Tensor fresh(at::IntArrayRef size, at::IntArrayRef stride, at::ScalarType dtype, const at::Tensor& like)
{
    return at::empty_strided(size, stride, at::TensorOptions().dtype(dtype).device(like.device()));
}

template <typename T>
T* data(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }

// Other threads may run Python while this one allocates and enqueues: a launch
// waits where a queue is full.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    Unlocked() = default;
    Unlocked(const Unlocked&) = delete;
    ~Unlocked() { PyEval_RestoreThread(state); }
};

hipStream_t stream() { return c10::hip::getCurrentHIPStream().stream(); }

// Arguments are of the Python code's making; a failed conversion raises.
bool ints(PyObject* const* args, int n, int64_t* out)
{
    for (int i = 0; i < n; ++i) {
        out[i] = PyLong_AsLongLong(args[i]);
        if (out[i] == -1 && PyErr_Occurred()) return false;
    }
    return true;
}

struct Codes {
    at::Tensor q, s;
    int64_t ldq = 0, ps = 0;
};
Codes fresh_codes(int64_t rows, int64_t cols, const at::Tensor& like)
{
    Codes c;
    c.ldq = 128 * ((cols + 255) / 256);
    c.ps = 16 * rows;
    c.q = fresh({rows, c.ldq}, {c.ldq, 1}, at::kByte, like);
    c.s = fresh({(cols + 511) / 512, rows, 16}, {c.ps, 16, 1}, at::kByte, like);
    return c;
}

// (q, s, cols): the distances of rows and panels, if q and s hold [.., rows, cols].
PyObject* mx4_held(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const at::Tensor* q = n == 3 ? plain(args[0]) : nullptr;
    const at::Tensor* s = q ? plain(args[1]) : nullptr;
    if (!s || !PyLong_CheckExact(args[2])) Py_RETURN_NONE;
    int64_t cols;
    if (!ints(args + 2, 1, &cols)) return nullptr;
    const int64_t d = q->dim();
    if ((d != 2 && d != 3) || s->dim() != d + 1 || q->scalar_type() != at::kByte || s->scalar_type() != at::kByte ||
        cols < 1 || cols >= (int64_t)1 << 31 || q->numel() == 0)
        Py_RETURN_NONE;
    const int64_t rows = q->size(d - 2), panels = (cols + 511) / 512;
    if (q->size(d - 1) != 128 * ((cols + 255) / 256) || (d == 3 && q->size(0) != s->size(0)) ||
        s->size(d - 2) != panels || s->size(d - 1) != rows || s->size(d) != 16 || q->stride(d - 1) != 1 ||
        s->stride(d) != 1 || (rows > 1 && s->stride(d - 1) != 16))
        Py_RETURN_NONE;
    return Py_BuildValue("LL", (long long)(rows > 1 ? q->stride(d - 2) : q->size(d - 1)),
                         (long long)(panels > 1 ? s->stride(d - 2) : 16 * rows));
    END_HANDLE_TH_ERRORS
}

// (x, want_t, seed): (q, s) or (q, s, q_t, s_t).
PyObject* mx4_quantize(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const at::Tensor* x = n == 3 ? plain(args[0]) : nullptr;
    const at::Tensor* seed = nullptr;
    int64_t ld;
    if (!x || !matrix(*x, ld) || !here(*x)) Py_RETURN_NONE;
    const bool bf16 = x->scalar_type() == at::kBFloat16;
    if (!bf16 && x->scalar_type() != at::kFloat) Py_RETURN_NONE;
    if (args[2] != Py_None) {
        seed = plain(args[2]);
        if (!seed || seed->scalar_type() != at::kLong || seed->dim() != 1 || seed->size(0) != 1 || !here(*seed))
            Py_RETURN_NONE;
    }
    const int64_t rows = x->size(0), cols = x->size(1);
    const bool want_t = args[1] == Py_True;
    at::AutoDispatchBelowADInplaceOrView guard;
    Codes c, t;
    fp8_status st;
    {
        Unlocked unlocked;
        c = fresh_codes(rows, cols, *x);
        if (want_t) t = fresh_codes(cols, rows, *x);
        st = fp8_mx4_quantize(x->data_ptr(), bf16 ? FP8_IN_BF16 : FP8_IN_FP32, rows, cols, ld,
                              data<uint8_t>(c.q), c.ldq, data<uint8_t>(c.s), c.ps,
                              want_t ? data<uint8_t>(t.q) : nullptr, t.ldq,
                              want_t ? data<uint8_t>(t.s) : nullptr, t.ps,
                              seed ? data<const uint64_t>(*seed) : nullptr, nullptr, stream());
    }
    if (st != FP8_OK) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(want_t ? 4 : 2);
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(std::move(c.q)));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(std::move(c.s)));
    if (want_t) {
        PyTuple_SET_ITEM(out, 2, THPVariable_Wrap(std::move(t.q)));
        PyTuple_SET_ITEM(out, 3, THPVariable_Wrap(std::move(t.s)));
    }
    return out;
    END_HANDLE_TH_ERRORS
}

// Codes and scales of an Mx4 matrix: q, s, (row, panel distances), cols.
struct Held {
    const at::Tensor* q;
    const at::Tensor* s;
    int64_t ldq, ps, cols;
};
bool held(PyObject* const* args, Held& h)
{
    h.q = plain(args[0]);
    h.s = h.q ? plain(args[1]) : nullptr;
    if (!h.s || h.q->dim() != 2 || !here(*h.q) || !here(*h.s) || !PyTuple_CheckExact(args[2]) ||
        PyTuple_GET_SIZE(args[2]) != 2)
        return false;
    PyObject* d[3] = {PyTuple_GET_ITEM(args[2], 0), PyTuple_GET_ITEM(args[2], 1), args[3]};
    int64_t v[3];
    if (!ints(d, 3, v)) return false;
    h.ldq = v[0];
    h.ps = v[1];
    h.cols = v[2];
    return h.q->size(0) > 0 && h.cols > 0;
}

// (q, s, distances, cols, to fp32): y
PyObject* mx4_dequantize(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Held a;
    if (n != 5 || !held(args, a)) {
        if (PyErr_Occurred()) return nullptr;
        Py_RETURN_NONE;
    }
    const bool fp32 = args[4] == Py_True;
    const int64_t rows = a.q->size(0);
    at::AutoDispatchBelowADInplaceOrView guard;
    at::Tensor y;
    fp8_status st;
    {
        Unlocked unlocked;
        y = fresh({rows, a.cols}, {a.cols, 1}, fp32 ? at::kFloat : at::kBFloat16, *a.q);
        st = fp8_mx4_dequantize(data<const uint8_t>(*a.q), a.ldq, data<const uint8_t>(*a.s), a.ps, rows,
                                a.cols, y.data_ptr(), fp32 ? FP8_IN_FP32 : FP8_IN_BF16, a.cols, stream());
    }
    if (st != FP8_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(std::move(y));
    END_HANDLE_TH_ERRORS
}

// (q, s, distances, cols) of A, then of B: y
PyObject* mx4_mm(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Held a, b;
    if (n != 8 || !held(args, a) || !held(args + 4, b) || a.cols != b.cols) {
        if (PyErr_Occurred()) return nullptr;
        Py_RETURN_NONE;
    }
    const int64_t rows = a.q->size(0), cols = b.q->size(0);
    at::AutoDispatchBelowADInplaceOrView guard;
    at::Tensor y;
    fp8_status st;
    {
        Unlocked unlocked;
        y = fresh({rows, cols}, {cols, 1}, at::kBFloat16, *a.q);
        st = fp8_mx4_mm(data<const uint8_t>(*a.q), a.ldq, data<const uint8_t>(*a.s), a.ps,
                        data<const uint8_t>(*b.q), b.ldq, data<const uint8_t>(*b.s), b.ps, rows, cols,
                        a.cols, y.data_ptr(), cols, nullptr, stream());
    }
    if (st != FP8_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(std::move(y));
    END_HANDLE_TH_ERRORS
}

// (x, router, workspace, address of w1, of w2, experts, inner, top_k,
// renormalize, max_tokens): (y, ids, weights)
PyObject* mx4_moe(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const at::Tensor* x = n == 10 ? plain(args[0]) : nullptr;
    const at::Tensor* router = x ? plain(args[1]) : nullptr;
    const at::Tensor* ws = router ? plain(args[2]) : nullptr;
    int64_t ldx, ldr, v[7];
    if (!ws || !matrix(*x, ldx) || !matrix(*router, ldr)) Py_RETURN_NONE;
    if (!ints(args + 3, 7, v)) return nullptr;
    const int64_t tokens = x->size(0), hidden = x->size(1), top_k = v[4];
    if (x->scalar_type() != at::kBFloat16 || hidden != router->size(1) || tokens > v[6] || !here(*x) || !here(*router) ||
        !here(*ws))
        Py_RETURN_NONE;
    at::AutoDispatchBelowADInplaceOrView guard;
    at::Tensor y, ids, weights;
    fp8_status st;
    {
        Unlocked unlocked;
        y = fresh({tokens, hidden}, {hidden, 1}, at::kBFloat16, *x);
        ids = fresh({tokens, top_k}, {top_k, 1}, at::kInt, *x);
        weights = fresh({tokens, top_k}, {top_k, 1}, at::kFloat, *x);
        st = fp8_mx4_moe(x->data_ptr(), tokens, hidden, ldx, router->data_ptr(), ldr,
                         reinterpret_cast<const fp8_mx4_experts*>(v[0]),
                         reinterpret_cast<const fp8_mx4_experts*>(v[1]), v[2], v[3], top_k, (int32_t)v[5],
                         y.data_ptr(), hidden, data<int32_t>(ids), data<float>(weights), ws->data_ptr(),
                         (size_t)ws->numel(), nullptr, stream());
    }
    if (st != FP8_OK) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(3);
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(std::move(y)));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(std::move(ids)));
    PyTuple_SET_ITEM(out, 2, THPVariable_Wrap(std::move(weights)));
    return out;
    END_HANDLE_TH_ERRORS
}

// A vector of `n` adjacent elements here, or nothing.
bool vector(PyObject* o, at::ScalarType dtype, int64_t n, const at::Tensor*& t)
{
    t = plain(o);
    return t && t->scalar_type() == dtype && t->dim() == 1 && t->size(0) == n && (n <= 1 || t->stride(0) == 1) && here(*t);
}
bool contiguous(PyObject* o, at::ScalarType dtype, int64_t rows, int64_t cols, const at::Tensor*& t)
{
    t = plain(o);
    return t && t->scalar_type() == dtype && t->dim() == 2 && t->size(0) == rows && t->size(1) == cols && t->is_contiguous() &&
           here(*t);
}
bool number(PyObject* o, double& v)
{
    if (!PyFloat_CheckExact(o)) return false;
    v = PyFloat_AS_DOUBLE(o);
    return true;
}
bool values(const at::Tensor& t) { return t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat; }
fp8_dtype code(const at::Tensor& t) { return t.scalar_type() == at::kBFloat16 ? FP8_IN_BF16 : FP8_IN_FP32; }

PyObject* tuple(std::initializer_list<at::Tensor*> of)
{
    PyObject* out = PyTuple_New((Py_ssize_t)of.size());
    if (!out) return nullptr;
    Py_ssize_t i = 0;
    for (at::Tensor* t : of) {
        if (t->defined()) {
            PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(std::move(*t)));
        } else {
            Py_INCREF(Py_None);
            PyTuple_SET_ITEM(out, i++, Py_None);
        }
    }
    return out;
}

// (x, rate, seed, residual): y
PyObject* dropout(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const at::Tensor* x = n == 4 ? plain(args[0]) : nullptr;
    const at::Tensor *seed = nullptr, *residual = nullptr;
    int64_t ld, ldr = 0;
    double rate;
    if (!x || !matrix(*x, ld) || !here(*x) || !values(*x) || !number(args[1], rate) || !vector(args[2], at::kLong, 1, seed))
        Py_RETURN_NONE;
    if (args[3] != Py_None) {
        residual = plain(args[3]);
        if (!residual || !matrix(*residual, ldr) || !here(*residual) || residual->scalar_type() != x->scalar_type() ||
            residual->sizes() != x->sizes())
            Py_RETURN_NONE;
    }
    const int64_t rows = x->size(0), cols = x->size(1);
    at::AutoDispatchBelowADInplaceOrView guard;
    at::Tensor y;
    fp8_status st;
    {
        Unlocked unlocked;
        y = fresh({rows, cols}, {cols, 1}, x->scalar_type(), *x);
        st = fp8_dropout(x->data_ptr(), code(*x), rows, cols, ld, residual ? residual->data_ptr() : nullptr, ldr, rate,
                         data<const uint64_t>(*seed), y.data_ptr(), cols, stream());
    }
    if (st != FP8_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(std::move(y));
    END_HANDLE_TH_ERRORS
}

// (logits, top_k, renormalize, mask): (ids, weights, counts, balance)
PyObject* moe_route(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const at::Tensor* l = n == 4 ? plain(args[0]) : nullptr;
    const at::Tensor* mask = nullptr;
    int64_t ld, k;
    if (!l || !matrix(*l, ld) || !here(*l) || !values(*l)) Py_RETURN_NONE;
    if (!ints(args + 1, 1, &k)) return nullptr;
    const int64_t tokens = l->size(0), experts = l->size(1);
    if (k < 1 || k > experts || (args[3] != Py_None && !vector(args[3], at::kBool, tokens, mask))) Py_RETURN_NONE;
    at::AutoDispatchBelowADInplaceOrView guard;
    at::Tensor ids, weights, counts, balance, ws;
    fp8_status st;
    {
        Unlocked unlocked;
        ids = fresh({tokens, k}, {k, 1}, at::kInt, *l);
        weights = fresh({tokens, k}, {k, 1}, at::kFloat, *l);
        counts = fresh({experts}, {1}, at::kInt, *l);
        balance = fresh({}, {}, at::kFloat, *l);
        const int64_t need = std::max<int64_t>((int64_t)fp8_moe_route_workspace_size(tokens, experts), 1);
        ws = fresh({need}, {1}, at::kByte, *l);
        st = fp8_moe_route(l->data_ptr(), code(*l), tokens, experts, ld, k, args[2] == Py_True,
                           mask ? data<const uint8_t>(*mask) : nullptr, data<int32_t>(ids), data<float>(weights),
                           data<int32_t>(counts), data<float>(balance), ws.data_ptr(), (size_t)need, stream());
    }
    if (st != FP8_OK) return PyLong_FromLong(st);
    return tuple({&ids, &weights, &counts, &balance});
    END_HANDLE_TH_ERRORS
}

// (logits, ids, weights, counts, renormalize, gradient of the weights, of the balance): dlogits
PyObject* moe_route_backward(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const at::Tensor* l = n == 7 ? plain(args[0]) : nullptr;
    const at::Tensor* i = l ? plain(args[1]) : nullptr;
    const at::Tensor *ids, *weights, *counts, *gw = nullptr, *gb = nullptr;
    int64_t ld;
    if (!i || !matrix(*l, ld) || !here(*l) || !values(*l) || i->dim() != 2) Py_RETURN_NONE;
    const int64_t tokens = l->size(0), experts = l->size(1), k = i->size(1);
    if (!contiguous(args[1], at::kInt, tokens, k, ids) || !contiguous(args[2], at::kFloat, tokens, k, weights) ||
        !vector(args[3], at::kInt, experts, counts) ||
        (args[5] != Py_None && !contiguous(args[5], at::kFloat, tokens, k, gw)))
        Py_RETURN_NONE;
    if (args[6] != Py_None) {
        gb = plain(args[6]);
        if (!gb || gb->scalar_type() != at::kFloat || gb->numel() != 1 || !here(*gb)) Py_RETURN_NONE;
    }
    at::AutoDispatchBelowADInplaceOrView guard;
    at::Tensor dl;
    fp8_status st;
    {
        Unlocked unlocked;
        dl = fresh({tokens, experts}, {experts, 1}, l->scalar_type(), *l);
        st = fp8_moe_route_backward(l->data_ptr(), code(*l), tokens, experts, ld, k, args[4] == Py_True,
                                    data<const int32_t>(*ids), data<const float>(*weights), data<const int32_t>(*counts),
                                    gw ? data<const float>(*gw) : nullptr, gb ? data<const float>(*gb) : nullptr,
                                    dl.data_ptr(), experts, stream());
    }
    if (st != FP8_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(std::move(dl));
    END_HANDLE_TH_ERRORS
}

// x [tokens, hidden], w [vocab, hidden], targets [tokens], softcap.
struct Head {
    const at::Tensor *x, *w, *targets;
    int64_t ldx, ldw, tokens, vocab, hidden;
    double softcap;
};
bool head(PyObject* const* args, Head& h)
{
    h.x = plain(args[0]);
    h.w = h.x ? plain(args[1]) : nullptr;
    if (!h.w || !matrix(*h.x, h.ldx) || !matrix(*h.w, h.ldw) || !here(*h.x) || !here(*h.w) ||
        h.x->scalar_type() != at::kBFloat16 || h.w->scalar_type() != at::kBFloat16 || h.x->size(1) != h.w->size(1))
        return false;
    h.tokens = h.x->size(0);
    h.vocab = h.w->size(0);
    h.hidden = h.x->size(1);
    return vector(args[2], at::kLong, h.tokens, h.targets) && number(args[3], h.softcap);
}

// (x, w, targets, softcap): (loss, lse)
PyObject* linear_ce(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Head h;
    if (n != 4 || !head(args, h)) Py_RETURN_NONE;
    at::AutoDispatchBelowADInplaceOrView guard;
    at::Tensor loss, lse, ws;
    fp8_status st;
    {
        Unlocked unlocked;
        loss = fresh({h.tokens}, {1}, at::kFloat, *h.x);
        lse = fresh({h.tokens}, {1}, at::kFloat, *h.x);
        const int64_t need = std::max<int64_t>((int64_t)fp8_linear_ce_workspace_size(h.tokens, h.vocab, h.hidden, 0), 1);
        ws = fresh({need}, {1}, at::kByte, *h.x);
        st = fp8_linear_ce(h.x->data_ptr(), h.ldx, h.w->data_ptr(), h.ldw, h.tokens, h.vocab, h.hidden,
                           data<const int64_t>(*h.targets), (float)h.softcap, data<float>(loss), data<float>(lse),
                           ws.data_ptr(), (size_t)need, stream());
    }
    if (st != FP8_OK) return PyLong_FromLong(st);
    return tuple({&loss, &lse});
    END_HANDLE_TH_ERRORS
}

// (x, w, targets, softcap, lse, gradient of the losses, want dx, want dw): (dx, dw)
PyObject* linear_ce_backward(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Head h;
    const at::Tensor *lse, *grad;
    if (n != 8 || !head(args, h) || !vector(args[4], at::kFloat, h.tokens, lse)) Py_RETURN_NONE;
    grad = plain(args[5]);
    if (!grad || grad->scalar_type() != at::kFloat || grad->dim() != 1 || grad->size(0) != h.tokens || !here(*grad))
        Py_RETURN_NONE;
    at::AutoDispatchBelowADInplaceOrView guard;
    at::Tensor dx, dw, ws;
    fp8_status st;
    {
        Unlocked unlocked;
        if (args[6] == Py_True) dx = fresh({h.tokens, h.hidden}, {h.hidden, 1}, at::kBFloat16, *h.x);
        if (args[7] == Py_True) dw = fresh({h.vocab, h.hidden}, {h.hidden, 1}, at::kBFloat16, *h.x);
        const int64_t need = std::max<int64_t>((int64_t)fp8_linear_ce_workspace_size(h.tokens, h.vocab, h.hidden, 1), 1);
        ws = fresh({need}, {1}, at::kByte, *h.x);
        st = fp8_linear_ce_backward(h.x->data_ptr(), h.ldx, h.w->data_ptr(), h.ldw, h.tokens, h.vocab, h.hidden,
                                    data<const int64_t>(*h.targets), (float)h.softcap, data<const float>(*lse),
                                    data<const float>(*grad), h.tokens > 1 ? grad->stride(0) : 0,
                                    dx.defined() ? dx.data_ptr() : nullptr, h.hidden, dw.defined() ? dw.data_ptr() : nullptr,
                                    h.hidden, ws.data_ptr(), (size_t)need, stream());
    }
    if (st != FP8_OK) return PyLong_FromLong(st);
    return tuple({&dx, &dw});
    END_HANDLE_TH_ERRORS
}

#define FP8MI_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    {"mx4_held", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(mx4_held)), METH_FASTCALL, nullptr},
    {"mx4_quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(mx4_quantize)), METH_FASTCALL, nullptr},
    {"mx4_dequantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(mx4_dequantize)), METH_FASTCALL, nullptr},
    {"mx4_mm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(mx4_mm)), METH_FASTCALL, nullptr},
    {"mx4_moe", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(mx4_moe)), METH_FASTCALL, nullptr},
    FP8MI_METHOD(dropout),
    FP8MI_METHOD(moe_route),
    FP8MI_METHOD(moe_route_backward),
    FP8MI_METHOD(linear_ce),
    FP8MI_METHOD(linear_ce_backward),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8mi_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8mi_torch() { return PyModule_Create(&module); }
