// Python module _block_ops: checks, allocation and the library call of the
// operators around the routed layer, for torch tensors.
//
// A decode step calls these operators every few microseconds, and the same
// work written in Python (attribute reads, argument checks, torch.empty,
// ctypes) takes two to three times as long as the launch it prepares.  Only
// that work is here: the kernels are the library's, reached through the C ABI
// functions whose addresses bind() gets from the loaded library.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>

#include "moe_wna16.h"

namespace {

struct Functions {
    decltype(&moe_wna16_add_rmsnorm) add_rmsnorm;
    decltype(&moe_wna16_route_topk) route_topk;
    decltype(&moe_wna16_gemm_w8a8) gemm_w8a8;
    decltype(&moe_wna16_gemm_w8a8_workspace_size) gemm_w8a8_workspace_size;
    decltype(&moe_wna16_swiglu_quant) swiglu_quant;
} lib;
PyObject *g_load = nullptr;    // loads the library and calls bind(); raises if it is not built
PyObject *g_error = nullptr;   // MoeWna16Error(status, name)

// A Python exception is set; unwinds to the module function.
struct Raised {};

[[noreturn]] void fail(PyObject *kind, const char *format, ...)
{
    va_list a;
    va_start(a, format);
    PyErr_FormatV(kind, format, a);
    va_end(a);
    throw Raised{};
}

const char *name_of(at::ScalarType t) { return c10::toString(t); }

// Keyword and positional arguments by name; absent ones and None are null.
template <int N>
struct Args {
    PyObject *v[N] = {};

    // the first `positional` names may be given by position
    Args(const char *fn, PyObject *const (&names)[N], int positional, int required,
         PyObject *const *args, Py_ssize_t nargs, PyObject *kwnames)
    {
        if (nargs > positional)
            fail(PyExc_TypeError, "%s() takes at most %d positional arguments (%zd given)", fn,
                 positional, nargs);
        for (Py_ssize_t i = 0; i < nargs; ++i)
            v[i] = args[i];
        const Py_ssize_t nkw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
        for (Py_ssize_t k = 0; k < nkw; ++k) {
            PyObject *key = PyTuple_GET_ITEM(kwnames, k);
            int at = -1;
            for (int i = 0; i < N && at < 0; ++i)
                if (names[i] == key)                  // interned: the usual case
                    at = i;
            for (int i = 0; i < N && at < 0; ++i)
                if (PyUnicode_Compare(names[i], key) == 0)
                    at = i;
            if (at < 0)
                fail(PyExc_TypeError, "%s() got an unexpected keyword argument '%U'", fn, key);
            if (v[at])
                fail(PyExc_TypeError, "%s() got multiple values for argument '%U'", fn, key);
            v[at] = args[nargs + k];
        }
        for (int i = 0; i < N; ++i) {
            if (v[i] == Py_None && i >= required)
                v[i] = nullptr;
            if (i < required && !v[i])
                fail(PyExc_TypeError, "%s() missing required argument: '%U'", fn, names[i]);
        }
    }
};

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        fail(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

const at::Tensor &matrix(PyObject *o, const char *name)
{
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != 2)
        fail(PyExc_ValueError, "%s must be 2-D", name);
    if (!t.is_cuda())
        fail(PyExc_ValueError, "%s must be on the GPU", name);
    if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX)
        fail(PyExc_ValueError, "%s is too large", name);
    return t;
}

void check(const at::Tensor &t, const char *name, c10::IntArrayRef shape, at::ScalarType dtype,
           c10::Device dev)
{
    if (t.scalar_type() != dtype)
        fail(PyExc_TypeError, "%s has dtype %s, expected %s", name, name_of(t.scalar_type()),
             name_of(dtype));
    if (t.sizes() != shape)
        fail(PyExc_ValueError, "%s has another shape than expected", name);
    if (t.device() != dev)
        fail(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(),
             dev.str().c_str());
}

// A matrix of contiguous rows; its row stride.
int64_t rows(const at::Tensor &t, const char *name, c10::IntArrayRef shape, at::ScalarType dtype,
             c10::Device dev)
{
    check(t, name, shape, dtype, dev);
    if (shape[1] > 1 && t.stride(1) != 1)
        fail(PyExc_ValueError, "%s must have contiguous rows", name);
    if (shape[0] <= 1)
        return shape[1];        // a single row's stride means nothing
    if (t.stride(0) < shape[1])
        fail(PyExc_ValueError, "%s has overlapping rows", name);
    return t.stride(0);
}

// A contiguous tensor; its address.
void *flat(const at::Tensor &t, const char *name, c10::IntArrayRef shape, at::ScalarType dtype,
           c10::Device dev)
{
    check(t, name, shape, dtype, dev);
    if (!t.is_contiguous())
        fail(PyExc_ValueError, "%s must be contiguous", name);
    return t.data_ptr();
}

int dtype_code(at::ScalarType t, const char *name)
{
    switch (t) {
    case at::kBFloat16: return MOE_WNA16_BF16;
    case at::kHalf: return MOE_WNA16_FP16;
    case at::kFloat: return MOE_WNA16_FP32;
    default:
        fail(PyExc_TypeError, "%s has dtype %s, expected BFloat16, Half or Float", name, name_of(t));
    }
}

at::Tensor empty(c10::IntArrayRef shape, at::ScalarType dtype, c10::Device dev)
{
    return at::detail::empty_cuda(shape, dtype, dev, std::nullopt);   // at::empty, undispatched
}

// A product's workspace: its counters zeroed, by a fill kernel (a captured call
// replays it).
at::Tensor fresh_workspace(int64_t bytes, c10::Device dev)
{
    at::Tensor t = empty({bytes}, at::kByte, dev);
    t.narrow(0, 0, std::min<int64_t>(bytes, MOE_WNA16_GEMM_SYNC_BYTES)).zero_();
    return t;
}

// The caller's tensor, or a new one.
at::Tensor given_or_empty(PyObject *o, const char *name, c10::IntArrayRef shape,
                          at::ScalarType dtype, c10::Device dev)
{
    return o ? tensor(o, name) : empty(shape, dtype, dev);
}

double number(PyObject *o, double otherwise)
{
    if (!o)
        return otherwise;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Raised{};
    return v;
}

int integer(PyObject *o, int otherwise)
{
    if (!o)
        return otherwise;
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Raised{};
    if (v > INT32_MAX || v < INT32_MIN)
        fail(PyExc_ValueError, "an argument does not fit 32 bits");
    return (int)v;
}

bool truth(PyObject *o, bool otherwise)
{
    if (!o)
        return otherwise;
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw Raised{};
    return v != 0;
}

void ensure_library()
{
    if (!lib.add_rmsnorm) {
        PyObject *r = g_load ? PyObject_CallNoArgs(g_load) : nullptr;
        if (!r && !PyErr_Occurred())
            PyErr_SetString(PyExc_RuntimeError, "_block_ops is used before its package");
        Py_XDECREF(r);
        if (PyErr_Occurred())
            throw Raised{};
    }
}

// Calls f(stream) with dev current and its current stream, without the
// interpreter lock, and raises MoeWna16Error for a status other than OK.
template <class F>
void launch(const char *name, c10::Device dev, F &&f)
{
    int st;
    {
        const c10::DeviceGuard guard(dev);
        hipStream_t stream = c10::hip::getCurrentHIPStream(dev.index()).stream();
        Py_BEGIN_ALLOW_THREADS
        st = f(stream);
        Py_END_ALLOW_THREADS
    }
    if (st != MOE_WNA16_OK) {
        PyObject *e = PyObject_CallFunction(g_error, "is", st, name);
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
        throw Raised{};
    }
}

void put(PyObject *dict, PyObject *key, const at::Tensor &t)
{
    PyObject *o = THPVariable_Wrap(t);
    if (!o || PyDict_SetItem(dict, key, o) < 0) {
        Py_XDECREF(o);
        throw Raised{};
    }
    Py_DECREF(o);
}

PyObject *pair(const at::Tensor &a, const at::Tensor &b)
{
    PyObject *x = THPVariable_Wrap(a), *y = THPVariable_Wrap(b);
    PyObject *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

// Interned argument and result names.
PyObject *n_x, *n_weight, *n_residual, *n_eps, *n_quant, *n_normed, *n_residual_out, *n_out, *n_q,
    *n_scale, *n_y, *n_logits, *n_topk, *n_bias, *n_score, *n_groups, *n_topk_groups,
    *n_renormalize, *n_ids, *n_weights, *n_a, *n_a_scale, *n_w, *n_w_scale, *n_addend, *n_out_dtype,
    *n_workspace, *n_gu, *n_alpha, *n_beta, *n_clamp, *s_softmax, *s_sigmoid;

PyObject *add_rmsnorm(PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    PyObject *const names[] = {n_x,   n_weight, n_residual,     n_eps, n_quant,
                               n_normed, n_residual_out, n_out, n_q,   n_scale};
    const Args<10> p("add_rmsnorm", names, 3, 2, args, nargs, kw);
    const at::Tensor &x = matrix(p.v[0], "x");
    const at::Tensor &weight = tensor(p.v[1], "weight");
    const int64_t T = x.size(0), H = x.size(1);
    const auto shape = x.sizes();
    const at::ScalarType dt = x.scalar_type();
    const c10::Device dev = x.device();
    const int code = dtype_code(dt, "x");
    const int64_t xs = rows(x, "x", shape, dt, dev);
    const void *wp = flat(weight, "weight", {H}, dt, dev);
    const bool quant = truth(p.v[4], false), normed = truth(p.v[5], true);
    const float eps = (float)number(p.v[3], 1e-6);
    ensure_library();
    at::Tensor h, y, q, scale;
    int64_t rs = H, qs = H;
    const void *rp = nullptr;
    if (p.v[2]) {
        const at::Tensor &r = tensor(p.v[2], "residual");
        rs = rows(r, "residual", shape, dt, dev);
        rp = r.data_ptr();
        h = given_or_empty(p.v[6], "residual_out", shape, dt, dev);
        flat(h, "residual_out", shape, dt, dev);
    } else if (p.v[6]) {
        fail(PyExc_ValueError, "residual_out without a residual");
    }
    if (normed) {
        y = given_or_empty(p.v[7], "out", shape, dt, dev);
        flat(y, "out", shape, dt, dev);
    }
    if (quant) {
        q = given_or_empty(p.v[8], "q", shape, at::kChar, dev);
        qs = rows(q, "q", shape, at::kChar, dev);
        scale = given_or_empty(p.v[9], "scale", {T}, at::kFloat, dev);
        flat(scale, "scale", {T}, at::kFloat, dev);
    }
    auto ptr = [](const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; };
    launch("moe_wna16_add_rmsnorm", dev, [&](hipStream_t s) {
        return lib.add_rmsnorm(x.data_ptr(), rp, wp, (int)T, (int)H, xs, rs, code, eps, ptr(h),
                               ptr(y), (int8_t *)ptr(q), qs, (float *)ptr(scale), s);
    });
    PyObject *d = PyDict_New();
    if (!d)
        throw Raised{};
    try {
        if (h.defined())
            put(d, n_residual, h);
        if (normed)
            put(d, n_y, y);
        if (quant) {
            put(d, n_q, q);
            put(d, n_scale, scale);
        }
    } catch (...) {
        Py_DECREF(d);
        throw;
    }
    return d;
}

PyObject *route_topk(PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    PyObject *const names[] = {n_logits,      n_topk,  n_bias, n_score, n_groups, n_topk_groups,
                               n_renormalize, n_scale, n_ids,  n_weights};
    const Args<10> p("route_topk", names, 2, 2, args, nargs, kw);
    const at::Tensor &logits = matrix(p.v[0], "logits");
    const int64_t T = logits.size(0), E = logits.size(1);
    const c10::Device dev = logits.device();
    const int code = dtype_code(logits.scalar_type(), "logits");
    const int64_t ls = rows(logits, "logits", logits.sizes(), logits.scalar_type(), dev);
    const int topk = integer(p.v[1], 0);
    int score = MOE_WNA16_SOFTMAX;
    if (p.v[3] && p.v[3] != s_softmax) {
        if (!PyUnicode_Check(p.v[3]))
            fail(PyExc_TypeError, "score must be a string");
        if (PyUnicode_Compare(p.v[3], s_sigmoid) == 0)
            score = MOE_WNA16_SIGMOID;
        else if (PyUnicode_Compare(p.v[3], s_softmax) != 0)
            fail(PyExc_ValueError, "score is '%U', expected 'softmax' or 'sigmoid'", p.v[3]);
    }
    const void *bias = p.v[2] ? flat(tensor(p.v[2], "bias"), "bias", {E}, at::kFloat, dev) : nullptr;
    const int groups = integer(p.v[4], 1), topk_groups = integer(p.v[5], 1);
    const bool renormalize = truth(p.v[6], true);
    const float scale = (float)number(p.v[7], 1.0);
    if (topk < 1)
        fail(PyExc_ValueError, "topk must be at least 1");
    ensure_library();
    at::Tensor ids = given_or_empty(p.v[8], "ids", {T, topk}, at::kInt, dev);
    at::Tensor weights = given_or_empty(p.v[9], "weights", {T, topk}, at::kFloat, dev);
    void *ip = flat(ids, "ids", {T, topk}, at::kInt, dev);
    void *wp = flat(weights, "weights", {T, topk}, at::kFloat, dev);
    launch("moe_wna16_route_topk", dev, [&](hipStream_t s) {
        return lib.route_topk(logits.data_ptr(), (const float *)bias, (int)T, (int)E, ls, code,
                              topk, score, groups, topk_groups, renormalize, scale, (int32_t *)ip,
                              (float *)wp, s);
    });
    return pair(ids, weights);
}

PyObject *gemm_w8a8(PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    PyObject *const names[] = {n_a,      n_a_scale,   n_w,   n_w_scale,
                               n_addend, n_out_dtype, n_out, n_workspace};
    const Args<8> p("gemm_w8a8", names, 4, 4, args, nargs, kw);
    const at::Tensor &a = matrix(p.v[0], "a"), &w = matrix(p.v[2], "w");
    const int64_t T = a.size(0), K = a.size(1), N = w.size(0);
    const c10::Device dev = a.device();
    at::ScalarType dt = at::kBFloat16;
    if (p.v[5]) {
        if (!THPDtype_Check(p.v[5]))
            fail(PyExc_TypeError, "out_dtype must be a torch.dtype");
        dt = reinterpret_cast<THPDtype *>(p.v[5])->scalar_type;
    }
    const int code = dtype_code(dt, "out_dtype");
    const int64_t lda = rows(a, "a", {T, K}, at::kChar, dev);
    const int64_t ldw = rows(w, "w", {N, K}, at::kChar, dev);
    const void *sa = flat(tensor(p.v[1], "a_scale"), "a_scale", {T}, at::kFloat, dev);
    const void *sw = flat(tensor(p.v[3], "w_scale"), "w_scale", {N}, at::kFloat, dev);
    const void *ap = nullptr;
    int64_t lad = N;
    if (p.v[4]) {
        const at::Tensor &add = tensor(p.v[4], "addend");
        lad = rows(add, "addend", {T, N}, dt, dev);
        ap = add.data_ptr();
    }
    ensure_library();
    at::Tensor out = given_or_empty(p.v[6], "out", {T, N}, dt, dev);
    const int64_t ldo = rows(out, "out", {T, N}, dt, dev);
    at::Tensor ws;
    if (p.v[7]) {
        ws = tensor(p.v[7], "workspace");
        flat(ws, "workspace", {ws.numel()}, at::kByte, dev);
    } else {
        size_t bytes = 0;
        if (lib.gemm_w8a8_workspace_size((int)T, (int)N, (int)K, &bytes) == MOE_WNA16_OK && bytes)
            ws = fresh_workspace((int64_t)bytes, dev);
    }
    launch("moe_wna16_gemm_w8a8", dev, [&](hipStream_t s) {
        return lib.gemm_w8a8((const int8_t *)a.data_ptr(), (const float *)sa,
                             (const int8_t *)w.data_ptr(), (const float *)sw, ap, (int)T, (int)N,
                             (int)K, lda, ldw, lad, ldo, code, out.data_ptr(),
                             ws.defined() ? ws.data_ptr() : nullptr,
                             ws.defined() ? (size_t)ws.numel() : 0, s);
    });
    return THPVariable_Wrap(out);
}

PyObject *swiglu_quant(PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    PyObject *const names[] = {n_gu, n_alpha, n_beta, n_clamp, n_q, n_scale};
    const Args<6> p("swiglu_quant", names, 1, 1, args, nargs, kw);
    const at::Tensor &gu = matrix(p.v[0], "gu");
    const int64_t T = gu.size(0), I = gu.size(1) / 2;
    if (gu.size(1) % 2)
        fail(PyExc_ValueError, "gu must hold gate and up halves of equal length");
    const c10::Device dev = gu.device();
    const int code = dtype_code(gu.scalar_type(), "gu");
    const int64_t gs = rows(gu, "gu", gu.sizes(), gu.scalar_type(), dev);
    const float alpha = (float)number(p.v[1], 1.0), beta = (float)number(p.v[2], 0.0);
    const float clamp = (float)number(p.v[3], INFINITY);
    ensure_library();
    at::Tensor q = given_or_empty(p.v[4], "q", {T, I}, at::kChar, dev);
    at::Tensor scale = given_or_empty(p.v[5], "scale", {T}, at::kFloat, dev);
    const int64_t qs = rows(q, "q", {T, I}, at::kChar, dev);
    void *sp = flat(scale, "scale", {T}, at::kFloat, dev);
    launch("moe_wna16_swiglu_quant", dev, [&](hipStream_t s) {
        return lib.swiglu_quant(gu.data_ptr(), (int)T, (int)I, gs, code, alpha, beta, clamp,
                                (int8_t *)q.data_ptr(), qs, (float *)sp, s);
    });
    return pair(q, scale);
}

template <PyObject *(*F)(PyObject *const *, Py_ssize_t, PyObject *)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    HANDLE_TH_ERRORS            // torch's own errors (out of memory among them)
    try {
        return F(args, nargs, kw);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// bind(load, error, addresses): the loader, the exception class, and the five
// functions' addresses (0 before the library is loaded).
PyObject *bind(PyObject *, PyObject *args)
{
    PyObject *load, *error;
    unsigned long long f[5];
    if (!PyArg_ParseTuple(args, "OO(KKKKK)", &load, &error, &f[0], &f[1], &f[2], &f[3], &f[4]))
        return nullptr;
    Py_INCREF(load);
    Py_INCREF(error);
    Py_XSETREF(g_load, load);
    Py_XSETREF(g_error, error);
    lib.add_rmsnorm = reinterpret_cast<decltype(lib.add_rmsnorm)>(f[0]);
    lib.route_topk = reinterpret_cast<decltype(lib.route_topk)>(f[1]);
    lib.gemm_w8a8 = reinterpret_cast<decltype(lib.gemm_w8a8)>(f[2]);
    lib.gemm_w8a8_workspace_size = reinterpret_cast<decltype(lib.gemm_w8a8_workspace_size)>(f[3]);
    lib.swiglu_quant = reinterpret_cast<decltype(lib.swiglu_quant)>(f[4]);
    Py_RETURN_NONE;
}

const char k_add_rmsnorm[] = R"(add_rmsnorm(x, weight, residual=None, *, eps=1e-6, quant=False, normed=True, residual_out=None, out=None, q=None, scale=None) -> dict

Residual addition and root-mean-square norm of rows x [T, H].

Returns a dict: "residual" (the sum h, if a residual is given: rounded to x's
type), "y" (h * weight / rms(h), if normed) and, with quant, "q" int8 [T, H] and
"scale" float32 [T] with y about q * scale.  x, residual: bf16, fp16 or fp32, rows
may be strided; weight [H] of the same type.  Outputs are contiguous (q may have
strided rows); pass them in to reuse memory (residual_out may be x or residual
itself).  No gradient: outputs carry no graph.)";

const char k_route_topk[] = R"(route_topk(logits, topk, *, bias=None, score="softmax", groups=1, topk_groups=1, renormalize=True, scale=1.0, ids=None, weights=None) -> (ids, weights)

Expert ids int32 [T, topk] and routing weights float32 [T, topk], as forward()
reads them, of router logits [T, E] (bf16, fp16 or fp32; rows may be strided).

score "softmax" or "sigmoid"; bias [E] float32 is added for picking only; with
groups > 1 only the experts of the topk_groups best groups (by the sum of their
two largest) are picked.  Experts with a logit of -inf or NaN are never picked;
slots without an expert get id -1 and weight 0.  No gradient: outputs carry no
graph.)";

const char k_gemm_w8a8[] = R"(gemm_w8a8(a, a_scale, w, w_scale, *, addend=None, out_dtype=torch.bfloat16, out=None, workspace=None) -> out

(a @ w.T) * a_scale[:, None] * w_scale + addend, the sum exact in int32, the rest in
FP32, rounded to out_dtype at the end.

a int8 [T, K], a_scale float32 [T]; w int8 [N, K], w_scale float32 [N]; addend
[T, N] of out_dtype (bf16, fp16, fp32).  Rows may be strided.  out may be the
addend.  workspace: from gemm_w8a8_workspace_for, kept by the caller and used by
one call at a time; allocated here when it is needed and not given.  No gradient:
the output carries no graph.)";

const char k_swiglu_quant[] = R"(swiglu_quant(gu, *, alpha=1.0, beta=0.0, clamp=None, q=None, scale=None) -> (q, scale)

SwiGLU of rows gu = [gate (I), up (I)] [T, 2I] (bf16, fp16 or fp32; rows may be
strided) in 8 bits: codes int8 [T, I] and scale float32 [T].  alpha, beta, clamp
as in forward().  No gradient: outputs carry no graph.)";

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f>))
PyMethodDef methods[] = {
    {"add_rmsnorm", FAST(add_rmsnorm), METH_FASTCALL | METH_KEYWORDS, k_add_rmsnorm},
    {"route_topk", FAST(route_topk), METH_FASTCALL | METH_KEYWORDS, k_route_topk},
    {"gemm_w8a8", FAST(gemm_w8a8), METH_FASTCALL | METH_KEYWORDS, k_gemm_w8a8},
    {"swiglu_quant", FAST(swiglu_quant), METH_FASTCALL | METH_KEYWORDS, k_swiglu_quant},
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block_ops", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block_ops(void)
{
    struct { PyObject **at; const char *name; } const all[] = {
        {&n_x, "x"}, {&n_weight, "weight"}, {&n_residual, "residual"}, {&n_eps, "eps"},
        {&n_quant, "quant"}, {&n_normed, "normed"}, {&n_residual_out, "residual_out"},
        {&n_out, "out"}, {&n_q, "q"}, {&n_scale, "scale"}, {&n_y, "y"}, {&n_logits, "logits"},
        {&n_topk, "topk"}, {&n_bias, "bias"}, {&n_score, "score"}, {&n_groups, "groups"},
        {&n_topk_groups, "topk_groups"}, {&n_renormalize, "renormalize"}, {&n_ids, "ids"},
        {&n_weights, "weights"}, {&n_a, "a"}, {&n_a_scale, "a_scale"}, {&n_w, "w"},
        {&n_w_scale, "w_scale"}, {&n_addend, "addend"}, {&n_out_dtype, "out_dtype"},
        {&n_workspace, "workspace"}, {&n_gu, "gu"}, {&n_alpha, "alpha"}, {&n_beta, "beta"},
        {&n_clamp, "clamp"}, {&s_softmax, "softmax"}, {&s_sigmoid, "sigmoid"}};
    for (const auto &n : all)
        if (!(*n.at = PyUnicode_InternFromString(n.name)))
            return nullptr;
    return PyModule_Create(&module);
}
