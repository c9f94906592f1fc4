// What the Python module _block_ops needs for every operator: arguments by
// name, checks of torch tensors, allocation, and the library call on the
// device's current stream.
#pragma once

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
#include <cstring>

#include "moe_wna16.h"

namespace moe_module {

struct Functions {
    decltype(&moe_wna16_add_rmsnorm) add_rmsnorm;
    decltype(&moe_wna16_route_topk) route_topk;
    decltype(&moe_wna16_gemm_w8a8) gemm_w8a8;
    decltype(&moe_wna16_gemm_w8a8_workspace_size) gemm_w8a8_workspace_size;
    decltype(&moe_wna16_swiglu_quant) swiglu_quant;
    decltype(&moe_wna16_quant_fp8) quant_fp8;
    decltype(&moe_wna16_swiglu_quant_fp8) swiglu_quant_fp8;
    decltype(&moe_wna16_gemm_fp8) gemm_fp8;
    decltype(&moe_wna16_gemm_fp8_workspace_size) gemm_fp8_workspace_size;
    decltype(&moe_wna16_gemm_fp8_grouped) gemm_fp8_grouped;
    decltype(&moe_wna16_sort_tokens) sort_tokens;
    decltype(&moe_wna16_sort_tokens_workspace_size) sort_tokens_workspace_size;
    decltype(&moe_wna16_combine_tokens) combine_tokens;
    decltype(&moe_wna16_combine_tokens_grad) combine_tokens_grad;
};
inline Functions lib;
inline PyObject *g_load = nullptr;    // loads the library and calls bind(); raises if it is not built
inline PyObject *g_error = nullptr;   // MoeWna16Error(status, name)

// A Python exception is set; unwinds to the module function.
struct Raised {};

[[noreturn]] inline void fail(PyObject *kind, const char *format, ...)
{
    va_list a;
    va_start(a, format);
    PyErr_FormatV(kind, format, a);
    va_end(a);
    throw Raised{};
}

inline const char *name_of(at::ScalarType t) { return c10::toString(t); }

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

inline const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        fail(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

inline const at::Tensor &matrix(PyObject *o, const char *name)
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

inline void check(const at::Tensor &t, const char *name, c10::IntArrayRef shape, at::ScalarType dtype,
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
inline int64_t rows(const at::Tensor &t, const char *name, c10::IntArrayRef shape, at::ScalarType dtype,
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
inline void *flat(const at::Tensor &t, const char *name, c10::IntArrayRef shape, at::ScalarType dtype,
           c10::Device dev)
{
    check(t, name, shape, dtype, dev);
    if (!t.is_contiguous())
        fail(PyExc_ValueError, "%s must be contiguous", name);
    return t.data_ptr();
}

inline int dtype_code(at::ScalarType t, const char *name)
{
    switch (t) {
    case at::kBFloat16: return MOE_WNA16_BF16;
    case at::kHalf: return MOE_WNA16_FP16;
    case at::kFloat: return MOE_WNA16_FP32;
    default:
        fail(PyExc_TypeError, "%s has dtype %s, expected BFloat16, Half or Float", name, name_of(t));
    }
}

inline at::Tensor empty(c10::IntArrayRef shape, at::ScalarType dtype, c10::Device dev)
{
    return at::detail::empty_cuda(shape, dtype, dev, std::nullopt);   // at::empty, undispatched
}

// A product's workspace: its counters zeroed, by a fill kernel (a captured call
// replays it).
inline at::Tensor fresh_workspace(int64_t bytes, c10::Device dev)
{
    at::Tensor t = empty({bytes}, at::kByte, dev);
    t.narrow(0, 0, std::min<int64_t>(bytes, MOE_WNA16_GEMM_SYNC_BYTES)).zero_();
    return t;
}

// The caller's tensor, or a new one.  The caller's counts as changed: a graph that
// has kept it for its gradient says so instead of using the new values.
inline at::Tensor given_or_empty(PyObject *o, const char *name, c10::IntArrayRef shape,
                          at::ScalarType dtype, c10::Device dev)
{
    if (!o)
        return empty(shape, dtype, dev);
    const at::Tensor &t = tensor(o, name);
    if (t.defined() && !t.is_inference())
        t.unsafeGetTensorImpl()->bump_version();
    return t;
}

inline double number(PyObject *o, double otherwise)
{
    if (!o)
        return otherwise;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Raised{};
    return v;
}

inline int integer(PyObject *o, int otherwise)
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

inline bool truth(PyObject *o, bool otherwise)
{
    if (!o)
        return otherwise;
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw Raised{};
    return v != 0;
}

inline void ensure_library()
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

inline void put(PyObject *dict, PyObject *key, const at::Tensor &t)
{
    PyObject *o = THPVariable_Wrap(t);
    if (!o || PyDict_SetItem(dict, key, o) < 0) {
        Py_XDECREF(o);
        throw Raised{};
    }
    Py_DECREF(o);
}

inline PyObject *pair(const at::Tensor &a, const at::Tensor &b)
{
    PyObject *x = THPVariable_Wrap(a), *y = THPVariable_Wrap(b);
    PyObject *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
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

#define MOE_MODULE_FAST(f) \
    reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(moe_module::entry<f>))

// The operators for experts in 8-bit floating point (expert_ops_module.cpp).
bool add_expert_ops(PyObject *module);

}  // namespace moe_module
