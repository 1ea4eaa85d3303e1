// binding_util.hpp -- what the two halves of the Python binding share: argument
// checks, output allocation, the current stream and the way errors are raised.
#pragma once

#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>

#include <cmath>
#include <stdexcept>
#include <string>
#include <vector>

namespace w4a8_binding {

typedef void* Stream;
typedef const char* (*StatusFn)(int);

// set once, by init
inline PyObject *g_error = nullptr, *g_raw_stream = nullptr;
inline StatusFn g_status = nullptr;

constexpr int64_t kGroup = 128;
constexpr int kActSwiglu = 5;

// named by a call that needs no workspace, and never followed: null would ask
// for the size, and null is the address of every empty tensor
alignas(16) inline char g_no_workspace[16];

// the message of a W4A8Error
struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
// a Python error that is set already
struct Raised {};

[[noreturn]] inline void refuse(const std::string& what)
{
    throw Refused(what);
}

// a tensor argument, or null for None
inline const at::Tensor* tensor(PyObject* o, const char* what)
{
    if (o == Py_None)
        return nullptr;
    if (!THPVariable_Check(o))
        refuse(std::string(what) + " must be a tensor");
    return &THPVariable_Unpack(o);
}
inline const at::Tensor& required(PyObject* o, const char* what)
{
    const at::Tensor* t = tensor(o, what);
    if (t == nullptr)
        refuse(std::string(what) + " must be a tensor");
    return *t;
}
inline int64_t integer(PyObject* o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Raised();
    return v;
}
inline float number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Raised();
    return (float)v;
}
inline bool truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw Raised();
    return v != 0;
}

inline std::string name(at::IntArrayRef s)
{
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i)
        r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

inline int type_of(const at::Tensor& t, bool half = false)
{
    switch (t.scalar_type()) {
    case at::kFloat: return 0;
    case at::kBFloat16: return 1;
    case at::kHalf:
        if (half)
            return 2;
        break;
    default: break;
    }
    refuse(std::string("unsupported tensor type ") + c10::toString(t.scalar_type()));
}

// the address of a tensor that must lie on `device` (null: none)
inline void* addr(const at::Tensor* t, const at::Device& device)
{
    if (t == nullptr)
        return nullptr;
    if (t->device() != device)
        refuse("all tensors must be on one GPU");
    return t->data_ptr();
}

// row stride of a [rows, cols] tensor with unit column stride
inline int64_t row_stride(const at::Tensor& t, int64_t rows, int64_t cols, const char* what)
{
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
        refuse(std::string(what) + " must be " + name({rows, cols}) + ", not " + name(t.sizes()));
    if (t.stride(1) != 1 && cols > 1)
        refuse(std::string(what) + " must have unit column stride");
    return rows > 1 ? t.stride(0) : cols;
}

inline void whole(const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type, const char* what)
{
    if (t.sizes() != shape || t.scalar_type() != type || !t.is_contiguous())
        refuse(std::string(what) + " must be a contiguous " + c10::toString(type) + " tensor of shape " + name(shape));
}

// an output: torch's caching allocator, without the way through its dispatcher
inline at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Device& device)
{
    return at::Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
}

inline void need_gpu(const at::Tensor& t)
{
    if (!t.is_cuda())
        refuse("all tensors must be on the GPU");
}

inline Stream stream_of(const at::Device& device)
{
    PyObject* index = PyLong_FromLong(device.index());
    PyObject* s = index ? PyObject_CallOneArg(g_raw_stream, index) : nullptr;
    Py_XDECREF(index);
    if (s == nullptr)
        throw Raised();
    const unsigned long long v = PyLong_AsUnsignedLongLong(s);
    Py_DECREF(s);
    if (PyErr_Occurred())
        throw Raised();
    return (Stream)(uintptr_t)v;
}

// the launch itself runs without the interpreter's lock
template <typename F>
void launch(const char* what, F&& call)
{
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call();
    Py_END_ALLOW_THREADS
    if (rc != 0)
        refuse(std::string(what) + " failed: " + g_status(rc) + " (" + std::to_string(rc) + ")");
}

inline PyObject* given_or(PyObject* given, const at::Tensor& made)
{
    if (given == Py_None)
        return THPVariable_Wrap(made);
    Py_INCREF(given);
    return given;
}
inline PyObject* none_or(PyObject* given, const at::Tensor& made)
{
    if (given == Py_None && !made.defined())
        Py_RETURN_NONE;
    return given_or(given, made);
}

template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& body)
{
    if (g_error == nullptr || got != want) {
        PyErr_SetString(PyExc_TypeError, "binding called with wrong arguments or before init");
        return nullptr;
    }
    try {
        return body();
    } catch (const Raised&) {
    } catch (const Refused& e) {
        PyErr_SetString(g_error, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(g_error, e.what());
    } catch (...) {
        PyErr_SetString(g_error, "unknown C++ exception");
    }
    return nullptr;
}

// the address of an export, as init is given it
inline uintptr_t address(PyObject* o)
{
    const uintptr_t p = (uintptr_t)PyLong_AsUnsignedLongLong(o);
    if (PyErr_Occurred())
        throw Raised();
    return p;
}

// the calls of binding_attn.cpp, whose init takes the addresses of its exports
constexpr Py_ssize_t kAttnExports = 4;
void attn_init(PyObject* const* addresses);
PyObject* gemm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n);
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n);
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n);
PyObject* attn_decode(PyObject*, PyObject* const* a, Py_ssize_t n);

}  // namespace w4a8_binding
