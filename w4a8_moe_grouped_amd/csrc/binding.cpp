// binding.cpp -- the host side of the Python calls whose kernels take a few
// microseconds (moe_route, norm_residual, gemm_epilogue): argument checks,
// output allocation and the call into libw4a8, in one native call.  Through
// ctypes the same steps took 8 to 11 us of host time, more than the kernels of
// a decode batch.  lib.py holds the signatures and the documentation.
//
// The module is given, once, the exception to raise, torch's accessor of the
// current raw stream and the addresses of the three exports.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>

#include <stdexcept>
#include <string>
#include <vector>

namespace {

typedef void* Stream;
typedef int (*RouteFn)(const void*, int, int64_t, int64_t, int64_t, const float*, int, int64_t, int64_t, int, int64_t,
                       int, float, const int32_t*, int32_t*, float*, Stream);
typedef int (*NormFn)(const void*, int, int64_t, const void*, int, int64_t, int64_t, int64_t, int, const void*,
                      const void*, int64_t, int64_t, float, const void*, float, float, void*, int64_t, void*, int64_t,
                      uint8_t*, float*, Stream);
typedef int (*GemmFn)(const uint8_t*, const float*, int64_t, int64_t, const uint8_t*, const float*, int64_t, const void*,
                      int, int, const void*, int64_t, void*, int64_t, void*, size_t*, Stream);
typedef const char* (*StatusFn)(int);

PyObject *g_error = nullptr, *g_raw_stream = nullptr;
RouteFn g_route = nullptr;
NormFn g_norm = nullptr;
GemmFn g_gemm = nullptr;
StatusFn g_status = nullptr;

constexpr int64_t kGroup = 128;
constexpr int kActSwiglu = 5;

// named by a call that needs no workspace, and never followed: null would ask
// for the size, and null is the address of every empty tensor
alignas(16) char g_no_workspace[16];

// the message of a W4A8Error
struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
// a Python error that is set already
struct Raised {};

[[noreturn]] void refuse(const std::string& what)
{
    throw Refused(what);
}

// a tensor argument, or null for None
const at::Tensor* tensor(PyObject* o, const char* what)
{
    if (o == Py_None)
        return nullptr;
    if (!THPVariable_Check(o))
        refuse(std::string(what) + " must be a tensor");
    return &THPVariable_Unpack(o);
}
const at::Tensor& required(PyObject* o, const char* what)
{
    const at::Tensor* t = tensor(o, what);
    if (t == nullptr)
        refuse(std::string(what) + " must be a tensor");
    return *t;
}
int64_t integer(PyObject* o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Raised();
    return v;
}
float number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Raised();
    return (float)v;
}
bool truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw Raised();
    return v != 0;
}

std::string name(at::IntArrayRef s)
{
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i)
        r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

int type_of(const at::Tensor& t, bool half = false)
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
void* addr(const at::Tensor* t, const at::Device& device)
{
    if (t == nullptr)
        return nullptr;
    if (t->device() != device)
        refuse("all tensors must be on one GPU");
    return t->data_ptr();
}

// row stride of a [rows, cols] tensor with unit column stride
int64_t row_stride(const at::Tensor& t, int64_t rows, int64_t cols, const char* what)
{
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
        refuse(std::string(what) + " must be " + name({rows, cols}) + ", not " + name(t.sizes()));
    if (t.stride(1) != 1 && cols > 1)
        refuse(std::string(what) + " must have unit column stride");
    return rows > 1 ? t.stride(0) : cols;
}

void whole(const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type, const char* what)
{
    if (t.sizes() != shape || t.scalar_type() != type || !t.is_contiguous())
        refuse(std::string(what) + " must be a contiguous " + c10::toString(type) + " tensor of shape " + name(shape));
}

// an output: torch's caching allocator, without the way through its dispatcher
at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Device& device)
{
    return at::Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
}

void need_gpu(const at::Tensor& t)
{
    if (!t.is_cuda())
        refuse("all tensors must be on the GPU");
}

Stream stream_of(const at::Device& device)
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

PyObject* given_or(PyObject* given, const at::Tensor& made)
{
    if (given == Py_None)
        return THPVariable_Wrap(made);
    Py_INCREF(given);
    return given;
}
PyObject* none_or(PyObject* given, const at::Tensor& made)
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

// logits, topk, score, bias, num_groups, topk_groups, group_top, renormalize,
// scale, num_tokens, topk_ids, topk_weights
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 12, [&]() -> PyObject* {
        const at::Tensor& logits = required(a[0], "logits");
        need_gpu(logits);
        const at::Device device = logits.device();
        const c10::DeviceGuard guard(device);
        if (logits.dim() != 2)
            refuse("logits must be [T, E]");
        const int64_t T = logits.size(0), E = logits.size(1), k = integer(a[1]);
        if (k < 1 || k > E)
            refuse("topk must be in 1..E");
        const at::Tensor* bias = tensor(a[3], "bias");
        if (bias != nullptr)
            whole(*bias, {E}, at::kFloat, "bias");
        const at::Tensor* num = tensor(a[9], "num_tokens");
        if (num != nullptr && (num->numel() != 1 || num->scalar_type() != at::kInt))
            refuse("num_tokens must be one int32");
        at::Tensor made_ids, made_w;
        const at::Tensor *ids = tensor(a[10], "topk_ids"), *w = tensor(a[11], "topk_weights");
        if (ids != nullptr)
            whole(*ids, {T, k}, at::kInt, "topk_ids");
        if (w != nullptr)
            whole(*w, {T, k}, at::kFloat, "topk_weights");
        if (ids == nullptr)
            made_ids = make({T, k}, at::kInt, device), ids = &made_ids;
        if (w == nullptr)
            made_w = make({T, k}, at::kFloat, device), w = &made_w;
        const int type = type_of(logits, true);
        const int64_t ld = row_stride(logits, T, E, "logits");
        const int score = (int)integer(a[2]);
        const int64_t groups = integer(a[4]), kept = integer(a[5]), group_top = integer(a[6]);
        const int top = group_top == 1 || group_top == 2 ? (int)group_top : 0;  // 0: refused
        const int renorm = truth(a[7]);
        const float scale = number(a[8]);
        const void* x = logits.data_ptr();
        const float* b = (const float*)addr(bias, device);
        const int32_t* nt = (const int32_t*)addr(num, device);
        int32_t* ip = (int32_t*)addr(ids, device);
        float* wp = (float*)addr(w, device);
        const Stream s = stream_of(device);
        launch("w4a8_moe_route", [&] {
            return g_route(x, type, T, E, ld, b, score, groups, kept, top, k, renorm, scale, nt, ip, wp, s);
        });
        PyObject* i = given_or(a[10], made_ids);
        PyObject* v = given_or(a[11], made_w);
        PyObject* r = i != nullptr && v != nullptr ? PyTuple_Pack(2, i, v) : nullptr;
        Py_XDECREF(i);
        Py_XDECREF(v);
        return r;
    });
}

// x, residual, post_weight, gate, residual_scale, pre_weight, weight_offset,
// eps, quantize, keep_residual, residual_out, out, out_scales
PyObject* norm_residual(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 13, [&]() -> PyObject* {
        const at::Tensor *x = tensor(a[0], "x"), *residual = tensor(a[1], "residual");
        const at::Tensor* like = residual != nullptr ? residual : x;
        if (like == nullptr)
            refuse("x or residual must be given");
        need_gpu(*like);
        const at::Device device = like->device();
        const c10::DeviceGuard guard(device);
        if (like->dim() != 2)
            refuse("x and residual must be [T, H]");
        const int64_t T = like->size(0), H = like->size(1), G = H / kGroup;
        const at::ScalarType r_dtype = like->scalar_type();
        const int r_type = type_of(*like);
        int x_type = r_type;
        int64_t ldx = H, ldr = H, ldo = H, ldy = H;
        if (residual != nullptr)
            ldr = row_stride(*residual, T, H, "residual");
        if (x != nullptr) {
            ldx = row_stride(*x, T, H, "x");
            x_type = type_of(*x);
        }
        const at::Tensor *post = tensor(a[2], "post_weight"), *gate = tensor(a[3], "gate"), *pre = tensor(a[5], "pre_weight");
        int p_type = -1;
        for (const at::Tensor* p : {post, pre, gate}) {
            if (p == nullptr)
                continue;
            const int t = type_of(*p);
            if (p_type >= 0 && t != p_type)
                refuse("post_weight, pre_weight and gate must be of one type");
            p_type = t;
            if (p != gate)
                whole(*p, {H}, p->scalar_type(), "a norm's weight");
        }
        int64_t gate_rs = 0, gate_cs = 0;
        if (gate != nullptr) {
            if (gate->dim() == 1 && gate->size(0) == H && gate->is_contiguous()) {
                gate_cs = 1;
            } else if (gate->dim() == 2 && gate->size(0) == T && gate->size(1) == H) {
                gate_rs = row_stride(*gate, T, H, "gate"), gate_cs = 1;
            } else if (gate->dim() == 2 && gate->size(0) == T && gate->size(1) == 1) {
                gate_rs = T > 1 ? gate->stride(0) : 1;
            } else {
                refuse("gate must be a contiguous [H], or [T, H] or [T, 1]");
            }
        }
        const bool quantize = truth(a[8]), keep = truth(a[9]);
        at::Tensor made_r, made_y, made_s;
        const at::Tensor *r_out = tensor(a[10], "residual_out"), *out = tensor(a[11], "out"), *scales = tensor(a[12], "out_scales");
        if (r_out != nullptr) {
            if (r_out->scalar_type() != r_dtype || !keep)
                refuse("residual_out must have the residual's type");
            ldo = row_stride(*r_out, T, H, "residual_out");
        } else if (keep) {
            made_r = make({T, H}, r_dtype, device), r_out = &made_r;
        }
        void *y = nullptr, *codes = nullptr;
        if (pre == nullptr) {
            if (quantize || out != nullptr || scales != nullptr)
                refuse("an output y needs pre_weight");
        } else if (quantize) {
            if (H % kGroup != 0)
                refuse("quantize needs H % 128 == 0");
            if (out != nullptr)
                whole(*out, {T, H}, at::kByte, "out");
            if (scales != nullptr)
                whole(*scales, {T, G}, at::kFloat, "out_scales");
            if (out == nullptr)
                made_y = make({T, H}, at::kByte, device), out = &made_y;
            if (scales == nullptr)
                made_s = make({T, G}, at::kFloat, device), scales = &made_s;
            codes = addr(out, device);
        } else {
            if (scales != nullptr)
                refuse("out_scales needs quantize");
            if (out != nullptr) {
                if (out->scalar_type() != at::kBFloat16)
                    refuse("out must be bf16");
                ldy = row_stride(*out, T, H, "out");
            } else {
                made_y = make({T, H}, at::kBFloat16, device), out = &made_y;
            }
            y = addr(out, device);
        }
        const float r_scale = number(a[4]), offset = number(a[6]), eps = number(a[7]);
        const void *xp = addr(x, device), *rp = addr(residual, device), *wp = addr(post, device), *gp = addr(gate, device),
                   *pp = addr(pre, device);
        void* op = addr(r_out, device);
        float* sp = (float*)addr(scales, device);
        const Stream s = stream_of(device);
        launch("w4a8_norm_residual", [&] {
            return g_norm(xp, x_type, ldx, rp, r_type, ldr, T, H, p_type < 0 ? 0 : p_type, wp, gp, gate_rs, gate_cs, r_scale,
                          pp, offset, eps, op, ldo, y, ldy, (uint8_t*)codes, sp, s);
        });
        PyObject* ro = none_or(a[10], made_r);
        PyObject* yo = none_or(a[11], made_y);
        PyObject* so = none_or(a[12], made_s);
        PyObject* r = ro != nullptr && yo != nullptr && so != nullptr ? PyTuple_Pack(3, ro, yo, so) : nullptr;
        Py_XDECREF(ro);
        Py_XDECREF(yo);
        Py_XDECREF(so);
        return r;
    });
}

// a_q, a_scales, w, w_scales, bias, act, residual, out, workspace
PyObject* gemm_epilogue(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 9, [&]() -> PyObject* {
        const at::Tensor &q = required(a[0], "a_q"), &sa = required(a[1], "a_scales"), &w = required(a[2], "w"),
                         &sw = required(a[3], "w_scales");
        need_gpu(q);
        const at::Device device = q.device();
        const c10::DeviceGuard guard(device);
        if (q.dim() != 2 || w.dim() != 2)
            refuse("a_q must be [M, K] and w [rows, K/2]");
        const int64_t M = q.size(0), K = q.size(1), R = w.size(0), G = K / kGroup;
        const int act = (int)integer(a[5]);
        const int64_t N = act == kActSwiglu ? R / 2 : R;
        if (w.size(1) * 2 != K || N == 0 || (R != N && R != 2 * N))
            refuse("bad operand shapes");
        whole(q, {M, K}, at::kByte, "a_q");
        whole(sa, {M, G}, at::kFloat, "a_scales");
        whole(w, {R, K / 2}, at::kByte, "w");
        whole(sw, {R, G}, at::kFloat, "w_scales");
        const at::Tensor *bias = tensor(a[4], "bias"), *residual = tensor(a[6], "residual");
        int bias_type = 0;
        if (bias != nullptr) {
            bias_type = type_of(*bias);
            whole(*bias, {R}, bias->scalar_type(), "bias");
        }
        int64_t ldr = N, ldo = N;
        if (residual != nullptr) {
            if (residual->scalar_type() != at::kBFloat16)
                refuse("residual must be bf16");
            ldr = row_stride(*residual, M, N, "residual");
        }
        at::Tensor made_out, made_ws;
        const at::Tensor *out = tensor(a[7], "out"), *ws = tensor(a[8], "workspace");
        if (out != nullptr) {
            if (out->scalar_type() != at::kBFloat16)
                refuse("out must be bf16");
            ldo = row_stride(*out, M, N, "out");
        } else {
            made_out = make({M, N}, at::kBFloat16, device), out = &made_out;
        }
        const void *bp = addr(bias, device), *rp = addr(residual, device);
        void* op = addr(out, device);
        const float *sap = (const float*)addr(&sa, device), *swp = (const float*)addr(&sw, device);
        const uint8_t *qp = (const uint8_t*)addr(&q, device), *wp = (const uint8_t*)addr(&w, device);
        if (M > 0) {
            size_t need = 0;
            launch("w4a8_gemm_epilogue(query)", [&] {
                return g_gemm(nullptr, nullptr, M, K, nullptr, nullptr, N, nullptr, 0, act, nullptr, N, nullptr, N, nullptr,
                              &need, nullptr);
            });
            if (ws != nullptr) {
                addr(ws, device);
                if (!ws->is_contiguous())
                    refuse("workspace must be contiguous");
                const size_t given = ws->numel() * ws->element_size();
                if (given < need)
                    refuse("workspace holds " + std::to_string(given) + " bytes, " + std::to_string(need) + " are needed");
            } else if (need > 0) {
                made_ws = make({(int64_t)need}, at::kByte, device), ws = &made_ws;
            }
            void* const given = addr(ws, device);
            void* const wsp = need > 0 ? given : g_no_workspace;
            const Stream s = stream_of(device);
            launch("w4a8_gemm_epilogue", [&] {
                return g_gemm(qp, sap, M, K, wp, swp, N, bp, bias_type, act, rp, ldr, op, ldo, wsp, &need, s);
            });
        }
        return given_or(a[7], made_out);
    });
}

// error, raw_stream, addresses of w4a8_status_string, w4a8_moe_route,
// w4a8_norm_residual, w4a8_gemm_epilogue
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "init takes 6 arguments");
        return nullptr;
    }
    uintptr_t p[4];
    for (int i = 0; i < 4; ++i) {
        p[i] = (uintptr_t)PyLong_AsUnsignedLongLong(a[2 + i]);
        if (PyErr_Occurred())
            return nullptr;
    }
    g_status = (StatusFn)p[0];
    g_route = (RouteFn)p[1];
    g_norm = (NormFn)p[2];
    g_gemm = (GemmFn)p[3];
    Py_INCREF(a[0]);
    Py_INCREF(a[1]);
    Py_XDECREF(g_error);
    Py_XDECREF(g_raw_stream);
    g_error = a[0];
    g_raw_stream = a[1];
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"init", (PyCFunction)(void (*)())init, METH_FASTCALL, nullptr},
    {"moe_route", (PyCFunction)(void (*)())moe_route, METH_FASTCALL, nullptr},
    {"norm_residual", (PyCFunction)(void (*)())norm_residual, METH_FASTCALL, nullptr},
    {"gemm_epilogue", (PyCFunction)(void (*)())gemm_epilogue, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__binding()
{
    return PyModule_Create(&g_module);
}
