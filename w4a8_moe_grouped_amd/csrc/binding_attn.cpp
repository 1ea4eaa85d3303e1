// binding_attn.cpp -- the host side of the Python calls of the attention half of
// a served block (gemm_fp8, rope, kv_append, attn_decode), as binding.cpp has it
// for the others.
#include "binding_util.hpp"

#include "w4a8.h"

namespace w4a8_binding {

namespace {

typedef decltype(&w4a8_gemm_fp8) GemmFn;
typedef decltype(&w4a8_rope) RopeFn;
typedef decltype(&w4a8_kv_append) AppendFn;
typedef decltype(&w4a8_attn_decode) AttnFn;

GemmFn g_gemm = nullptr;
RopeFn g_rope = nullptr;
AppendFn g_append = nullptr;
AttnFn g_attn = nullptr;

// [n, heads, D] with unit stride in D
struct Heads {
    int64_t first, heads, D, first_stride, head_stride;
};
Heads heads_of(const at::Tensor& t, const char* what)
{
    if (t.dim() != 3)
        refuse(std::string(what) + " must have three dimensions, not " + std::to_string(t.dim()));
    const int64_t n = t.size(0), h = t.size(1), D = t.size(2);
    if (D > 1 && t.stride(2) != 1)
        refuse(std::string(what) + " must have unit stride in its last dimension");
    // strides along one element are never used
    return Heads{n, h, D, n > 1 ? t.stride(0) : 0, h > 1 ? t.stride(1) : 0};
}
Heads heads_like(const at::Tensor& t, const char* what, int64_t n, int64_t heads, int64_t D, at::ScalarType type)
{
    const Heads h = heads_of(t, what);
    if (h.first != n || h.heads != heads || h.D != D || t.scalar_type() != type)
        refuse(std::string(what) + " must be " + c10::toString(type) + " " + name({n, heads, D}) + ", not " +
               c10::toString(t.scalar_type()) + " " + name(t.sizes()));
    return h;
}

// an int32 vector
const int32_t* ints(const at::Tensor& t, int64_t n, const char* what, const at::Device& device)
{
    whole(t, {n}, at::kInt, what);
    return (const int32_t*)addr(&t, device);
}

struct Rotation {
    const int32_t* positions = nullptr;
    const double* frequencies = nullptr;
    int64_t R = 0;
};
Rotation rotation(PyObject* positions, PyObject* frequencies, int64_t T, const at::Device& device)
{
    Rotation r;
    const at::Tensor *p = tensor(positions, "positions"), *f = tensor(frequencies, "frequencies");
    if ((p == nullptr) != (f == nullptr))
        refuse("positions and frequencies go together");
    if (f == nullptr)
        return r;
    if (f->dim() != 1)
        refuse("frequencies must be one-dimensional");
    whole(*f, {f->size(0)}, at::kDouble, "frequencies");
    r.R = 2 * f->size(0);
    r.positions = ints(*p, T, "positions", device);
    r.frequencies = (const double*)addr(f, device);
    return r;
}

// k_cache, v_cache [pages, page_size, kv heads, D], k_scales, v_scales [pages, kv heads, page_size]
w4a8_kv_cache cache_of(PyObject* k_cache, PyObject* v_cache, PyObject* k_scales, PyObject* v_scales, const at::Device& device)
{
    const at::Tensor &k = required(k_cache, "k_cache"), &v = required(v_cache, "v_cache");
    const at::Tensor *ks = tensor(k_scales, "k_scales"), *vs = tensor(v_scales, "v_scales");
    w4a8_kv_cache c = {};
    if (k.dim() != 4 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
        refuse("k_cache and v_cache must be [pages, page_size, kv_heads, D] of one type");
    switch (k.scalar_type()) {
    case at::kBFloat16: c.type = W4A8_TYPE_BF16; break;
    case at::kHalf: c.type = W4A8_TYPE_FP16; break;
    case at::kByte:
    case at::kFloat8_e4m3fn: c.type = W4A8_TYPE_E4M3; break;
    default: refuse(std::string("unsupported cache type ") + c10::toString(k.scalar_type()));
    }
    c.num_pages = k.size(0), c.page_size = k.size(1), c.kv_heads = k.size(2), c.head_dim = k.size(3);
    if (k.numel() == 0)
        refuse("the cache is empty");
    const bool codes = c.type == W4A8_TYPE_E4M3;
    if ((ks != nullptr) != codes || (vs != nullptr) != codes)
        refuse("a cache of e4m3 codes, and no other, has k_scales and v_scales");
    if (codes) {
        whole(*ks, {c.num_pages, c.kv_heads, c.page_size}, at::kFloat, "k_scales");
        whole(*vs, {c.num_pages, c.kv_heads, c.page_size}, at::kFloat, "v_scales");
    }
    int64_t* strides[2][3] = {{&c.k_page_stride, &c.k_token_stride, &c.k_head_stride},
                              {&c.v_page_stride, &c.v_token_stride, &c.v_head_stride}};
    const at::Tensor* sides[2] = {&k, &v};
    for (int i = 0; i < 2; ++i) {
        if (c.head_dim > 1 && sides[i]->stride(3) != 1)
            refuse("k_cache and v_cache must have unit stride in their last dimension");
        for (int j = 0; j < 3; ++j)
            *strides[i][j] = sides[i]->size(j) > 1 ? sides[i]->stride(j) : 0;
    }
    c.k = addr(&k, device);
    c.v = addr(&v, device);
    c.k_scales = (float*)addr(ks, device);
    c.v_scales = (float*)addr(vs, device);
    return c;
}

// the workspace of a call: the one given, checked, or a new one
void* workspace_of(const at::Tensor* given, size_t need, at::Tensor& made, const at::Device& device)
{
    if (given != nullptr) {
        addr(given, device);
        if (!given->is_contiguous())
            refuse("workspace must be contiguous");
        const size_t bytes = given->numel() * given->element_size();
        if (bytes < need)
            refuse("workspace holds " + std::to_string(bytes) + " bytes, " + std::to_string(need) + " are needed");
    } else if (need > 0) {
        made = make({(int64_t)need}, at::kByte, device);
        given = &made;
    }
    return need > 0 ? addr(given, device) : g_no_workspace;
}

}  // namespace

void attn_init(PyObject* const* a)
{
    g_gemm = (GemmFn)address(a[0]);
    g_rope = (RopeFn)address(a[1]);
    g_append = (AppendFn)address(a[2]);
    g_attn = (AttnFn)address(a[3]);
}

// a_q, a_scales, w, w_scales, bias, act, residual, out, workspace
PyObject* gemm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 9, [&]() -> PyObject* {
        const at::Tensor &q = required(a[0], "a_q"), &sa = required(a[1], "a_scales"), &w = required(a[2], "w"),
                         &sw = required(a[3], "w_scales");
        need_gpu(q);
        const at::Device device = q.device();
        const c10::DeviceGuard guard(device);
        if (q.dim() != 2 || w.dim() != 2)
            refuse("a_q must be [M, K] and w [rows, K]");
        const int64_t M = q.size(0), K = q.size(1), R = w.size(0), G = K / kGroup;
        const int act = (int)integer(a[5]);
        const int64_t N = act == kActSwiglu ? R / 2 : R;
        if (w.size(1) != K || N == 0 || (R != N && R != 2 * N))
            refuse("bad operand shapes");
        auto codes = [](const at::Tensor& t, at::IntArrayRef shape, const char* what) {
            whole(t, shape, t.scalar_type() == at::kFloat8_e4m3fn ? at::kFloat8_e4m3fn : at::kByte, what);
        };
        codes(q, {M, K}, "a_q");
        whole(sa, {M, G}, at::kFloat, "a_scales");
        codes(w, {R, K}, "w");
        whole(sw, {(R + kGroup - 1) / kGroup, G}, at::kFloat, "w_scales");
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
            launch("w4a8_gemm_fp8(query)", [&] {
                return g_gemm(nullptr, nullptr, M, K, nullptr, nullptr, N, nullptr, 0, act, nullptr, N, nullptr, N, nullptr,
                              &need, nullptr);
            });
            void* const wsp = workspace_of(ws, need, made_ws, device);
            const hipStream_t s = (hipStream_t)stream_of(device);
            launch("w4a8_gemm_fp8", [&] {
                return g_gemm(qp, sap, M, K, wp, swp, N, bp, bias_type, act, rp, ldr, op, ldo, wsp, &need, s);
            });
        }
        return given_or(a[7], made_out);
    });
}

// x, positions, frequencies, interleaved, magnitude, out
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 6, [&]() -> PyObject* {
        const at::Tensor& x = required(a[0], "x");
        need_gpu(x);
        const at::Device device = x.device();
        const c10::DeviceGuard guard(device);
        const Heads h = heads_of(x, "x");
        const int type = type_of(x, true);
        const Rotation r = rotation(a[1], a[2], h.first, device);
        const bool interleaved = truth(a[3]);
        const float magnitude = number(a[4]);
        at::Tensor made;
        const at::Tensor* out = tensor(a[5], "out");
        if (out == nullptr)
            made = make({h.first, h.heads, h.D}, x.scalar_type(), device), out = &made;
        const Heads o = heads_like(*out, "out", h.first, h.heads, h.D, x.scalar_type());
        const void* xp = addr(&x, device);
        void* op = addr(out, device);
        const hipStream_t s = (hipStream_t)stream_of(device);
        launch("w4a8_rope", [&] {
            return g_rope(xp, type, h.first, h.heads, h.D, h.first_stride, h.head_stride, r.positions, r.frequencies, r.R,
                          interleaved, magnitude, op, o.first_stride, o.head_stride, s);
        });
        return given_or(a[5], made);
    });
}

// k, v, k_cache, v_cache, slots, k_scales, v_scales, positions, frequencies,
// interleaved, magnitude, q, q_out
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 13, [&]() -> PyObject* {
        const at::Tensor &k = required(a[0], "k"), &v = required(a[1], "v"), &slots = required(a[4], "slots");
        need_gpu(k);
        const at::Device device = k.device();
        const c10::DeviceGuard guard(device);
        const w4a8_kv_cache cache = cache_of(a[2], a[3], a[5], a[6], device);
        const int type = type_of(k, true);
        const Heads hk = heads_of(k, "k");
        const int64_t T = hk.first;
        if (hk.heads != cache.kv_heads || hk.D != cache.head_dim)
            refuse("k must be [T, kv_heads, D] as the cache has them, not " + name(k.sizes()));
        const Heads hv = heads_like(v, "v", T, hk.heads, hk.D, k.scalar_type());
        whole(slots, {T}, at::kLong, "slots");
        const Rotation r = rotation(a[7], a[8], T, device);
        const bool interleaved = truth(a[9]);
        const float magnitude = number(a[10]);
        const at::Tensor *q = tensor(a[11], "q"), *q_out = tensor(a[12], "q_out");
        at::Tensor made;
        Heads hq = {}, ho = {};
        if (q != nullptr) {
            hq = heads_of(*q, "q");
            heads_like(*q, "q", T, hq.heads, hk.D, k.scalar_type());
            if (q_out == nullptr)
                made = make({T, hq.heads, hq.D}, q->scalar_type(), device), q_out = &made;
            ho = heads_like(*q_out, "q_out", T, hq.heads, hq.D, q->scalar_type());
        } else if (q_out != nullptr) {
            refuse("q_out needs q");
        }
        if (T > 0) {
            const void *kp = addr(&k, device), *vp = addr(&v, device), *qp = addr(q, device);
            const int64_t* sp = (const int64_t*)addr(&slots, device);
            void* op = addr(q_out, device);
            if (hq.heads == 0)  // an empty tensor's address is null
                qp = op = nullptr;
            const hipStream_t s = (hipStream_t)stream_of(device);
            launch("w4a8_kv_append", [&] {
                return g_append(qp, hq.first_stride, hq.head_stride, hq.heads, kp, hk.first_stride, hk.head_stride, vp,
                                hv.first_stride, hv.head_stride, type, T, sp, r.positions, r.frequencies, r.R, interleaved,
                                magnitude, &cache, op, ho.first_stride, ho.head_stride, s);
            });
        }
        if (q == nullptr)
            Py_RETURN_NONE;
        return given_or(a[12], made);
    });
}

// q, k_cache, v_cache, page_table, seq_lens, k_scales, v_scales, scale,
// window, return_lse, out, lse, workspace
PyObject* attn_decode(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 13, [&]() -> PyObject* {
        const at::Tensor &q = required(a[0], "q"), &table = required(a[3], "page_table"), &lens = required(a[4], "seq_lens");
        need_gpu(q);
        const at::Device device = q.device();
        const c10::DeviceGuard guard(device);
        const w4a8_kv_cache cache = cache_of(a[1], a[2], a[5], a[6], device);
        const int type = type_of(q, true);
        const Heads h = heads_of(q, "q");
        const int64_t B = h.first;
        if (h.D != cache.head_dim)
            refuse("q must be [B, q_heads, D] with the cache's D, not " + name(q.sizes()));
        if (table.dim() != 2 || table.size(0) != B || table.scalar_type() != at::kInt ||
            (table.size(1) > 1 && table.stride(1) != 1))
            refuse("page_table must be int32 [B, max_pages] with unit column stride");
        const int64_t max_pages = table.size(1), ld = B > 1 ? table.stride(0) : max_pages;
        const int32_t* lp = ints(lens, B, "seq_lens", device);
        const float scale = a[7] == Py_None ? (float)(1.0 / std::sqrt((double)h.D)) : number(a[7]);
        const int64_t window = integer(a[8]);
        const bool want_lse = truth(a[9]);
        at::Tensor made_out, made_lse, made_ws;
        const at::Tensor *out = tensor(a[10], "out"), *lse = tensor(a[11], "lse"), *ws = tensor(a[12], "workspace");
        if (out == nullptr)
            made_out = make({B, h.heads, h.D}, q.scalar_type(), device), out = &made_out;
        const Heads o = heads_like(*out, "out", B, h.heads, h.D, q.scalar_type());
        if (lse != nullptr)
            whole(*lse, {B, h.heads}, at::kFloat, "lse");
        else if (want_lse)
            made_lse = make({B, h.heads}, at::kFloat, device), lse = &made_lse;
        if (B > 0) {
            size_t need = 0;
            launch("w4a8_attn_decode(query)", [&] {
                return g_attn(nullptr, type, B, h.heads, 0, 0, &cache, nullptr, max_pages, ld, nullptr, scale, window, nullptr,
                              0, 0, nullptr, nullptr, &need, nullptr);
            });
            void* const wsp = workspace_of(ws, need, made_ws, device);
            const void* qp = addr(&q, device);
            const int32_t* tp = (const int32_t*)addr(&table, device);
            void* op = addr(out, device);
            float* ep = (float*)addr(lse, device);
            const hipStream_t s = (hipStream_t)stream_of(device);
            launch("w4a8_attn_decode", [&] {
                return g_attn(qp, type, B, h.heads, h.first_stride, h.head_stride, &cache, tp, max_pages, ld, lp, scale, window,
                              op, o.first_stride, o.head_stride, ep, wsp, &need, s);
            });
        }
        PyObject* oo = given_or(a[10], made_out);
        PyObject* lo = none_or(a[11], made_lse);
        PyObject* r = oo != nullptr && lo != nullptr ? PyTuple_Pack(2, oo, lo) : nullptr;
        Py_XDECREF(oo);
        Py_XDECREF(lo);
        return r;
    });
}

}  // namespace w4a8_binding
