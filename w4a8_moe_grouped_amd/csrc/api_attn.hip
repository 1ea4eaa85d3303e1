// api_attn.hip -- the C ABI of the attention half of a served block (declared
// and documented in include/w4a8.h): the fp8 linear, rotary positions, the
// append to the paged cache and the attention over it.  Host-side only:
// validation before any HIP call, then the launch.
#include "w4a8.h"

#include "api_util.hpp"
#include "internal.hpp"

#include <math.h>

namespace {

using namespace w4a8::api;

constexpr int64_t kMaxDenseK = (int64_t)1 << 22;
constexpr int64_t kMaxTokens = (int64_t)1 << 25;
constexpr int64_t kMaxHeads = 4096;
constexpr int64_t kMaxHeadDim = 256;
constexpr int64_t kMaxSequences = 65536;
constexpr int64_t kMaxItems = (int64_t)1 << 22;  // workgroups of 512 threads in one launch
constexpr int64_t kMaxPositions = (int64_t)1 << 30;
constexpr int64_t kMaxStride = (int64_t)1 << 48;  // elements

inline bool misaligned(const void* p, uintptr_t bytes)
{
    return ((uintptr_t)p & (bytes - 1)) != 0;
}

// a stride that keeps rows 16-byte aligned (8-byte for codes)
inline bool bad_stride(int64_t s)
{
    return s < 0 || s % 8 != 0 || s > kMaxStride;
}

// rows that are written lie apart
inline bool rows_meet(int64_t n, int64_t stride)
{
    return n > 1 && stride == 0;
}

// -1: proceed
int check_rotation(int64_t T, int64_t D, int64_t R, const void* positions, const void* frequencies)
{
    if (R < 0 || R > D || R % 2 != 0 || (T > 0 && R > 0 && (positions == nullptr || frequencies == nullptr)))
        return W4A8_ERR_INVALID_ARG;
    if (D % 8 != 0 || D > kMaxHeadDim || misaligned(positions, 4) || misaligned(frequencies, 8))
        return W4A8_ERR_UNSUPPORTED;
    return -1;
}

int check_cache(const w4a8_kv_cache* c)
{
    if (c == nullptr || c->num_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->head_dim < 1 || c->k == nullptr ||
        c->v == nullptr)
        return W4A8_ERR_INVALID_ARG;
    if (c->type != W4A8_TYPE_BF16 && c->type != W4A8_TYPE_FP16 && c->type != W4A8_TYPE_E4M3)
        return W4A8_ERR_INVALID_ARG;
    const bool codes = c->type == W4A8_TYPE_E4M3;
    if ((c->k_scales != nullptr) != codes || (c->v_scales != nullptr) != codes)
        return W4A8_ERR_INVALID_ARG;
    if (c->head_dim % 8 != 0 || c->head_dim > kMaxHeadDim || c->kv_heads > kMaxHeads || c->page_size > kMaxPositions ||
        c->num_pages > INT32_MAX || mul_sat(c->num_pages, c->page_size) > ((int64_t)1 << 40))
        return W4A8_ERR_UNSUPPORTED;
    if (bad_stride(c->k_page_stride) || bad_stride(c->k_token_stride) || bad_stride(c->k_head_stride) ||
        bad_stride(c->v_page_stride) || bad_stride(c->v_token_stride) || bad_stride(c->v_head_stride))
        return W4A8_ERR_UNSUPPORTED;
    if (misaligned(c->k, codes ? 8 : 16) || misaligned(c->v, codes ? 8 : 16) || !aligned16(c->k_scales) ||
        !aligned16(c->v_scales))
        return W4A8_ERR_UNSUPPORTED;
    return -1;
}

void set_cache(const w4a8_kv_cache& c, w4a8::CacheRows& k, w4a8::CacheRows& v)
{
    k = w4a8::CacheRows{c.k, c.k_page_stride, c.k_token_stride, c.k_head_stride, c.k_scales};
    v = w4a8::CacheRows{c.v, c.v_page_stride, c.v_token_stride, c.v_head_stride, c.v_scales};
}

}  // namespace

extern "C" {

int w4a8_gemm_fp8(const uint8_t* a_e4m3, const float* a_scales, int64_t M, int64_t K,
                  const uint8_t* b_e4m3, const float* b_scales, int64_t N, const void* bias,
                  int bias_type, int activation, const void* residual_bf16, int64_t ld_residual,
                  void* out_bf16, int64_t ld_out, void* workspace, size_t* workspace_bytes,
                  hipStream_t stream)
{
    if (M < 0 || K <= 0 || N <= 0 || activation < W4A8_ACT_NONE || activation > W4A8_ACT_SWIGLU)
        return W4A8_ERR_INVALID_ARG;
    const bool glu = activation == W4A8_ACT_SWIGLU;
    const int64_t R = mul_sat(N, glu ? 2 : 1);
    if (K % W4A8_GROUP != 0 || K > kMaxDenseK || M > INT32_MAX || R > INT32_MAX || (glu && N % W4A8_GROUP != 0))
        return W4A8_ERR_UNSUPPORTED;
    // one buffer resource holds the block scales
    if (mul_sat(ceil_div(R, W4A8_GROUP), K / W4A8_GROUP * 4) > UINT32_MAX || !w4a8::gemm_fp8_fits(M, K, N, activation))
        return W4A8_ERR_UNSUPPORTED;
    const int ws_rc = check_workspace(workspace, workspace_bytes, w4a8::gemm_fp8_workspace(M, K, N, activation));
    if (ws_rc >= 0)
        return ws_rc;
    if (M > 0 && (a_e4m3 == nullptr || a_scales == nullptr || out_bf16 == nullptr))
        return W4A8_ERR_INVALID_ARG;
    if (b_e4m3 == nullptr || b_scales == nullptr || ld_out < N || (residual_bf16 != nullptr && ld_residual < N) ||
        (bias != nullptr && bias_type != W4A8_TYPE_FP32 && bias_type != W4A8_TYPE_BF16))
        return W4A8_ERR_INVALID_ARG;
    if (residual_bf16 != nullptr && residual_bf16 == out_bf16 && ld_residual != ld_out)
        return W4A8_ERR_INVALID_ARG;
    if (!aligned16(a_e4m3) || !aligned16(a_scales) || !aligned16(b_e4m3) || !aligned16(b_scales) || !aligned16(bias) ||
        !aligned16(residual_bf16) || !aligned16(out_bf16))
        return W4A8_ERR_UNSUPPORTED;
    if (M == 0)
        return W4A8_OK;
    w4a8::DenseArgs d = {};
    d.a = a_e4m3;
    d.sa = a_scales;
    d.w = b_e4m3;
    d.sw = b_scales;
    d.M = M;
    d.K = K;
    d.N = N;
    d.bias = bias;
    d.bias_bf16 = bias_type == W4A8_TYPE_BF16;
    d.act = activation;
    d.residual = (const uint16_t*)residual_bf16;
    d.ldr = ld_residual;
    d.out = (uint16_t*)out_bf16;
    d.ldo = ld_out;
    return hip_status(w4a8::launch_gemm_fp8(d, workspace, stream));
}

int w4a8_rope_frequencies(int64_t rotary_dim, double base, int scaling, double factor,
                          double original_length, double beta_fast, double beta_slow,
                          double* frequencies, hipStream_t stream)
{
    const int64_t R = rotary_dim;
    if (R < 2 || R > kMaxHeadDim || R % 2 != 0 || !(base > 1.0) || !isfinite(base) || scaling < W4A8_ROPE_PLAIN ||
        scaling > W4A8_ROPE_YARN || frequencies == nullptr)
        return W4A8_ERR_INVALID_ARG;
    if (scaling != W4A8_ROPE_PLAIN && (!(factor > 0.0) || !isfinite(factor)))
        return W4A8_ERR_INVALID_ARG;
    if (scaling == W4A8_ROPE_NTK && R == 2)
        return W4A8_ERR_INVALID_ARG;
    if (misaligned(frequencies, 8))
        return W4A8_ERR_UNSUPPORTED;
    w4a8::FrequencyArgs f = {};
    f.R = (int32_t)R;
    f.scaling = scaling;
    f.base = base;
    f.factor = factor;
    if (scaling == W4A8_ROPE_NTK) {
        f.base = base * pow(factor, (double)R / (double)(R - 2));
        f.scaling = W4A8_ROPE_PLAIN;
    } else if (scaling == W4A8_ROPE_YARN) {
        if (!(beta_slow > 0.0) || !(beta_fast >= beta_slow) || !isfinite(beta_fast) || !(original_length > 0.0) ||
            !isfinite(original_length))
            return W4A8_ERR_INVALID_ARG;
        // the (fractional) pair that turns `beta` times over the original length
        auto pair = [&](double beta) { return R * log(original_length / (6.283185307179586477 * beta)) / (2.0 * log(base)); };
        f.lo = fmax(floor(pair(beta_fast)), 0.0);
        f.hi = fmin(ceil(pair(beta_slow)), (double)(R - 1));
    }
    return hip_status(w4a8::launch_rope_frequencies(f, frequencies, stream));
}

int w4a8_rope(const void* x, int type, int64_t T, int64_t heads, int64_t head_dim,
              int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions,
              const double* frequencies, int64_t rotary_dim, int interleaved, float magnitude,
              void* out, int64_t out_token_stride, int64_t out_head_stride, hipStream_t stream)
{
    if (T < 0 || heads < 0 || head_dim < 1 || (type != W4A8_TYPE_FP32 && type != W4A8_TYPE_BF16 && type != W4A8_TYPE_FP16))
        return W4A8_ERR_INVALID_ARG;
    const bool any = T > 0 && heads > 0;
    if (any && (x == nullptr || out == nullptr))
        return W4A8_ERR_INVALID_ARG;
    if (any && x == out && (x_token_stride != out_token_stride || x_head_stride != out_head_stride))
        return W4A8_ERR_INVALID_ARG;
    if (any && (rows_meet(T, out_token_stride) || rows_meet(heads, out_head_stride)))
        return W4A8_ERR_INVALID_ARG;
    const int rc = check_rotation(any ? T : 0, head_dim, rotary_dim, positions, frequencies);
    if (rc >= 0)
        return rc;
    if (T > kMaxTokens || heads > kMaxHeads || bad_stride(x_token_stride) || bad_stride(x_head_stride) ||
        bad_stride(out_token_stride) || bad_stride(out_head_stride) || !aligned16(x) || !aligned16(out))
        return W4A8_ERR_UNSUPPORTED;
    if (!any)
        return W4A8_OK;
    w4a8::RopeArgs a = {};
    a.q = w4a8::Rows{x, x_token_stride, x_head_stride};
    a.q_out = out;
    a.qo_ts = out_token_stride;
    a.qo_hs = out_head_stride;
    a.type = type;
    a.T = T;
    a.q_heads = (int32_t)heads;
    a.D = (int32_t)head_dim;
    a.R = (int32_t)rotary_dim;
    a.interleaved = interleaved != 0;
    a.magnitude = magnitude;
    a.positions = positions;
    a.frequencies = frequencies;
    a.page_size = 1;
    if (!w4a8::rope_fits(a))
        return W4A8_ERR_UNSUPPORTED;
    return hip_status(w4a8::launch_rope(a, stream));
}

int w4a8_kv_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t q_heads,
                   const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                   int64_t v_token_stride, int64_t v_head_stride, int type, int64_t T,
                   const int64_t* slots, const int32_t* positions, const double* frequencies,
                   int64_t rotary_dim, int interleaved, float magnitude, const w4a8_kv_cache* cache,
                   void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                   hipStream_t stream)
{
    if (T < 0 || q_heads < 0 || (type != W4A8_TYPE_BF16 && type != W4A8_TYPE_FP16))
        return W4A8_ERR_INVALID_ARG;
    int rc = check_cache(cache);
    if (rc >= 0)
        return rc;
    if (cache->type != W4A8_TYPE_E4M3 && cache->type != type)
        return W4A8_ERR_INVALID_ARG;
    if ((q != nullptr) != (q_out != nullptr))
        return W4A8_ERR_INVALID_ARG;
    if (T > 0 && (k == nullptr || v == nullptr || slots == nullptr || (q == nullptr && q_heads > 0)))
        return W4A8_ERR_INVALID_ARG;
    if (q != nullptr && q == q_out && (q_token_stride != q_out_token_stride || q_head_stride != q_out_head_stride))
        return W4A8_ERR_INVALID_ARG;
    if (rows_meet(T, q_out_token_stride) && q_heads > 0)
        return W4A8_ERR_INVALID_ARG;
    if (T > 0 && rows_meet(q_heads, q_out_head_stride))
        return W4A8_ERR_INVALID_ARG;
    if (rows_meet(cache->num_pages, cache->k_page_stride) || rows_meet(cache->page_size, cache->k_token_stride) ||
        rows_meet(cache->kv_heads, cache->k_head_stride) || rows_meet(cache->num_pages, cache->v_page_stride) ||
        rows_meet(cache->page_size, cache->v_token_stride) || rows_meet(cache->kv_heads, cache->v_head_stride))
        return W4A8_ERR_INVALID_ARG;
    rc = check_rotation(T, cache->head_dim, rotary_dim, positions, frequencies);
    if (rc >= 0)
        return rc;
    if (T > kMaxTokens || q_heads > kMaxHeads || q_heads + 2 * cache->kv_heads > kMaxHeads || bad_stride(q_token_stride) ||
        bad_stride(q_head_stride) || bad_stride(k_token_stride) || bad_stride(k_head_stride) || bad_stride(v_token_stride) ||
        bad_stride(v_head_stride) || bad_stride(q_out_token_stride) || bad_stride(q_out_head_stride) || !aligned16(q) ||
        !aligned16(k) || !aligned16(v) || !aligned16(q_out) || misaligned(slots, 8))
        return W4A8_ERR_UNSUPPORTED;
    if (T == 0)
        return W4A8_OK;
    w4a8::RopeArgs a = {};
    a.q = w4a8::Rows{q, q_token_stride, q_head_stride};
    a.k = w4a8::Rows{k, k_token_stride, k_head_stride};
    a.v = w4a8::Rows{v, v_token_stride, v_head_stride};
    a.q_out = q_out;
    a.qo_ts = q_out_token_stride;
    a.qo_hs = q_out_head_stride;
    a.type = type;
    a.cache_type = cache->type;
    a.T = T;
    a.q_heads = (int32_t)q_heads;
    a.kv_heads = (int32_t)cache->kv_heads;
    a.D = (int32_t)cache->head_dim;
    a.R = (int32_t)rotary_dim;
    a.interleaved = interleaved != 0;
    a.magnitude = magnitude;
    a.positions = positions;
    a.frequencies = frequencies;
    set_cache(*cache, a.kc, a.vc);
    a.slots = slots;
    a.num_slots = cache->num_pages * cache->page_size;
    a.page_size = (int32_t)cache->page_size;
    if (!w4a8::rope_fits(a))
        return W4A8_ERR_UNSUPPORTED;
    return hip_status(w4a8::launch_rope(a, stream));
}

int w4a8_attn_decode(const void* q, int q_type, int64_t B, int64_t q_heads, int64_t q_seq_stride,
                     int64_t q_head_stride, const w4a8_kv_cache* cache, const int32_t* page_table,
                     int64_t max_pages, int64_t ld_table, const int32_t* seq_lens, float scale,
                     int64_t window, void* out, int64_t out_seq_stride, int64_t out_head_stride,
                     float* lse, void* workspace, size_t* workspace_bytes, hipStream_t stream)
{
    // the workspace depends on B, q_heads, max_pages and the cache's sizes alone
    if (B < 0 || q_heads < 1 || max_pages < 1 || cache == nullptr || cache->kv_heads < 1 || cache->page_size < 1 ||
        cache->head_dim < 1 || q_heads % cache->kv_heads != 0)
        return W4A8_ERR_INVALID_ARG;
    const int64_t D = cache->head_dim;
    if (B > kMaxSequences || q_heads > kMaxHeads || D % 8 != 0 || D > kMaxHeadDim ||
        mul_sat(max_pages, cache->page_size) > kMaxPositions ||
        mul_sat(B, cache->kv_heads * ceil_div(q_heads / cache->kv_heads, 16)) > kMaxItems)
        return W4A8_ERR_UNSUPPORTED;
    const int ws_rc = check_workspace(
        workspace, workspace_bytes,
        w4a8::attn_decode_workspace(B, q_heads, cache->kv_heads, D, max_pages * cache->page_size));
    if (ws_rc >= 0)
        return ws_rc;
    const int rc = check_cache(cache);
    if (rc >= 0)
        return rc;
    if (q_type != (cache->type == W4A8_TYPE_E4M3 ? W4A8_TYPE_BF16 : cache->type) || window < 0 || ld_table < max_pages)
        return W4A8_ERR_INVALID_ARG;
    if (rows_meet(B, out_seq_stride) || (B > 0 && rows_meet(q_heads, out_head_stride)))
        return W4A8_ERR_INVALID_ARG;
    if (B > 0 && (q == nullptr || out == nullptr || q == out || page_table == nullptr || seq_lens == nullptr))
        return W4A8_ERR_INVALID_ARG;
    if (bad_stride(q_seq_stride) || bad_stride(q_head_stride) || bad_stride(out_seq_stride) || bad_stride(out_head_stride) ||
        !aligned16(q) || !aligned16(out) || misaligned(page_table, 4) || misaligned(seq_lens, 4) || misaligned(lse, 4))
        return W4A8_ERR_UNSUPPORTED;
    if (B == 0)
        return W4A8_OK;
    w4a8::AttnArgs a = {};
    a.q = q;
    a.q_bs = q_seq_stride;
    a.q_hs = q_head_stride;
    a.q_type = q_type;
    a.cache_type = cache->type;
    a.B = (int32_t)B;
    a.q_heads = (int32_t)q_heads;
    a.kv_heads = (int32_t)cache->kv_heads;
    a.D = (int32_t)D;
    set_cache(*cache, a.kc, a.vc);
    a.num_pages = cache->num_pages;
    a.page_size = (int32_t)cache->page_size;
    a.table = page_table;
    a.ld_table = ld_table;
    a.max_pages = (int32_t)max_pages;
    a.lens = seq_lens;
    a.scale = scale;
    a.window = window;
    a.out = out;
    a.o_bs = out_seq_stride;
    a.o_hs = out_head_stride;
    a.lse = lse;
    return hip_status(w4a8::launch_attn_decode(a, workspace, stream));
}

}  // extern "C"
