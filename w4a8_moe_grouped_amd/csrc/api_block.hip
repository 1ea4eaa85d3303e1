// api_block.hip -- the C ABI of the operators around the expert forward
// (declared and documented in include/w4a8.h): the router, the norms between
// two blocks and the dense linear with an epilogue.  Host-side only:
// validation before any HIP call, then the launch.
#include "w4a8.h"

#include "api_util.hpp"
#include "internal.hpp"

#include <float.h>

namespace {

using namespace w4a8::api;

constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxGroups = 64;
constexpr int64_t kMaxDenseK = (int64_t)1 << 22;
// a launch holds less than 2^32 threads: up to 64 a token, a short row; 1024 a row
constexpr int64_t kMaxTokens = (int64_t)1 << 25;
constexpr int64_t kMaxLongRows = ((int64_t)1 << 22) - 1;

inline bool float_or_bf16(int type)
{
    return type == W4A8_TYPE_FP32 || type == W4A8_TYPE_BF16;
}

}  // namespace

extern "C" {

int w4a8_moe_route(const void* logits, int logits_type, int64_t T, int64_t E, int64_t ld_logits,
                   const float* bias, int score, int64_t num_groups, int64_t topk_groups,
                   int group_top, int64_t topk, int renormalize, float scale,
                   const int32_t* num_tokens, int32_t* topk_ids, float* topk_weights,
                   hipStream_t stream)
{
    if (T < 0 || E < 1 || ld_logits < E || topk < 1 || num_groups < 1 || topk_groups < 1 ||
        topk_groups > num_groups || E % num_groups != 0 || topk > mul_sat(topk_groups, E / num_groups))
        return W4A8_ERR_INVALID_ARG;
    if ((logits_type != W4A8_TYPE_FP32 && logits_type != W4A8_TYPE_BF16 && logits_type != W4A8_TYPE_FP16) ||
        (score != W4A8_SCORE_SIGMOID && score != W4A8_SCORE_SOFTMAX) || (group_top != 1 && group_top != 2))
        return W4A8_ERR_INVALID_ARG;
    if (topk > W4A8_MAX_TOPK || E > kMaxExperts || num_groups > kMaxGroups || T > kMaxTokens)
        return W4A8_ERR_UNSUPPORTED;
    if (T > 0 && (logits == nullptr || topk_ids == nullptr || topk_weights == nullptr))
        return W4A8_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(bias) || !aligned16(topk_ids) || !aligned16(topk_weights) ||
        ((uintptr_t)num_tokens & 3u) != 0)
        return W4A8_ERR_UNSUPPORTED;
    if (T == 0)
        return W4A8_OK;
    w4a8::RouteArgs a = {};
    a.logits = logits;
    a.type = logits_type;
    a.T = T;
    a.ld = ld_logits;
    a.E = (int32_t)E;
    a.bias = bias;
    a.softmax = score == W4A8_SCORE_SOFTMAX;
    a.groups = (int32_t)num_groups;
    a.kept = (int32_t)topk_groups;
    a.group_top = group_top;
    a.topk = (int32_t)topk;
    a.renorm = renormalize != 0;
    a.scale = scale;
    a.num_tokens = num_tokens;
    a.ids = topk_ids;
    a.weights = topk_weights;
    return hip_status(w4a8::launch_route(a, stream));
}

int w4a8_norm_residual(const void* x, int x_type, int64_t ldx, const void* residual,
                       int residual_type, int64_t ldr, int64_t T, int64_t H, int param_type,
                       const void* post_weight, const void* gate, int64_t gate_row_stride,
                       int64_t gate_col_stride, float residual_scale, const void* pre_weight,
                       float weight_offset, float eps, void* residual_out, int64_t ldr_out,
                       void* y_bf16, int64_t ldy, uint8_t* q_e4m3, float* q_scales,
                       hipStream_t stream)
{
    if (T < 0 || H <= 0 || !(eps >= FLT_MIN) || !float_or_bf16(x_type) || !float_or_bf16(residual_type) ||
        !float_or_bf16(param_type))
        return W4A8_ERR_INVALID_ARG;
    const bool want_y = y_bf16 != nullptr || q_e4m3 != nullptr;
    if ((q_e4m3 == nullptr) != (q_scales == nullptr))
        return W4A8_ERR_INVALID_ARG;
    if (T > 0 && ((x == nullptr && residual == nullptr) || (pre_weight != nullptr) != want_y ||
                  (!want_y && residual_out == nullptr)))
        return W4A8_ERR_INVALID_ARG;
    if (T > 0 && x == nullptr && (post_weight != nullptr || gate != nullptr))
        return W4A8_ERR_INVALID_ARG;
    if ((x != nullptr && ldx < H) || (residual != nullptr && ldr < H) ||
        (residual_out != nullptr && ldr_out < H) || (y_bf16 != nullptr && ldy < H))
        return W4A8_ERR_INVALID_ARG;
    if (gate != nullptr && ((gate_col_stride != 0 && gate_col_stride != 1) || gate_row_stride < 0 ||
                            (gate_row_stride != 0 && gate_row_stride < (gate_col_stride == 1 ? H : 1))))
        return W4A8_ERR_INVALID_ARG;
    if (residual_out != nullptr && residual_out == residual && ldr_out != ldr)
        return W4A8_ERR_INVALID_ARG;
    if (H > w4a8::kNormMaxH || T > (H <= w4a8::kNormShortH ? kMaxTokens : kMaxLongRows) || (q_e4m3 != nullptr && H % W4A8_GROUP != 0))
        return W4A8_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(post_weight) || !aligned16(gate) ||
        !aligned16(pre_weight) || !aligned16(residual_out) || !aligned16(y_bf16) || !aligned16(q_e4m3) ||
        !aligned16(q_scales))
        return W4A8_ERR_UNSUPPORTED;
    if (T == 0)
        return W4A8_OK;
    w4a8::NormArgs a = {};
    a.x = x;
    a.residual = residual;
    a.x_type = x_type;
    a.r_type = residual_type;
    a.p_type = param_type;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldr_out = ldr_out;
    a.ldy = ldy;
    a.T = T;
    a.H = (int32_t)H;
    a.post_w = post_weight;
    a.gate = gate;
    a.gate_rs = gate_row_stride;
    a.gate_cs = gate_col_stride;
    a.r_scale = residual_scale;
    a.pre_w = pre_weight;
    a.w_offset = weight_offset;
    a.eps = eps;
    a.r_out = residual_out;
    a.y = (uint16_t*)y_bf16;
    a.q = q_e4m3;
    a.q_scales = q_scales;
    return hip_status(w4a8::launch_norm(a, stream));
}

int w4a8_gemm_epilogue(const uint8_t* a_e4m3, const float* a_scales, int64_t M, int64_t K,
                       const uint8_t* b_int4, const float* b_scales, int64_t N, const void* bias,
                       int bias_type, int activation, const void* residual_bf16,
                       int64_t ld_residual, void* out_bf16, int64_t ld_out, void* workspace,
                       size_t* workspace_bytes, hipStream_t stream)
{
    if (M < 0 || K <= 0 || N <= 0 || activation < W4A8_ACT_NONE || activation > W4A8_ACT_SWIGLU)
        return W4A8_ERR_INVALID_ARG;
    if (K % W4A8_GROUP != 0 || K > kMaxDenseK || M > INT32_MAX ||
        mul_sat(N, activation == W4A8_ACT_SWIGLU ? 2 : 1) > INT32_MAX)
        return W4A8_ERR_UNSUPPORTED;
    if (mul_sat(ceil_div(M, 32), ceil_div(N, 16)) > INT32_MAX || !w4a8::dense_epilogue_fits(M, K, N, activation))
        return W4A8_ERR_UNSUPPORTED;
    const size_t need = w4a8::dense_epilogue_workspace(M, K, N, activation);
    const int ws_rc = check_workspace(workspace, workspace_bytes, need);
    if (ws_rc >= 0)
        return ws_rc;
    if (M > 0 && (a_e4m3 == nullptr || a_scales == nullptr || out_bf16 == nullptr))
        return W4A8_ERR_INVALID_ARG;
    if (b_int4 == nullptr || b_scales == nullptr || ld_out < N ||
        (residual_bf16 != nullptr && ld_residual < N) || (bias != nullptr && !float_or_bf16(bias_type)))
        return W4A8_ERR_INVALID_ARG;
    if (residual_bf16 != nullptr && residual_bf16 == out_bf16 && ld_residual != ld_out)
        return W4A8_ERR_INVALID_ARG;
    if (!aligned16(a_e4m3) || !aligned16(a_scales) || !aligned16(b_int4) || !aligned16(b_scales) ||
        !aligned16(bias) || !aligned16(residual_bf16) || !aligned16(out_bf16))
        return W4A8_ERR_UNSUPPORTED;
    if (M == 0)
        return W4A8_OK;
    w4a8::DenseArgs d = {};
    d.a = a_e4m3;
    d.sa = a_scales;
    d.w = b_int4;
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
    return hip_status(w4a8::launch_dense_epilogue(d, workspace, stream));
}

}  // extern "C"
