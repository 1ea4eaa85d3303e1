// route.hip -- router scores to expert ids and weights (w4a8_moe_route).
//
// One wave per token.  Lane l holds the PL consecutive experts l*PL .. l*PL +
// PL - 1, so a row is one coalesced load and the lower index of equal values
// is in the lower lane.  Which experts are chosen is decided by 64-bit
// values: differences of scores that 32 bits would round away still order
// the experts.
#include "w4a8.h"

#include "common.hpp"
#include "internal.hpp"

#include <hip/hip_fp16.h>

namespace w4a8 {

namespace {

constexpr int kRWaves = 4;  // tokens per workgroup

__device__ __forceinline__ double neg_inf()
{
    return -__builtin_inf();
}

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t t, int e)
{
    const int64_t i = t * a.ld + e;
    if (a.type == W4A8_TYPE_FP32)
        return ((const float*)a.logits)[i];
    if (a.type == W4A8_TYPE_BF16)
        return bf16_to_f32(((const uint16_t*)a.logits)[i]);
    return __half2float(((const __half*)a.logits)[i]);
}

__device__ __forceinline__ double shfl_xor_d(double v, int o)
{
    return __shfl_xor(v, o, 64);
}

}  // namespace

template <int PL>
__global__ __launch_bounds__(64 * kRWaves) void route_kernel(const RouteArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kRWaves + (threadIdx.x >> 6);
    if (t >= a.T)
        return;
    int32_t* const ids = a.ids + t * a.topk;
    float* const wts = a.weights + t * a.topk;
    if (a.num_tokens != nullptr && t >= *a.num_tokens) {
        if (lane < a.topk) {
            ids[lane] = -1;
            wts[lane] = 0.0f;
        }
        return;
    }
    // scores; `choice` is -inf where the expert cannot be chosen
    float x[PL];
    bool ok[PL];
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int e = lane * PL + i;
        x[i] = e < a.E ? load_logit(a, t, e) : -__builtin_inff();
        ok[i] = x[i] > -__builtin_inff();  // false for NaN too
        if (ok[i])
            top = fmaxf(top, x[i]);
    }
    top = group_max<64>(top);
    double score[PL], choice[PL], total = 0.0;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        if (a.softmax) {
            score[i] = ok[i] ? (x[i] == top ? 1.0 : exp((double)x[i] - (double)top)) : 0.0;
            total += score[i];
        } else {
            score[i] = ok[i] ? 1.0 / (1.0 + exp(-(double)x[i])) : 0.0;
        }
    }
    if (a.softmax) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1)
            total += shfl_xor_d(total, o);
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        if (a.softmax && ok[i])
            score[i] /= total;
        const int e = lane * PL + i;
        double c = score[i];
        if (a.bias != nullptr && e < a.E)
            c += (double)a.bias[e];
        choice[i] = ok[i] && c > neg_inf() ? c : neg_inf();
    }
    // without a bias the logits order the scores, also where 64 bits round
    // two of them alike; the sums of two are of the scores
    if (a.bias == nullptr && (a.groups == 1 || a.group_top == 1)) {
#pragma unroll
        for (int i = 0; i < PL; ++i)
            choice[i] = ok[i] ? (double)x[i] : neg_inf();
    }
    // groups: value of each, then the rank of each among them
    if (a.groups > 1) {
        const int size = a.E / a.groups;
        uint64_t open = 0;  // groups that stay
        double mine = neg_inf();  // lane g: the value of group g
        for (int g = 0; g < a.groups; ++g) {
            double b1 = neg_inf(), b2 = neg_inf();
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const int e = lane * PL + i;
                const double c = e >= g * size && e < (g + 1) * size ? choice[i] : neg_inf();
                b2 = fmax(b2, fmin(b1, c));
                b1 = fmax(b1, c);
            }
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) {
                const double c1 = shfl_xor_d(b1, o), c2 = shfl_xor_d(b2, o);
                b2 = fmax(fmax(b2, c2), fmin(b1, c1));
                b1 = fmax(b1, c1);
            }
            const double v = a.group_top == 2 && b2 > neg_inf() ? b1 + b2 : b1;
            if (lane == g)
                mine = v;
        }
        int better = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double v = __shfl(mine, g, 64);
            better += (v > mine || (v == mine && g < lane)) ? 1 : 0;
        }
        open = __ballot(lane < a.groups && better < a.kept);
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int e = lane * PL + i;
            if (e < a.E && !((open >> (e / size)) & 1))
                choice[i] = neg_inf();
            else if (a.bias == nullptr && ok[i])
                choice[i] = (double)x[i];
        }
    }
    // the k best, one at a time
    int my_id = -1;
    double my_score = 0.0;
    for (int j = 0; j < a.topk; ++j) {
        double best = choice[0];
#pragma unroll
        for (int i = 1; i < PL; ++i)
            best = fmax(best, choice[i]);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1)
            best = fmax(best, shfl_xor_d(best, o));
        if (!(best > neg_inf()))
            break;
        int at = PL;  // this lane's first slot that holds it
#pragma unroll
        for (int i = PL - 1; i >= 0; --i)
            at = choice[i] == best ? i : at;
        const int win = __ffsll((unsigned long long)__ballot(at < PL)) - 1;
        const int slot = __shfl(at, win, 64);
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            s = i == slot ? score[i] : s;
            if (lane == win && i == slot)
                choice[i] = neg_inf();
        }
        s = __shfl(s, win, 64);
        if (lane == j) {
            my_id = win * PL + slot;
            my_score = s;
        }
    }
    if (a.renorm) {
        double sum = my_score;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1)
            sum += shfl_xor_d(sum, o);
        my_score = sum > 0.0 ? my_score / sum : 0.0;
    }
    if (lane < a.topk) {
        ids[lane] = my_id;
        wts[lane] = (float)((double)a.scale * my_score);
    }
}

hipError_t launch_route(const RouteArgs& a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.T + kRWaves - 1) / kRWaves)), block(64 * kRWaves);
    if (a.E <= 64)
        hipLaunchKernelGGL(route_kernel<1>, grid, block, 0, s, a);
    else if (a.E <= 128)
        hipLaunchKernelGGL(route_kernel<2>, grid, block, 0, s, a);
    else if (a.E <= 256)
        hipLaunchKernelGGL(route_kernel<4>, grid, block, 0, s, a);
    else if (a.E <= 512)
        hipLaunchKernelGGL(route_kernel<8>, grid, block, 0, s, a);
    else
        hipLaunchKernelGGL(route_kernel<16>, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace w4a8
