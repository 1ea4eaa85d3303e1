// route.hip -- router scores to expert ids and weights (w4a8_moe_route).
//
// One wave per token.  Lane l holds the PL consecutive experts l*PL .. l*PL +
// PL - 1, so a row is one coalesced load and the lower index of equal values
// is in the lower lane, or in the lower slot of one lane.
//
// Which experts are chosen is decided by 64-bit values, since differences of
// scores that 32 bits round away still order the experts; but the search runs
// on 32-bit keys: the choice rounded to fp32 is monotone in it, so the largest
// key belongs to the largest choice unless several experts share it, and only
// then (a wave-uniform branch) are the 64-bit values compared.  Without a bias
// the logits order the scores, and the key is the logit itself.  A round of
// the search is one DPP maximum over the wave (no LDS) and one ballot per
// slot.  The scores of the chosen are evaluated once more, one per lane.
//
// Bound: instruction issue (about 300 a token with 256 experts in groups,
// 100 of them the 64-bit sigmoids), not the 4 E bytes read per token.
#include "w4a8.h"

#include "common.hpp"
#include "internal.hpp"

#include <hip/hip_fp16.h>

namespace w4a8 {

namespace {

constexpr int kRWaves = 4;  // tokens per workgroup
constexpr double kNone = -__builtin_inf();

// exp to 64 bits for z in [-800, 709]: 2^n * e^r, |r| <= ln(2)/2, by the
// Taylor sum to r^13/13! (the rest is below 4e-18)
__device__ __forceinline__ double exp64(double z)
{
    const double n = __builtin_rint(z * 1.4426950408889634);
    double r = fma(n, -0x1.62e42fefa0000p-1, z);  // ln 2 to 38 bits, exact times n
    r = fma(n, -0x1.cf79abc9e3b3ap-40, r);           // the rest of it
    double p = 1.0 / 6227020800.0;
    p = fma(p, r, 1.0 / 479001600.0);
    p = fma(p, r, 1.0 / 39916800.0);
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return __builtin_amdgcn_ldexp(p, (int)n);
}

// 1/(1 + e^-x) for any x that is not NaN; 0 where e^-x leaves the doubles
__device__ __forceinline__ double sigmoid64(float x)
{
    const double b = 1.0 + exp64(fmin(fmax(-(double)x, -800.0), 709.0));
    double y = __builtin_amdgcn_rcp(b);
    y = fma(fma(-b, y, 1.0), y, y);
    y = fma(fma(-b, y, 1.0), y, y);
    return x < -709.0f ? 0.0 : y;
}

// e^(x - top) for x <= top; 1 where they are equal, +inf included
__device__ __forceinline__ double exp_below64(float x, float top)
{
    return x == top ? 1.0 : exp64(fmax((double)x - (double)top, -800.0));
}

// floats as unsigned numbers of the same order (0 stays free for "none")
__device__ __forceinline__ uint32_t order_key(float f)
{
    const uint32_t u = __float_as_uint(f + 0.0f);  // -0 equals +0
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp0(uint32_t v)  // 0 where no lane is read
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xf, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E;             // quad_perm
constexpr int kHalfMirror = 0x141, kMirror = 0x140;   // lane i <- 7 - i of 8, 15 - i of 16

// the wave's maximum, in a scalar register
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = max(v, dpp0<0x111>(v));  // row_shr 1, 2, 4, 8
    v = max(v, dpp0<0x112>(v));
    v = max(v, dpp0<0x114>(v));
    v = max(v, dpp0<0x118>(v));
    v = max(v, dpp0<0x142>(v));  // row_bcast 15, 31
    v = max(v, dpp0<0x143>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// a value that is equal in the 2^step lanes of every aligned run, from the
// neighbouring run of that length
template <int STEP>
__device__ __forceinline__ double other_run(double v)
{
    if (STEP == 0)
        return dpp_d<kXor1>(v);
    if (STEP == 1)
        return dpp_d<kXor2>(v);
    if (STEP == 2)
        return dpp_d<kHalfMirror>(v);
    if (STEP == 3)
        return dpp_d<kMirror>(v);
    return __shfl_xor(v, 1 << STEP, 64);
}

// the two largest values of every aligned run of `lanes` lanes (a power of 2)
template <int STEP>
__device__ __forceinline__ void run_top2(double& b1, double& b2, int lanes)
{
    if ((1 << STEP) < lanes) {
        const double c1 = other_run<STEP>(b1), c2 = other_run<STEP>(b2);
        b2 = fmax(fmax(b2, c2), fmin(b1, c1));
        b1 = fmax(b1, c1);
        if constexpr (STEP < 5)
            run_top2<STEP + 1>(b1, b2, lanes);
    }
}
template <int STEP>
__device__ __forceinline__ double run_sum(double v, int lanes)
{
    if ((1 << STEP) < lanes) {
        v += other_run<STEP>(v);
        if constexpr (STEP < 5)
            v = run_sum<STEP + 1>(v, lanes);
    }
    return v;
}

__device__ __forceinline__ double read_lane(double v, int lane)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ float half_bits(uint32_t h)
{
    return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}
__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t i)
{
    if (a.type == W4A8_TYPE_FP32)
        return ((const float*)a.logits)[i];
    const uint32_t h = ((const uint16_t*)a.logits)[i];
    return a.type == W4A8_TYPE_BF16 ? __uint_as_float(h << 16) : half_bits(h);
}

// logits e0 .. e0 + PL - 1 of a row; -inf behind its end.  a.wide: every row
// starts at a multiple of 16 bytes and E % PL == 0, so a lane's run is whole.
template <int PL>
__device__ __forceinline__ void load_run(const RouteArgs& a, int64_t row, int e0, float* x)
{
    if (a.wide) {
#pragma unroll
        for (int i = 0; i < PL; ++i)
            x[i] = -__builtin_inff();
        if (e0 >= a.E)
            return;
        if (a.type == W4A8_TYPE_FP32) {
            const float* p = (const float*)a.logits + row + e0;
            if constexpr (PL >= 4) {
#pragma unroll
                for (int i = 0; i < PL; i += 4) {
                    const float4 v = *(const float4*)(p + i);
                    x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
                }
            } else if constexpr (PL == 2) {
                const float2 v = *(const float2*)p;
                x[0] = v.x, x[1] = v.y;
            } else {
                x[0] = *p;
            }
        } else {
            const uint16_t* p = (const uint16_t*)a.logits + row + e0;
            uint32_t raw[PL / 2 > 0 ? PL / 2 : 1];
            if constexpr (PL >= 8) {
#pragma unroll
                for (int i = 0; i < PL / 8; ++i) {
                    const uint4 v = *(const uint4*)(p + 8 * i);
                    raw[4 * i] = v.x, raw[4 * i + 1] = v.y, raw[4 * i + 2] = v.z, raw[4 * i + 3] = v.w;
                }
            } else if constexpr (PL == 4) {
                const uint2 v = *(const uint2*)p;
                raw[0] = v.x, raw[1] = v.y;
            } else if constexpr (PL == 2) {
                raw[0] = *(const uint32_t*)p;
            } else {
                raw[0] = *p;
            }
            const bool bf16 = a.type == W4A8_TYPE_BF16;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const uint32_t h = (i & 1) ? raw[i / 2] >> 16 : raw[i / 2] & 0xFFFFu;
                x[i] = bf16 ? __uint_as_float(h << 16) : half_bits(h);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
        x[i] = e0 + i < a.E ? load_logit(a, row + e0 + i) : -__builtin_inff();
}

}  // namespace

// SCORES: the 64-bit scores of all experts are needed (a bias, sums of two per
// group, or the softmax's whole sum); else the logits alone decide.
template <int PL, bool SCORES>
__global__ __launch_bounds__(64 * kRWaves) void route_kernel(const RouteArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kRWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
    const int e0 = lane * PL;
    float x[PL];
    load_run<PL>(a, t * a.ld, e0, x);
    uint32_t key[PL];  // of the logit, then of the choice; 0: cannot be chosen
#pragma unroll
    for (int i = 0; i < PL; ++i)
        key[i] = x[i] > -__builtin_inff() ? order_key(x[i]) : 0;  // false for NaN

    float top = 0.0f;  // largest logit of the softmax
    if (a.softmax) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < PL; ++i)
            m = max(m, key[i]);
        m = wave_max(m);
        top = __uint_as_float(m & 0x80000000u ? m ^ 0x80000000u : ~m);
    }
    double choice[PL], total = 1.0;
    if (SCORES) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            choice[i] = 0.0;
            if (key[i] != 0)
                choice[i] = a.softmax ? exp_below64(x[i], top) : sigmoid64(x[i]);
            sum += choice[i];
        }
        if (a.softmax) {
            total = run_sum<0>(sum, 64);
            const double inv = 1.0 / total;
#pragma unroll
            for (int i = 0; i < PL; ++i)
                choice[i] *= inv;
        }
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            if (a.bias != nullptr) {
                const int e = e0 + i;
                choice[i] += (double)a.bias[e < a.E ? e : a.E - 1];
            }
            if (!(choice[i] > kNone))
                key[i] = 0;
            if (key[i] == 0)
                choice[i] = kNone;
            else if (a.bias != nullptr)
                key[i] = order_key((float)choice[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < PL; ++i)
            choice[i] = key[i] != 0 ? (double)x[i] : kNone;
    }
    if (a.groups > 1) {
        // b1, b2: the two best of the lane's own group (runs), or of group
        // `lane` (any other size)
        const int size = a.E / a.groups;
        const int run = size / PL;  // lanes of a group
        double mine = kNone;
        int better = 0;
        uint64_t open = 0;  // lanes, or groups, that stay
        const bool runs = run * PL == size && (run & (run - 1)) == 0;
        if (runs) {
            double b1 = choice[0], b2 = kNone;
#pragma unroll
            for (int i = 1; i < PL; ++i) {
                b2 = fmax(b2, fmin(b1, choice[i]));
                b1 = fmax(b1, choice[i]);
            }
            run_top2<0>(b1, b2, run);
            mine = SCORES && a.group_top == 2 && b2 > kNone ? b1 + b2 : b1;
            for (int g = 0; g < a.groups; ++g) {
                const double v = read_lane(mine, g * run);
                better += (v > mine || (v == mine && lane >= (g + 1) * run)) ? 1 : 0;
            }
            open = __ballot(better < a.kept);
            if (!((open >> lane) & 1)) {
#pragma unroll
                for (int i = 0; i < PL; ++i)
                    key[i] = 0;
            }
        } else {
            for (int g = 0; g < a.groups; ++g) {
                double b1 = kNone, b2 = kNone;
#pragma unroll
                for (int i = 0; i < PL; ++i) {
                    const int e = e0 + i;
                    const double c = e >= g * size && e < (g + 1) * size ? choice[i] : kNone;
                    b2 = fmax(b2, fmin(b1, c));
                    b1 = fmax(b1, c);
                }
                run_top2<0>(b1, b2, 64);
                const double v = SCORES && a.group_top == 2 && b2 > kNone ? b1 + b2 : b1;
                if (lane == g)
                    mine = v;
            }
            for (int g = 0; g < a.groups; ++g) {
                const double v = read_lane(mine, g);
                better += (v > mine || (v == mine && g < lane)) ? 1 : 0;
            }
            open = __ballot(lane < a.groups && better < a.kept);
#pragma unroll
            for (int i = 0; i < PL; ++i)
                if (e0 + i < a.E && !((open >> ((e0 + i) / size)) & 1))
                    key[i] = 0;
        }
    }
    // the k best, one at a time
    int my_id = -1;  // lane j: the j-th
    for (int j = 0; j < a.topk; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < PL; ++i)
            m = max(m, key[i]);
        m = wave_max(m);
        if (m == 0)
            break;
        uint64_t at[PL], any = 0;
        int count = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            at[i] = __ballot(key[i] == m);
            any |= at[i];
            count += __popcll(at[i]);
        }
        if (SCORES && count > 1 && a.bias != nullptr) {  // 32 bits do not tell
            double best = kNone;
#pragma unroll
            for (int i = 0; i < PL; ++i)
                best = key[i] == m ? fmax(best, choice[i]) : best;
#pragma unroll
            for (int o = 32; o > 0; o >>= 1)
                best = fmax(best, __shfl_xor(best, o, 64));
            any = 0;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                at[i] = __ballot(key[i] == m && choice[i] == best);
                any |= at[i];
            }
        }
        const int win = __ffsll((unsigned long long)any) - 1;
        int slot = PL - 1;
#pragma unroll
        for (int i = PL - 2; i >= 0; --i)
            slot = (at[i] >> win) & 1 ? i : slot;
        const bool here = lane == win;
#pragma unroll
        for (int i = 0; i < PL; ++i)
            key[i] = here && slot == i ? 0 : key[i];
        my_id = lane == j ? win * PL + slot : my_id;
    }
    // scores of the chosen, one per lane
    double s = 0.0;
    if (my_id >= 0) {
        const float v = load_logit(a, t * a.ld + my_id);
        s = a.softmax ? exp_below64(v, top) : sigmoid64(v);
    }
    if (a.renorm) {
        const double sum = run_sum<0>(s, a.topk);
        s = sum > 0.0 ? s / sum : 0.0;
    } else if (a.softmax) {
        s = s / total;
    }
    if (lane < a.topk) {
        ids[lane] = my_id;
        wts[lane] = (float)((double)a.scale * s);
    }
}

namespace {

template <int PL>
void launch_lanes(const RouteArgs& a, bool scores, hipStream_t s)
{
    const dim3 grid((unsigned)((a.T + kRWaves - 1) / kRWaves)), block(64 * kRWaves);
    RouteArgs b = a;
    const int elem = a.type == W4A8_TYPE_FP32 ? 4 : 2;
    b.wide = (a.ld * elem) % 16 == 0 && a.E % PL == 0;
    if (scores)
        hipLaunchKernelGGL((route_kernel<PL, true>), grid, block, 0, s, b);
    else
        hipLaunchKernelGGL((route_kernel<PL, false>), grid, block, 0, s, b);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s)
{
    const bool scores =
        a.bias != nullptr || (a.groups > 1 && a.group_top == 2) || (a.softmax && !a.renorm);
    if (a.E <= 64)
        launch_lanes<1>(a, scores, s);
    else if (a.E <= 128)
        launch_lanes<2>(a, scores, s);
    else if (a.E <= 256)
        launch_lanes<4>(a, scores, s);
    else if (a.E <= 512)
        launch_lanes<8>(a, scores, s);
    else
        launch_lanes<16>(a, scores, s);
    return hipGetLastError();
}

}  // namespace w4a8
