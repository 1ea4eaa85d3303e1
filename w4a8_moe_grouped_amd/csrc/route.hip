// route.hip -- router scores to expert ids and weights (w4a8_moe_route):
//   s = sigmoid(x) or softmax(x),  c = s + bias,  groups by the sum of their two
//   best c,  the k best c of the groups kept,  weights scale * s / sum of s.
//
// Which experts are chosen, and in which order, is decided by 64-bit values,
// since differences of scores that 32 bits round away still order the
// experts.  But few tokens need that many bits, so the search runs in 32: the
// fast kernel (route_rows_kernel, four tokens per wave) bounds the error of its
// choices and hands the tokens it cannot decide to the exact one (route_token,
// one token per wave, also for more experts or groups than fit 16 lanes).
// There, too, the search runs on 32-bit keys: the choice rounded to fp32 is
// monotone in it, so the largest key belongs to the largest choice unless
// several experts share it, and only then (a wave-uniform branch) are the
// 64-bit values compared.  Without a bias the logits order the scores, and the
// key is the logit itself.  The scores of the chosen are evaluated once more in
// 64 bits, one per lane, and rounded once.
//
// In the exact kernel lane l holds the PL consecutive experts l*PL .. l*PL + PL
// - 1, so a row is one coalesced load and the lower index of equal values is in
// the lower lane, or in the lower slot of one lane; a round of the search is a
// DPP maximum over the wave (no LDS) and one ballot per slot.
//
// Bound: instruction issue.  32768 tokens, 256 experts in 8 groups, top 8,
// sigmoid and bias: 20 us, 1.8 TB/s of logits; 195 vector operations a token
// (780 per wave of four), which alone are 10.5 us of every SIMD; the exact kernel
// takes 52 us.  How many waves a CU holds does not matter (12 to 24: 20.4 to
// 22.8 us), nor does loading the next tokens ahead.  64 tokens: 5 us, all
// latency.
#include "w4a8.h"

#include "common.hpp"
#include "internal.hpp"

#include <hip/hip_fp16.h>

namespace w4a8 {

namespace {

constexpr int kRWaves = 4;  // tokens per workgroup
constexpr double kNone = -__builtin_inf();

// A constant in scalar registers: a 64-bit fma takes one such operand, where a
// literal would first be moved into a pair of vector registers.
__device__ __forceinline__ double in_sgprs(double c)
{
    asm("" : "+s"(c));
    return c;
}

// exp to 64 bits for z in [-800, 709]: 2^n * e^r, |r| <= ln(2)/2, by the
// Taylor sum to r^13/13! (the rest is below 4.3e-18)
__device__ __forceinline__ double exp64(double z)
{
    const double n = __builtin_rint(z * in_sgprs(1.4426950408889634));
    double r = fma(n, in_sgprs(-0x1.62e42fefa0000p-1), z);  // ln 2 to 38 bits, exact times n
    r = fma(n, in_sgprs(-0x1.cf79abc9e3b3ap-40), r);        // the rest of it
    double p = in_sgprs(1.0 / 6227020800.0);
    p = fma(p, r, in_sgprs(1.0 / 479001600.0));
    p = fma(p, r, in_sgprs(1.0 / 39916800.0));
    p = fma(p, r, in_sgprs(1.0 / 3628800.0));
    p = fma(p, r, in_sgprs(1.0 / 362880.0));
    p = fma(p, r, in_sgprs(1.0 / 40320.0));
    p = fma(p, r, in_sgprs(1.0 / 5040.0));
    p = fma(p, r, in_sgprs(1.0 / 720.0));
    p = fma(p, r, in_sgprs(1.0 / 120.0));
    p = fma(p, r, in_sgprs(1.0 / 24.0));
    p = fma(p, r, in_sgprs(1.0 / 6.0));
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

// floats as unsigned numbers of the same order; -inf (0x007FFFFF) and 0 below
// every number
__device__ __forceinline__ uint32_t order_bits(float f)  // f is not -0
{
    const uint32_t u = __float_as_uint(f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t order_key(float f)
{
    return order_bits(f + 0.0f);  // -0 equals +0
}
constexpr uint32_t kNoKey = 0x007FFFFFu;

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

// wide accesses at the alignment of an element, which are one instruction also
// where they are misaligned (32768 x 256 in rows of 257: 18 us, element by
// element 26; 32768 x 250 of bf16: 11.4 and 21)
typedef float float4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef float float2_any __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t uint4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t uint2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t uint1_any __attribute__((aligned(2)));

// logits e0 .. e0 + count - 1 of a row, then -inf; a lane whose PL logits all lie
// in the row reads them at once, whose ever they are (E: the row's length)
template <int PL>
__device__ __forceinline__ void load_run(const RouteArgs& a, int64_t row, int e0, int count, float* x)
{
    const bool inside = count > 0 && e0 + PL <= a.E;
    auto cut = [&] {
        if (count < PL) {
#pragma unroll
            for (int i = 0; i < PL; ++i)
                x[i] = i < count ? x[i] : -__builtin_inff();
        }
    };
#pragma unroll
    for (int i = 0; i < PL; ++i)
        x[i] = -__builtin_inff();
    if (a.type == W4A8_TYPE_FP32) {
        const float* p = (const float*)a.logits + row + e0;
        if (!inside) {
#pragma unroll
            for (int i = 0; i < PL; ++i)
                if (i < count)
                    x[i] = p[i];
        } else {
            if constexpr (PL >= 4) {
#pragma unroll
                for (int i = 0; i < PL; i += 4) {
                    const float4_any v = *(const float4_any*)(p + i);
                    x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
                }
            } else if constexpr (PL == 2) {
                const float2_any v = *(const float2_any*)p;
                x[0] = v.x, x[1] = v.y;
            } else {
                x[0] = *p;
            }
            cut();
        }
        return;
    }
    constexpr uint32_t kLow = 0xFF80FC00u;  // -inf: bf16 in the high half, fp16 in the low one
    const uint32_t none = a.type == W4A8_TYPE_BF16 ? kLow >> 16 : kLow & 0xFFFFu;
    uint32_t raw[(PL + 1) / 2];
#pragma unroll
    for (int i = 0; i < (PL + 1) / 2; ++i)
        raw[i] = none | none << 16;
    const uint16_t* p = (const uint16_t*)a.logits + row + e0;
    if (!inside) {
#pragma unroll
        for (int i = 0; i < PL; ++i)
            if (i < count)
                raw[i / 2] = (i & 1) ? (raw[i / 2] & 0xFFFFu) | (uint32_t)p[i] << 16
                                     : (raw[i / 2] & 0xFFFF0000u) | p[i];
    } else {
        if constexpr (PL >= 8) {
#pragma unroll
            for (int i = 0; i < PL / 8; ++i) {
                const uint4_any v = *(const uint4_any*)(p + 8 * i);
                raw[4 * i] = v.x, raw[4 * i + 1] = v.y, raw[4 * i + 2] = v.z, raw[4 * i + 3] = v.w;
            }
        } else if constexpr (PL == 4) {
            const uint2_any v = *(const uint2_any*)p;
            raw[0] = v.x, raw[1] = v.y;
        } else if constexpr (PL == 2) {
            raw[0] = *(const uint1_any*)p;
        } else {
            raw[0] = *p;
        }
    }
    if (a.type == W4A8_TYPE_BF16) {
#pragma unroll
        for (int i = 0; i < PL; ++i)
            x[i] = __uint_as_float((i & 1) ? raw[i / 2] & 0xFFFF0000u : raw[i / 2] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < PL; ++i)
            x[i] = half_bits((i & 1) ? raw[i / 2] >> 16 : raw[i / 2] & 0xFFFFu);
    }
    cut();
}

}  // namespace

// SCORES: the 64-bit scores of all experts are needed (a bias, sums of two per
// group, or the softmax's whole sum); else the logits alone decide.
template <int PL, bool SCORES>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t)
{
    const int lane = threadIdx.x & 63;
    int32_t* const ids = a.ids + t * a.topk;
    float* const wts = a.weights + t * a.topk;
    const int e0 = lane * PL;
    float x[PL];
    load_run<PL>(a, t * a.ld, e0, min(a.E - e0, PL), x);
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
            else if (a.group_top == 1)
                choice[i] = (double)x[i];  // groups too go by the logits
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
    } else if (a.softmax && my_id >= 0) {
        s = s / total;
    }
    if (lane < a.topk) {
        ids[lane] = my_id;
        wts[lane] = (float)((double)a.scale * s);
    }
}

template <int PL, bool SCORES>
__global__ __launch_bounds__(64 * kRWaves) void route_kernel(const RouteArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kRWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= a.T)
        return;
    if (a.num_tokens != nullptr && t >= *a.num_tokens) {
        if (lane < a.topk) {
            a.ids[t * a.topk + lane] = -1;
            a.weights[t * a.topk + lane] = 0.0f;
        }
        return;
    }
    route_token<PL, SCORES>(a, t);
}

// ---- four tokens per wave ------------------------------------------------------------
//
// 16 lanes per token, up to PL consecutive experts each; the lanes of a group
// are a run of 1, 2, 4, 8 or 16, whatever its size.  The search runs on keys
// of 32 bits that carry the expert's slot in their low bits, so each lane
// sorts its own with a plain min/max network, and a round is a DPP maximum
// over the row of 16 lanes that leaves the result in all of them; scores are
// fp32.  That decides every token whose neighbouring choices differ by more
// than both can be off.  Closer ones are put in order by their 64-bit values,
// which the weights need anyway; where even these leave open which experts are
// chosen, or a group's place is too close to tell, route_token does the token
// again, the whole wave on it (8192 tokens, 440 experts, a bias: 12 us; with
// every disorder done again 18).

namespace {


template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v)
{
    return __uint_as_float(dpp_u<CTRL>(__float_as_uint(v)));
}
constexpr int kRor = 0x120;  // row_ror by n: kRor + n

// the row's maximum in all its lanes
__device__ __forceinline__ uint32_t row_max(uint32_t v)
{
    v = max(v, dpp_u<kRor + 1>(v));
    v = max(v, dpp_u<kRor + 2>(v));
    v = max(v, dpp_u<kRor + 4>(v));
    return max(v, dpp_u<kRor + 8>(v));
}
__device__ __forceinline__ float row_sum16(float v)
{
    v += dpp_f<kRor + 1>(v);
    v += dpp_f<kRor + 2>(v);
    v += dpp_f<kRor + 4>(v);
    return v + dpp_f<kRor + 8>(v);
}
__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// descending, by odd-even merges
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&v)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t hi = max(v[i + j], v[i + j + k]);
                        v[i + j + k] = min(v[i + j], v[i + j + k]);
                        v[i + j] = hi;
                    }
}

// What orders the experts: their choice in fp32 (with a bias), or their logits
// (without), exactly for the 16-bit types, whose keys hold the index too (they
// leave the low 13 or 16 bits of a float free).
enum RowKey { KEY_CHOICE, KEY_LOGIT32, KEY_LOGIT16 };

// Rounds J .. topk - 1 of the search, unrolled (a loop left rolled indexes the
// keys at run time: 2.5 us a round): lane J of each row gets the row's largest
// key and the lane that held it, and this moves on to its next.
template <int J, int KM, int KEY, int PL>
__device__ __forceinline__ void take_best(uint32_t (&key)[PL], int topk, int l, uint32_t& mine, uint32_t& lanes_lo,
                                          uint32_t& lanes_hi)
{
    if constexpr (J < KM) {
        if (J == topk)
            return;
        const uint32_t m = row_max(key[0]);
        bool won = key[0] == m;
        uint64_t lanes = __ballot(won);
        // every row has a winner, so no difference borrows from its neighbour
        if (KEY != KEY_LOGIT16 && (lanes & (lanes - 0x0001000100010001ull)) != 0) {  // one key in several lanes
            won = won && ((lanes >> (threadIdx.x & 48)) & ((1u << l) - 1)) == 0;     // the lowest first
            lanes = __ballot(won);
        }
        mine = l == J ? m : mine;
        lanes_lo = l == J ? (uint32_t)lanes : lanes_lo;
        lanes_hi = l == J ? (uint32_t)(lanes >> 32) : lanes_hi;
        // as far as later rounds, and the one behind them, can ask for them
#pragma unroll
        for (int i = 0; i <= KM - J && i < PL; ++i)
            key[i] = won ? (i + 1 < PL ? key[i + 1] : 0) : key[i];
        take_best<J + 1, KM, KEY>(key, topk, l, mine, lanes_lo, lanes_hi);
    }
}

// how many lanes of the row come before this one by value, then index
template <int N>
__device__ __forceinline__ int count_ahead(double value, int id)
{
    if constexpr (N < 16) {
        const double v = dpp_d<kRor + N>(value);
        const int i = (int)dpp_u<kRor + N>((uint32_t)id);
        return ((v > value || (v == value && i < id)) ? 1 : 0) + count_ahead<N + 1>(value, id);
    } else {
        return 0;
    }
}

// other groups of the row, one rotation after another (lane l reads l - N, a
// lower group unless that wraps): how many are better than this lane's, and
// whether any is too close to tell
template <int N>
__device__ __forceinline__ void rank_groups(float mine, int l, int run, float slack, int& better, bool& close)
{
    if constexpr (N < 16) {
        if ((N & (run - 1)) == 0) {
            const float v = dpp_f<kRor + N>(mine);
            better += (v > mine || (v == mine && l >= N)) ? 1 : 0;
            close |= fabsf(v - mine) <= slack;  // false for two equal infinities
        }
        rank_groups<N + 1>(mine, l, run, slack, better, close);
    }
}

}  // namespace

template <int PL, int KEY, int KM>  // KM: most experts per token, 8 or 16
__global__ __launch_bounds__(256) void route_rows_kernel(const RouteArgs a)
{
    constexpr uint32_t kSlots = PL <= 16 ? 15 : 31;       // low bits of a key: kSlots - slot
    constexpr uint32_t kIndexes = PL <= 16 ? 0xFF : 0x1FF;  // of KEY_LOGIT16: kIndexes - index
    const float ninf = -__builtin_inff();
    const int lane = threadIdx.x & 63, l = lane & 15;
    const int waves = (int)blockDim.x >> 6;
    const int64_t t0 =
        ((int64_t)blockIdx.x * waves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 4;
    if (t0 >= a.T)
        return;
    int64_t valid = a.T;  // rows from here on are padding
    if (a.num_tokens != nullptr)
        valid = min(valid, (int64_t)*a.num_tokens);
    const int64_t t = t0 + (lane >> 4);
    const bool live = t < valid;
    const int64_t row = (live ? t : t0) * a.ld;

    const int size = a.E / a.groups, run = 1 << a.run_log2;
    auto first_of = [&](int w) { return (w >> a.run_log2) * size + (w & (run - 1)) * a.per; };
    const int e0 = first_of(l);
    const int count = l >> a.run_log2 < a.groups ? min(size - (l & (run - 1)) * a.per, a.per) : 0;
    float x[PL];
    if (live) {
        load_run<PL>(a, row, e0, count, x);
    } else {
#pragma unroll
        for (int i = 0; i < PL; ++i)
            x[i] = ninf;
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
        x[i] = fmaxf(x[i], ninf);  // NaN: -inf, which is what cannot be chosen
    float top = ninf;
    double total = 1.0;  // of the softmax, where the weights need it
    if (a.softmax) {
#pragma unroll
        for (int i = 0; i < PL; ++i)
            top = fmaxf(top, x[i]);
        top = fmaxf(top, dpp_f<kRor + 1>(top));
        top = fmaxf(top, dpp_f<kRor + 2>(top));
        top = fmaxf(top, dpp_f<kRor + 4>(top));
        top = fmaxf(top, dpp_f<kRor + 8>(top));
        if (!a.renorm) {
            total = 0.0;
#pragma unroll
            for (int i = 0; i < PL; ++i)
                total += x[i] > ninf ? exp_below64(x[i], top) : 0.0;
            total = run_sum<0>(total, 16);
        }
    }
    // choices in fp32, off by at most `off` + 2^-23 of their value: the
    // sigmoid's product, exp2, sum and reciprocal cost 2^-22 (kept: 2^-21), the
    // softmax's sum of up to 20 (PL 32: 36) roundings 2^-19.7 (2^-18.8) of its
    // terms, the largest of which is 1 / sum (kept: 2^-19, 2^-18 of that)
    const bool sums = a.groups > 1 && a.group_top == 2;
    float off = 0x1p-21f;
    uint32_t key[PL], gkey[PL];  // of the experts' order, and of the groups'
    if (KEY == KEY_CHOICE || sums) {
        float c[PL];
        if (a.softmax) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                c[i] = x[i] == top ? 1.0f : __builtin_amdgcn_exp2f((x[i] - top) * 1.44269504f);
                sum += c[i];
            }
            const float inv = __builtin_amdgcn_rcpf(row_sum16(sum));
            off = (PL <= 16 ? 0x1p-19f : 0x1p-18f) * inv;
#pragma unroll
            for (int i = 0; i < PL; ++i)
                c[i] *= inv;
        } else {
#pragma unroll
            for (int i = 0; i < PL; ++i)
                c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x[i] * -1.44269504f));
        }
        float b[PL];  // small enough for the L1; loaded here to hold fewer registers
        if (KEY == KEY_CHOICE) {
#pragma unroll
            for (int i = 0; i < PL; ++i)
                b[i] = 0.0f;
            if (count > 0 && e0 + PL <= a.E) {
#pragma unroll
                for (int i = 0; i < PL; i += 4) {
                    const float4_any v = *(const float4_any*)(a.bias + e0 + i);
                    b[i] = v.x, b[i + 1] = v.y, b[i + 2] = v.z, b[i + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < PL; ++i)
                    if (i < count)
                        b[i] = a.bias[e0 + i];
            }
        }
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            if (KEY == KEY_CHOICE)
                c[i] = fmaxf(c[i] + b[i], ninf);  // a NaN bias: -inf
            gkey[i] = x[i] > ninf ? order_bits(c[i]) : kNoKey;
        }
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        if (KEY == KEY_CHOICE) {
            key[i] = gkey[i];
        } else {
            key[i] = order_key(x[i]);
            if (!sums)
                gkey[i] = key[i];
        }
    }
    bool close = false;  // some pair of the row is too close for 32 bits
    bool open = true;    // the lane's group stays
    if (a.groups > 1) {
        uint32_t b1 = gkey[0], b2 = kNoKey;
#pragma unroll
        for (int i = 1; i < PL; ++i) {
            b2 = max(b2, min(b1, gkey[i]));
            b1 = max(b1, gkey[i]);
        }
        auto merge = [&](uint32_t c1, uint32_t c2) {
            b2 = max(max(b2, c2), min(b1, c1));
            b1 = max(b1, c1);
        };
        if (run > 1)
            merge(dpp_u<kXor1>(b1), dpp_u<kXor1>(b2));
        if (run > 2)
            merge(dpp_u<kXor2>(b1), dpp_u<kXor2>(b2));
        if (run > 4)
            merge(dpp_u<kHalfMirror>(b1), dpp_u<kHalfMirror>(b2));
        const float v1 = key_value(b1), v2 = key_value(b2);
        const bool two = sums && b2 > kNoKey;
        // logits compare exactly; a sum is off by as much as both its terms,
        // whose magnitudes count where they cancel
        float slack = -1.0f;
        if (KEY == KEY_CHOICE || sums) {
            slack = 4.0f * off + 0x1p-21f * (fabsf(v1) + (two ? fabsf(v2) : 0.0f));
            // of any two groups of the row (infinite where one is: all close)
            slack = __uint_as_float(row_max(v1 > ninf ? __float_as_uint(slack) : 0));
        }
        const float value = two ? v1 + v2 : v1;
        // equal infinities tie in 64 bits too, but for a sum of finite choices
        // that only 32 bits cannot hold
        if (two)
            close = fabsf(value) == __builtin_inff() && fabsf(v1) < __builtin_inff() && fabsf(v2) < __builtin_inff();
        int better = 0;
        rank_groups<1>(value, l, run, slack, better, close);
        open = better < a.kept;
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
        key[i] = KEY == KEY_LOGIT16 ? (key[i] & ~kIndexes) | (uint32_t)((int)kIndexes - e0 - i)
                                    : (key[i] & ~kSlots) | (uint32_t)(kSlots - i);
    sort_down(key);
    key[0] = open ? key[0] : 0;  // this lane never holds the largest
    uint32_t mine = 0, lanes_lo = 0, lanes_hi = 0;  // lane j: key j, and which lane held it
    take_best<0, KM, KEY>(key, a.topk, l, mine, lanes_lo, lanes_hi);
    const uint32_t rest = row_max(key[0]);  // the best that is not chosen
    const uint32_t after = dpp_u<0x101>(mine);  // row_shl: of lane l + 1
    const uint32_t next = l + 1 == a.topk ? rest : after;
    const bool chosen = l < a.topk && mine > kNoKey;
    // whether a chosen key and a lower one are too close to tell
    auto too_near = [&](uint32_t high, uint32_t low) {
        if (KEY == KEY_LOGIT16 || low <= kNoKey)
            return false;
        if (KEY == KEY_LOGIT32)
            return ((high ^ low) & ~kSlots) == 0;
        // both off by `off` + 2^-23 and 15 (31) steps of 2^-23 for the slot
        const float v = key_value(high), w = key_value(low);
        return !(v - w > 2.0f * off + (PL <= 16 ? 0x1p-18f : 0x1p-17f) * (fabsf(v) + fabsf(w)));
    };
    const bool near = chosen && too_near(mine, next);
    int my_id = -1;
    int place = l;
    double s = 0.0, exact = kNone;
    if (chosen) {
        const uint32_t lanes = ((lane & 32 ? lanes_hi : lanes_lo) >> (lane & 16)) & 0xFFFF;
        my_id = KEY == KEY_LOGIT16 ? (int)(kIndexes - (mine & kIndexes))
                                   : first_of(__ffs((int)lanes) - 1) + (int)(kSlots - (mine & kSlots));
        const float v = load_logit(a, row + my_id);
        s = a.softmax ? exp_below64(v, top) : sigmoid64(v);
        exact = (double)v;
    }
    if (KEY != KEY_LOGIT16 && __ballot(near) != 0) {
        // The chosen ones are ordered by their 64-bit values.  They are the
        // right ones if the best that is not chosen is below all of them, in
        // 64 bits where it is near the last, and the one behind that far
        // enough (one key in several lanes: more than one is as good).
        const bool best = key[0] == rest && rest > kNoKey;
        const uint64_t all = __ballot(best);
        const uint32_t holders = ((uint32_t)(lane & 32 ? all >> 32 : all) >> (lane & 16)) & 0xFFFF;
        const uint32_t behind = row_max(best ? key[1] : key[0]);
        const bool last = near && l + 1 == a.topk;
        const bool against = chosen && ((__ballot(last) >> (lane & 48)) & 0xFFFF) != 0;
        int rest_id = 0;
        double rest_value = kNone;
        if (against) {
            rest_id = first_of(__ffs((int)holders) - 1) + (int)(kSlots - (rest & kSlots));
            rest_value = (double)load_logit(a, row + rest_id);
        }
        if (KEY == KEY_CHOICE) {
            double whole = total;
            if (a.softmax && a.renorm) {  // not needed so far, and seldom here
                float again[PL];
                load_run<PL>(a, row, e0, live ? count : 0, again);
                whole = 0.0;
#pragma unroll
                for (int i = 0; i < PL; ++i)
                    whole += again[i] > ninf ? exp_below64(again[i], top) : 0.0;
                whole = run_sum<0>(whole, 16);
            }
            if (chosen)
                exact = (a.softmax ? s / whole : s) + (double)a.bias[my_id];
            if (against) {
                const float v = (float)rest_value;
                rest_value = (a.softmax ? exp_below64(v, top) / whole : sigmoid64(v)) + (double)a.bias[rest_id];
            }
        }
        close |= chosen && !(exact > rest_value || (exact == rest_value && my_id < rest_id));  // NaN: close
        close |= last && ((holders & (holders - 1)) != 0 || too_near(mine, behind));
        const int ahead = count_ahead<1>(exact, my_id);
        place = chosen ? ahead : l;
    }
    if (a.renorm) {
        const double sum = run_sum<0>(s, a.topk);
        s = sum > 0.0 ? s / sum : 0.0;
    } else if (a.softmax && chosen) {
        s = s / total;
    }
    const uint64_t again = KEY != KEY_LOGIT16 || sums ? __ballot(close && live) : 0;
    if (t < a.T && l < a.topk && ((again >> (lane & 48)) & 0xFFFF) == 0) {
        a.ids[t * a.topk + place] = my_id;
        a.weights[t * a.topk + place] = (float)((double)a.scale * s);
    }
    if (again != 0) {
        for (int r = 0; r < 4; ++r)
            if ((again >> (16 * r)) & 0xFFFF) {
                if (PL == 4)
                    route_token<1, true>(a, t0 + r);
                else if (PL == 8)
                    route_token<2, true>(a, t0 + r);
                else
                    route_token<PL / 4, true>(a, t0 + r);
            }
    }
}

namespace {

template <int PL>
void launch_lanes(const RouteArgs& a, bool scores, hipStream_t s)
{
    const dim3 grid((unsigned)((a.T + kRWaves - 1) / kRWaves)), block(64 * kRWaves);
    if (scores)
        hipLaunchKernelGGL((route_kernel<PL, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((route_kernel<PL, false>), grid, block, 0, s, a);
}

}  // namespace

namespace {

template <int PL, int KM>
void launch_rows(const RouteArgs& a, hipStream_t s)
{
    // few tokens: a wave per workgroup, so that they spread over the CUs
    const int waves = a.T <= 4096 ? 1 : 4;
    const dim3 grid((unsigned)((a.T + 4 * waves - 1) / (4 * waves))), block(64 * waves);
    if (a.bias != nullptr)
        hipLaunchKernelGGL((route_rows_kernel<PL, KEY_CHOICE, KM>), grid, block, 0, s, a);
    else if (a.type == W4A8_TYPE_FP32)
        hipLaunchKernelGGL((route_rows_kernel<PL, KEY_LOGIT32, KM>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((route_rows_kernel<PL, KEY_LOGIT16, KM>), grid, block, 0, s, a);
}

// rows of 16 lanes: up to 16 experts of at most 16 groups, each of which gets
// the lanes of a power of two and fits them with 32 experts a lane
template <int PL>
bool try_rows(RouteArgs a, int per, int run_log2, hipStream_t s)
{
    if (per > PL)
        return false;
    a.per = a.groups == 1 ? PL : per;
    a.run_log2 = run_log2;
    if (a.topk <= 8)
        launch_rows<PL, 8>(a, s);
    else
        launch_rows<PL, 16>(a, s);
    return true;
}

}  // namespace

// Four tokens per wave where their rows fit 16 lanes, else one (32768 tokens,
// 256 experts in 8 groups, top 8: 20 us against 52; 8192 tokens, 440 experts,
// top 8: 12 us against 27).
hipError_t launch_route(const RouteArgs& a, hipStream_t s)
{
    if (a.topk <= 16 && a.groups <= 16) {
        int run_log2 = 4;
        while ((16 >> run_log2) < a.groups)
            --run_log2;
        const int lanes = 1 << run_log2, per = (a.E / a.groups + lanes - 1) / lanes;
        if (try_rows<4>(a, per, run_log2, s) || try_rows<8>(a, per, run_log2, s) || try_rows<16>(a, per, run_log2, s) ||
            try_rows<32>(a, per, run_log2, s))
            return hipGetLastError();
    }
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
