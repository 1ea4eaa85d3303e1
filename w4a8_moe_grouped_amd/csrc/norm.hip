// norm.hip -- the norm after a block with its gate and residual sum, and the
// norm before the next block with its fp8 quantisation (w4a8_norm_residual):
//   u = x * rsqrt(mean(x^2) + eps) * (wpost + off),  r' = scale*r + gate*u,
//   y = r' * rsqrt(mean(r'^2) + eps) * (wpre + off).
//
// HBM-bound: a row is read once, held in registers through both sums, and
// every output written once.  A thread holds NC chunks of 8 consecutive
// elements, chunk c of a row in thread c % (threads per row), so that wide
// accesses of a wave are contiguous and the 16 chunks of a 128-block, whose
// largest value sets its scale, lie in 16 neighbouring lanes.  Short rows take
// one wave each (no barrier), longer ones a workgroup each.  Sums and the
// values between them are fp32.  Measured at H = 7168: 4096 rows of bf16 to
// codes 46 us (4.5 TB/s of the 5.1 a copy reaches; loads and stores past the
// caches changed nothing), 16384 rows with an fp32 residual 262 us (5.4 TB/s),
// 64 rows 5.2 us, one row 3.4 us (two dependent sums behind one load: latency).
#include "w4a8.h"

#include "common.hpp"
#include "internal.hpp"

namespace w4a8 {

namespace {

constexpr int kNRows = 4;  // rows per workgroup with one wave per row

// Rows start at any element, so 16 bytes are accessed at the alignment of one
// of them; a misaligned wide access is one instruction here (16220 rows of 2085
// bf16: 51 us, element by element 224).
typedef float float4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t uint4_any __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ void load8(const float* p, int h, int H, float* v)
{
    if (h + 8 <= H) {
        const float4_any a = *(const float4_any*)(p + h), b = *(const float4_any*)(p + h + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = a[i], v[4 + i] = b[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = h + i < H ? p[h + i] : 0.0f;
}
__device__ __forceinline__ void load8(const uint16_t* p, int h, int H, float* v)
{
    if (h + 8 <= H) {
        const uint4_any raw = *(const uint4_any*)(p + h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(raw[i] << 16);
            v[2 * i + 1] = __uint_as_float(raw[i] & 0xFFFF0000u);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = h + i < H ? bf16_to_f32(p[h + i]) : 0.0f;
}
__device__ __forceinline__ void load8_param(const void* p, int64_t row, int type, int h, int H, float* v)
{
    if (type == W4A8_TYPE_FP32)
        load8((const float*)p + row, h, H, v);
    else
        load8((const uint16_t*)p + row, h, H, v);
}
__device__ __forceinline__ float load1_param(const void* p, int64_t i, int type)
{
    return type == W4A8_TYPE_FP32 ? ((const float*)p)[i] : bf16_to_f32(((const uint16_t*)p)[i]);
}

__device__ __forceinline__ void store8(float* p, int h, int H, const float* v)
{
    if (h + 8 <= H) {
        *(float4_any*)(p + h) = float4_any{v[0], v[1], v[2], v[3]};
        *(float4_any*)(p + h + 4) = float4_any{v[4], v[5], v[6], v[7]};
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (h + i < H)
            p[h + i] = v[i];
}
__device__ __forceinline__ void store8(uint16_t* p, int h, int H, const float* v)
{
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        d[i] = f32x2_to_bf16x2(v[2 * i], v[2 * i + 1]);
    if (h + 8 <= H) {
        *(uint4_any*)(p + h) = uint4_any{d[0], d[1], d[2], d[3]};
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (h + i < H)
            p[h + i] = (uint16_t)(d[i / 2] >> (16 * (i & 1)));
}

// the maximum of 16 neighbouring lanes
__device__ __forceinline__ uint32_t block_max(uint32_t v)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
    return v;
}

// the row's sum; s_part: one float per wave of the workgroup
template <bool WAVE_ROW>
__device__ __forceinline__ float row_sum(float v, float* s_part)
{
    v = group_sum<64>(v);
    if (WAVE_ROW)
        return v;
    if ((threadIdx.x & 63) == 0)
        s_part[threadIdx.x >> 6] = v;
    __syncthreads();
    const int waves = (int)blockDim.x >> 6;
    float sum = 0.0f;
    for (int w = 0; w < waves; ++w)
        sum += s_part[w];
    return sum;
}

}  // namespace

template <typename XT, typename RT, int NC, bool WAVE_ROW>
__global__ __launch_bounds__(WAVE_ROW ? 64 * kNRows : 1024) void norm_kernel(const NormArgs a)
{
    __shared__ float s_part[2][16];
    const int H = a.H;
    const int threads = WAVE_ROW ? 64 : (int)blockDim.x;
    const int tid = WAVE_ROW ? (int)threadIdx.x & 63 : (int)threadIdx.x;
    const int64_t t = WAVE_ROW ? (int64_t)blockIdx.x * kNRows + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
    if (WAVE_ROW && t >= a.T)
        return;
    const float inv_h = 1.0f / (float)H;

    float v[NC][8], r[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int h = (c * threads + tid) * 8;
        if (a.x != nullptr)
            load8((const XT*)a.x + t * a.ldx, h, H, v[c]);
        if (a.residual != nullptr)
            load8((const RT*)a.residual + t * a.ldr, h, H, r[c]);
    }
    // r' in v
    if (a.x != nullptr) {
        float mul = 1.0f;
        if (a.post_w != nullptr) {
            float ss = 0.0f;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    ss = fmaf(v[c][i], v[c][i], ss);
            mul = rsqrtf(fmaf(row_sum<WAVE_ROW>(ss, s_part[0]), inv_h, a.eps));
        }
        if (a.gate != nullptr && a.gate_cs == 0)
            mul *= load1_param(a.gate, t * a.gate_rs, a.p_type);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int h = (c * threads + tid) * 8;
            float w[8];
            if (a.post_w != nullptr) {
                load8_param(a.post_w, 0, a.p_type, h, H, w);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[c][i] *= w[i] + a.w_offset;
            }
            if (a.gate != nullptr && a.gate_cs != 0) {
                load8_param(a.gate, t * a.gate_rs, a.p_type, h, H, w);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[c][i] *= w[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[c][i] *= mul;
            if (a.residual != nullptr) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[c][i] = fmaf(a.r_scale, r[c][i], v[c][i]);
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[c][i] = a.r_scale * r[c][i];
    }
    if (a.r_out != nullptr) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
            store8((RT*)a.r_out + t * a.ldr_out, (c * threads + tid) * 8, H, v[c]);
    }
    if (a.pre_w == nullptr)
        return;
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ss = fmaf(v[c][i], v[c][i], ss);
    const float mul = rsqrtf(fmaf(row_sum<WAVE_ROW>(ss, s_part[1]), inv_h, a.eps));
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int h = (c * threads + tid) * 8;
        float w[8];
        load8_param(a.pre_w, 0, a.p_type, h, H, w);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[c][i] *= mul * (w[i] + a.w_offset);
        if (a.y != nullptr)
            store8(a.y + t * a.ldy, h, H, v[c]);
        if (a.q != nullptr) {
            // H is a multiple of 128: the 16 lanes of a block are all inside
            // the row or all behind it
            // magnitudes as integers: a NaN is the largest, and makes the
            // block's scale NaN
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                top = max(top, __float_as_uint(v[c][i]) & 0x7FFFFFFFu);
            top = block_max(top);
            const float amax = clamp_amax(__uint_as_float(top));
            const float inv = recip448(amax);
            uint32_t d[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                d[i] = cvt_e4m3x2(v[c][2 * i] * inv, v[c][2 * i + 1] * inv);
            if (h < H) {
                *(uint2*)(a.q + t * H + h) = make_uint2(d[0] | (d[1] << 16), d[2] | (d[3] << 16));
                if ((tid & 15) == 0)
                    a.q_scales[t * (H / kGroup) + h / kGroup] =
                        top > 0x7F800000u ? __uint_as_float(top) : scale_of(amax);
            }
        }
    }
}

namespace {

template <typename XT, typename RT>
void launch_typed(const NormArgs& a, hipStream_t s)
{
    const int chunks = (a.H + 7) / 8;
    const unsigned T = (unsigned)a.T;
    if (a.H <= kNormShortH) {
        hipLaunchKernelGGL((norm_kernel<XT, RT, 1, true>), dim3((T + kNRows - 1) / kNRows),
                           dim3(64 * kNRows), 0, s, a);
        return;
    }
    // up to 1024 threads a row; with more rows than stand on the GPU at once
    // half as many threads with two chunks each, so that more rows share a CU
    // (H 7168, bf16 to codes: 4096 rows 60 -> 46 us, 64 rows 5.4 -> 6.3)
    const int nc = chunks <= 1024 ? (a.T > 512 ? 2 : 1) : chunks <= 2048 ? 2 : 4;
    const dim3 block((unsigned)(((chunks + nc - 1) / nc + 63) / 64 * 64));
    if (nc == 1)
        hipLaunchKernelGGL((norm_kernel<XT, RT, 1, false>), dim3(T), block, 0, s, a);
    else if (nc == 2)
        hipLaunchKernelGGL((norm_kernel<XT, RT, 2, false>), dim3(T), block, 0, s, a);
    else
        hipLaunchKernelGGL((norm_kernel<XT, RT, 4, false>), dim3(T), block, 0, s, a);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t s)
{
    const bool x32 = a.x_type == W4A8_TYPE_FP32, r32 = a.r_type == W4A8_TYPE_FP32;
    if (x32)
        r32 ? launch_typed<float, float>(a, s) : launch_typed<float, uint16_t>(a, s);
    else
        r32 ? launch_typed<uint16_t, float>(a, s) : launch_typed<uint16_t, uint16_t>(a, s);
    return hipGetLastError();
}

}  // namespace w4a8
