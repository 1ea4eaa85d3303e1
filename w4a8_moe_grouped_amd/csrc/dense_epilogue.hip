// dense_epilogue.hip -- the dense W4AFP8 linear with bias, activation and
// residual in its epilogue (w4a8_gemm_epilogue):
//   out[m, n] = bf16(act(sum_g sa[m, g] sw[n, g] sum_{k in g} a[m, k] w[n, k] + bias[n]) + residual[m, n]).
//
// Few rows (dense_rows_kernel): bound by the weight bytes and by latency.  A
// workgroup owns NF fragments of 16 weight rows and MF slices of 16
// activation rows, and its 8 waves split K: each streams its own groups
// from memory straight into registers, with no barrier and no partial sums in
// memory, and the 8 sums of an output meet in LDS, in wave order.  The
// weights are the first MFMA operand, so a lane holds four consecutive
// outputs of one row, which the epilogue reads and writes as one access.
// With SwiGLU, fragment f of the up rows stands beside fragment f of the gate
// rows.
#include "dense_common.hpp"

namespace w4a8 {

namespace {

constexpr int kSWaves = 8;  // waves per workgroup, each a part of K

}  // namespace

// MF slices of 16 activation rows x NF fragments of 16 weight rows.
template <int MF, int NF, bool GLU>
__global__ __launch_bounds__(64 * kSWaves) void dense_rows_kernel(const DenseArgs a)
{
    static_assert(!GLU || NF % 2 == 0, "gate and up fragments come in pairs");
    constexpr int kOut = GLU ? NF / 2 : NF;  // fragments of outputs
    __shared__ float4 s_sum[kSWaves][MF * NF][64];

    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, c16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = (int)(a.K / kGroup);
    const int64_t col_blocks = (a.N + 16 * kOut - 1) / (16 * kOut);
    const int64_t mb = blockIdx.x / col_blocks;
    const int64_t n0 = (blockIdx.x - mb * col_blocks) * (16 * kOut);
    const int64_t m0 = mb * (16 * MF);

    // rows past the end read the last valid row
    const uint8_t* wp[NF];
    const float* wsp[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        const int64_t n = min(n0 + 16 * (f % kOut) + c16, a.N - 1);
        const int64_t row = GLU && f >= kOut ? a.N + n : n;
        wp[f] = a.w + row * (a.K / 2) + 16 * q;
        wsp[f] = a.sw + row * G;
    }
    const uint8_t* ap[MF];
    const float* asp[MF];
#pragma unroll
    for (int s = 0; s < MF; ++s) {
        const int64_t m = min(m0 + 16 * s + c16, a.M - 1);
        ap[s] = a.a + m * a.K + 32 * q;
        asp[s] = a.sa + m * G;
    }
    v4f acc[MF][NF];
#pragma unroll
    for (int s = 0; s < MF; ++s)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            acc[s][f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    const int g1 = (int)((int64_t)G * (wave + 1) / kSWaves);
    for (int g = (int)((int64_t)G * wave / kSWaves); g < g1; ++g) {
        v8i b[NF];
        float sw[NF][4];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            b[f] = int4_to_fp8(ldg16(wp[f] + (int64_t)g * (kGroup / 2)));
            const float own = wsp[f][g];  // scale of weight row c16; the sums are of rows 4q + i
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sw[f][i] = __shfl(own, 4 * q + i, 64);
        }
#pragma unroll
        for (int s = 0; s < MF; ++s) {
            const v4i a0 = ldg16(ap[s] + (int64_t)g * kGroup), a1 = ldg16(ap[s] + (int64_t)g * kGroup + 16);
            const v8i av = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
            const float sa = asp[s][g] * 512.0f;  // the weight codes count units of 2^-9
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const v4f raw = mfma16x16x128(b[f], av, v4f{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[s][f][i] = fmaf(sw[f][i], raw[i] * sa, acc[s][f][i]);
            }
        }
    }
#pragma unroll
    for (int s = 0; s < MF; ++s)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            s_sum[wave][s * NF + f][lane] = make_float4(acc[s][f][0], acc[s][f][1], acc[s][f][2], acc[s][f][3]);
    __syncthreads();
    // item (slice s, output fragment f, lane): row 16s + lane%16, columns 16f + 4(lane/16)..
    for (int item = wave; item < MF * kOut; item += kSWaves) {
        const int s = item / kOut, f = item - s * kOut;
        float y[4] = {0, 0, 0, 0}, up[4] = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kSWaves; ++w) {
            const float4 v = s_sum[w][s * NF + f][lane];
            y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
            if (GLU) {
                const float4 u = s_sum[w][s * NF + kOut + f][lane];
                up[0] += u.x, up[1] += u.y, up[2] += u.z, up[3] += u.w;
            }
        }
        const int64_t m = m0 + 16 * s + c16;
        if (m < a.M)
            epilogue4(a, m, n0 + 16 * f + 4 * q, y, up);
    }
}

namespace {

template <int MF>
hipError_t launch_rows(const DenseArgs& a, hipStream_t s)
{
    const bool glu = a.act == W4A8_ACT_SWIGLU;
    const int64_t cols = glu ? 16 : 32;
    const int64_t blocks = ((a.N + cols - 1) / cols) * ((a.M + 16 * MF - 1) / (16 * MF));
    if (blocks > INT32_MAX)
        return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block(64 * kSWaves);
    if (glu)
        hipLaunchKernelGGL((dense_rows_kernel<MF, 2, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((dense_rows_kernel<MF, 2, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t dense_epilogue_workspace(int64_t M, int64_t K, int64_t N, int act)
{
    return use_dense_tiles(M, K, N, act) ? dense_tiles_workspace(M, K, N, act) : 0;
}

hipError_t launch_dense_epilogue(const DenseArgs& a, void* ws, hipStream_t s)
{
    if (use_dense_tiles(a.M, a.K, a.N, a.act))
        return launch_dense_tiles(a, ws, s);
    if (a.M <= 16)
        return launch_rows<1>(a, s);
    if (a.M <= 32)
        return launch_rows<2>(a, s);
    return launch_rows<4>(a, s);
}

}  // namespace w4a8
