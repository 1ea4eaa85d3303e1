// dense_epilogue.hip -- the dense W4AFP8 linear with bias, activation and
// residual in its epilogue (w4a8_gemm_epilogue):
//   out[m, n] = bf16(act(sum_g sa[m, g] sw[n, g] sum_{k in g} a[m, k] w[n, k] + bias[n]) + residual[m, n]).
//
// Few rows (dense_rows_kernel; many rows: dense_tiles.hip): bound by the
// weight bytes and by latency.  A workgroup owns NF fragments of 16 weight
// rows and MF slices of 16 activation rows, and its 8 waves split K, so that
// all its bytes are asked for at once and no partial sums go through memory.
// Each wave streams its own groups into its own ring of D stages in LDS
// (buffer_load ... lds, no barrier): eight consecutive lanes read a row's 128
// activation bytes, four its 64 weight bytes.  (Loading straight into the
// lanes of the MFMA operands, where neighbouring lanes hold different rows,
// kept a CU's address unit busy for 4.5 us of a 12 us call.)  The 8 sums of
// an output meet in LDS, in wave order.
//
// M 1, K 7168, R 4096: 7.9 us for 15.6 MB (2.0 TB/s; 3.3 us of it at K = 128:
// launch, one load, the sums); M 64, K 2048, R 7168: 6.0 us.  The weights become
// the codes of their values, as in the tiles: codes of v + 8, which take less
// than half the decode (6.7 and 5.8 us), add 8 times the activations to what the
// matrix instruction sums in 13 bits and take them off again, so that small
// weights lose bits to large activations.
//
// The weights are the first MFMA operand, so a lane holds four consecutive
// outputs of one row, which the epilogue reads and writes as one access.  With
// SwiGLU, fragment f of the up rows stands beside fragment f of the gate rows.
#include "api_util.hpp"
#include "dense_common.hpp"
#include "lds_direct.hpp"

namespace w4a8 {

namespace {

constexpr int kChunk = 8;  // groups whose scales are staged at once

// 16-byte slots in a stage.  Of the two swizzles each spreads what the lanes
// of one LDS cycle read (8 rows, two neighbouring quarters) over all banks.
__device__ __forceinline__ int act_slot(int row, int chunk)
{
    return row * 8 + (chunk ^ ((row >> 1 & 1) | (row & 4)));
}
__device__ __forceinline__ int wgt_slot(int row, int chunk)
{
    return row * 4 + (chunk ^ ((row >> 1 & 2) | (row >> 3 & 1)));
}

template <int MF, int NF, int D, int WAVES>
struct RowsLds {
    static constexpr int kStage = NF * 1024 + MF * 2048;  // weights, then activations
    static constexpr int kScales = (NF + MF) * 16 * kChunk * 4;
    static constexpr int kWave = D * kStage + kScales;
    static_assert(MF * NF * 1024 <= kWave, "a wave's sums fit its own part");
    static_assert(WAVES * kWave <= 160 * 1024, "LDS of a CU");
};

}  // namespace

template <int MF, int NF, bool GLU, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void dense_rows_kernel(const DenseArgs a, const int32_t col_blocks)
{
    static_assert(!GLU || NF % 2 == 0, "gate and up fragments come in pairs");
    using Lds = RowsLds<MF, NF, D, WAVES>;
    constexpr int kOut = GLU ? NF / 2 : NF;  // fragments of outputs
    constexpr int kLoads = NF + 2 * MF;      // per group
    __shared__ __attribute__((aligned(16))) uint8_t smem[WAVES * Lds::kWave];

    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, c16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = (int)(a.K / kGroup);
    const int mb = (int)blockIdx.x / col_blocks;
    const int64_t n0 = (int64_t)((int)blockIdx.x - mb * col_blocks) * (16 * kOut);
    const int64_t m0 = (int64_t)mb * (16 * MF);

    // the first of this wave's items of the epilogue (slice, output fragment)
    const int item_s = wave / kOut, item_f = wave - item_s * kOut;
    const int64_t item_m = m0 + 16 * item_s + c16, item_n = n0 + 16 * item_f + 4 * q;
    EpiOperands pre = {};
    if (wave < MF * kOut && item_m < a.M)
        pre = load_epilogue4(a, item_m, item_n);

    // Rows of the block's first to last; those past the end read the last
    // valid one.  The resources begin at the block's first row, so 32 bits
    // hold every offset.  Up rows lie N rows behind their gate rows.
    const int rows_a = (int)min((int64_t)(16 * MF), a.M - m0);
    const int rows_w = (int)min((int64_t)(16 * kOut), a.N - n0);
    const uint32_t wrow = (uint32_t)(a.K / 2), arow = (uint32_t)a.K, srow = (uint32_t)G * 4;
    const v4i ra = sgpr_rsrc(a.a + m0 * a.K, rows_a * arow);
    const v4i rsa = sgpr_rsrc(a.sa + m0 * G, rows_a * srow);
    const v4i rw = sgpr_rsrc(a.w + n0 * (a.K / 2), rows_w * wrow);
    const v4i rsw = sgpr_rsrc(a.sw + n0 * G, rows_w * srow);
    const v4i ru = sgpr_rsrc(a.w + (n0 + (GLU ? a.N : 0)) * (a.K / 2), rows_w * wrow);
    const v4i rsu = sgpr_rsrc(a.sw + (n0 + (GLU ? a.N : 0)) * G, rows_w * srow);

    uint8_t* const mine = smem + wave * Lds::kWave;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)mine;
    // lane -> (row, chunk) of the direct loads, whose LDS side is linear
    uint32_t vw[kOut], va[2 * MF];
#pragma unroll
    for (int f = 0; f < kOut; ++f) {
        const int r = lane >> 2, c = (lane & 3) ^ ((r >> 1 & 2) | (r >> 3 & 1));
        vw[f] = (uint32_t)min(16 * f + r, rows_w - 1) * wrow + 16 * c;
    }
#pragma unroll
    for (int j = 0; j < 2 * MF; ++j) {
        const int r = 8 * j + (lane >> 3), c = (lane & 7) ^ ((r >> 1 & 1) | (r & 4));
        va[j] = (uint32_t)min(r, rows_a - 1) * arow + 16 * c;
    }
    auto issue = [&](int g, int st) {
        const uint32_t base = lds0 + (uint32_t)(st * Lds::kStage);
#pragma unroll
        for (int f = 0; f < NF; ++f)
            lds_load16(f < kOut ? rw : ru, base + 1024u * f, vw[f % kOut], (uint32_t)g * (kGroup / 2));
#pragma unroll
        for (int j = 0; j < 2 * MF; ++j)
            lds_load16(ra, base + 1024u * (NF + j), va[j], (uint32_t)g * kGroup);
    };
    // scales of groups c0 .. c0 + 7 as [row][8], weight rows first
    auto issue_scales = [&](int c0) {
        const uint32_t base = lds0 + (uint32_t)(D * Lds::kStage);
        const uint32_t g = 4u * (uint32_t)min(c0 + (lane & 7), G - 1);
#pragma unroll
        for (int j = 0; j < 2 * NF; ++j) {
            const int r = 8 * j + (lane >> 3);
            const bool up = GLU && j >= 2 * kOut;
            lds_load4(up ? rsu : rsw, base + 256u * j, (uint32_t)min(up ? r - 16 * kOut : r, rows_w - 1) * srow + g, 0);
        }
#pragma unroll
        for (int j = 0; j < 2 * MF; ++j)
            lds_load4(rsa, base + 256u * (2 * NF + j), (uint32_t)min(8 * j + (lane >> 3), rows_a - 1) * srow + g, 0);
    };

    v4f acc[MF][NF];
#pragma unroll
    for (int s = 0; s < MF; ++s)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            acc[s][f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const float* const scales = (const float*)(mine + D * Lds::kStage);
    auto multiply = [&](const uint8_t* st, int gi) {  // group gi of the chunk
        v8i b[NF];
        float sw[NF][4];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            b[f] = int4_to_fp8(*(const v4i*)(st + 1024 * f + 16 * wgt_slot(c16, q)));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sw[f][i] = scales[(16 * f + 4 * q + i) * kChunk + gi];
        }
#pragma unroll
        for (int s = 0; s < MF; ++s) {
            const v4i a0 = *(const v4i*)(st + 1024 * NF + 16 * act_slot(16 * s + c16, 2 * q));
            const v4i a1 = *(const v4i*)(st + 1024 * NF + 16 * act_slot(16 * s + c16, 2 * q + 1));
            const v8i av = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
            const float sa = scales[(16 * (NF + s) + c16) * kChunk + gi];
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const v4f raw = mfma16x16x128(b[f], av, v4f{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    // the scales meet first: the largest activation scale (a
                    // bf16 maximum / 448) has no room for the sum alone
                    acc[s][f][i] = fmaf(raw[i], sw[f][i] * sa, acc[s][f][i]);
            }
        }
    };
    const int g0 = (int)((int64_t)G * wave / WAVES), g1 = (int)((int64_t)G * (wave + 1) / WAVES);
    for (int c0 = g0; c0 < g1; c0 += kChunk) {
        const int n = min(kChunk, g1 - c0);
        issue_scales(c0);
#pragma unroll
        for (int i = 0; i < D; ++i)
            if (i < n)
                issue(c0 + i, i);
        int st = 0, i = 0;
        if constexpr (D % 2 == 0 && D > 2) {
            // two groups at a time: one's matrix products run under the other's
            // decode (1 x 7168 x 4096: 7.8 us against 8.2)
            for (; i + 1 < n; i += 2) {
                if (n - 2 - i >= D - 2)
                    wait_vmcnt<(D - 2) * kLoads>();
                else
                    wait_vmcnt<0>();
                asm volatile("" ::: "memory");
                multiply(mine + st * Lds::kStage, i);
                multiply(mine + (st + 1) * Lds::kStage, i + 1);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (i + D + j < n)
                        issue(c0 + i + D + j, st + j);
                st = st + 2 == D ? 0 : st + 2;
            }
        }
        for (; i < n; ++i) {
            // group i (and the scales before it) landed; up to D - 1 behind it fly
            if (D > 1 && n - 1 - i >= D - 1)
                wait_vmcnt<(D - 1) * kLoads>();
            else
                wait_vmcnt<0>();
            asm volatile("" ::: "memory");
            multiply(mine + st * Lds::kStage, i);
            // the stage has been read before it is filled again
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (i + D < n)
                issue(c0 + i + D, st);
            st = st + 1 == D ? 0 : st + 1;
        }
    }
    // the wave's sums, over its own ring (no load is in flight any more)
#pragma unroll
    for (int s = 0; s < MF; ++s)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            *(float4*)(mine + 1024 * (s * NF + f) + 16 * lane) =
                make_float4(acc[s][f][0], acc[s][f][1], acc[s][f][2], acc[s][f][3]);
    __syncthreads();
    // item (slice s, output fragment f, lane): row 16s + lane%16, columns 16f + 4(lane/16)..
    for (int item = wave; item < MF * kOut; item += WAVES) {
        const int s = item / kOut, f = item - s * kOut;
        float y[4] = {0, 0, 0, 0}, up[4] = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const uint8_t* part = smem + w * Lds::kWave + 1024 * (s * NF + f) + 16 * lane;
            const float4 v = *(const float4*)part;
            y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
            if (GLU) {
                const float4 u = *(const float4*)(part + 1024 * kOut);
                up[0] += u.x, up[1] += u.y, up[2] += u.z, up[3] += u.w;
            }
        }
        const int64_t m = m0 + 16 * s + c16, n = n0 + 16 * f + 4 * q;
        if (m < a.M)
            epilogue4(a, m, n, y, up, item == wave ? pre : load_epilogue4(a, m, n));
    }
}

namespace {

template <int MF, int NF, int D, int WAVES>
hipError_t launch_rows(const DenseArgs& a, hipStream_t s)
{
    const bool glu = a.act == W4A8_ACT_SWIGLU;
    const int64_t cols = 16 * (glu ? NF / 2 : NF), col_blocks = (a.N + cols - 1) / cols;
    const dim3 grid((unsigned)(col_blocks * ((a.M + 16 * MF - 1) / (16 * MF)))), block(64 * WAVES);
    if (glu)
        hipLaunchKernelGGL((dense_rows_kernel<MF, NF, true, D, WAVES>), grid, block, 0, s, a, (int32_t)col_blocks);
    else
        hipLaunchKernelGGL((dense_rows_kernel<MF, NF, false, D, WAVES>), grid, block, 0, s, a, (int32_t)col_blocks);
    return hipGetLastError();
}

}  // namespace

size_t dense_epilogue_workspace(int64_t M, int64_t K, int64_t N, int act)
{
    return use_dense_tiles(M, K, N, act) ? dense_tiles_workspace(M, K, N, act) : 0;
}

// Whether every launch of the call stays below 2^32 threads; the choices are
// those of launch_dense_epilogue (few workgroups always do).
bool dense_epilogue_fits(int64_t M, int64_t K, int64_t N, int act)
{
    if (use_dense_tiles(M, K, N, act))
        return dense_tiles_fit(M, K, N, act);
    const int64_t R = act == W4A8_ACT_SWIGLU ? 2 * N : N;
    const int64_t threads = M <= 16 ? api::ceil_div(R, 32) * 512 : api::ceil_div(M, 32) * api::ceil_div(R, 64) * 256;
    return threads <= UINT32_MAX;
}

hipError_t launch_dense_epilogue(const DenseArgs& a, void* ws, hipStream_t s)
{
    if (use_dense_tiles(a.M, a.K, a.N, a.act))
        return launch_dense_tiles(a, ws, s);
    // Few workgroups: 8 waves each and, for a decode batch's single slice, a
    // ring deep enough to ask for all of a wave's bytes at once.  More of them:
    // what counts is how many a CU holds (32 to 44 KB of LDS each, ring of one
    // stage), so that one's loads run under another's products, and from about
    // three rounds on wider ones, which load fewer activations.  Measured (us;
    // <slices, fragments, ring, waves>): M 64, K 7168, R 4096 <2,2,1,8> 9.6,
    // <2,2,1,4> 13.3, <2,4,1,4> 17.9; M 64, K 2048, R 7168 7.1 / 6.3 / 7.9; M 300
    // 23.4 / 19.5 / 18.3; M 512, K 7168, R 2048 28.0 / 27.3 / 26.4; a ring of two
    // stages with <2,4> and 8 waves takes 7.6, 31.1 and 30.0 on the last three.
    if (a.M <= 16)
        return launch_rows<1, 2, 4, 8>(a, s);
    const int64_t R = a.act == W4A8_ACT_SWIGLU ? 2 * a.N : a.N;
    const int64_t blocks = ((R + 31) / 32) * ((a.M + 31) / 32);
    if (blocks <= 256)
        return launch_rows<2, 2, 1, 8>(a, s);
    if (blocks <= 800)
        return launch_rows<2, 2, 1, 4>(a, s);
    return launch_rows<2, 4, 1, 4>(a, s);
}

}  // namespace w4a8
