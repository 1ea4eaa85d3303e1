// dense_tiles.hip -- w4a8_gemm_epilogue for many rows: tiles of 256 x 256, or
// 128 x 128, activation rows x weight rows.
//
// The product runs on the fp8 matrix instruction, whose operands are bytes,
// and what limits it is the vector work around it: two fp32 operations per
// output and 128-group apply the group's two scales, and in this schedule they
// hardly overlap the matrix core's (counters of the 4096 x 7168 x 4096 product:
// matrix core busy 36% of the cycles, other vector instructions 42%, neither a
// fifth).  So the int4 weights are not decoded in the K loop
// (13 vector operations per 8 weights, twice over, since two waves share each
// weight row): a first pass expands them once into e4m3 codes in the
// workspace, laid out as the stages of the K loop (16 KB per 128 weight rows and
// group, swizzled as they lie in LDS), and transposes both scale matrices.
//
// A wave holds 64 weight rows x 128 (or 64) activation rows; stage g + 1 loads
// straight into LDS while stage g is multiplied, with one barrier a group, and
// one slice's results get their scales while the next slice is multiplied (173
// -> 155 us; the operands' chunk order, free of bank conflicts, 155 -> 151).  The
// weights are the first MFMA operand, so a lane holds four consecutive outputs
// of one row.  With SwiGLU a wave's 64 weight rows are 32 gate rows and their 32
// up rows.
//
// Tiles are numbered in columns of 8 row tiles and cut into 8 contiguous
// ranges, one per XCD, so that the tiles that run at the same time on one XCD
// share their rows and weights in its L2.
//
// 4096 x 7168 x 4096 with SwiGLU, N(0, 1) activations: the tiles 125 to 150 us
// (1.6 to 1.9 PFLOP/s, by the power the operands draw), the first pass 13 us;
// torch's bf16 product of that shape's square runs at 1.2 to 1.3 PFLOP/s, its fp8
// product with one scale per tensor at 3.0.
#include "api_util.hpp"
#include "dense_common.hpp"
#include "lds_direct.hpp"

#include <math.h>

namespace w4a8 {

namespace {

// Operands are laid out in units of 128 rows: a unit's codes of one group are
// 16 KB, its scales 512 bytes.
constexpr int kUnit = 128;
constexpr int kUnitCodes = kUnit * kGroup;
constexpr int kUnitScales = kUnit * 4;

// 16-byte slot of (row, chunk 0..7 of its 128 bytes): the XOR spreads what the
// lanes of one LDS cycle read (8 rows, two neighbouring chunks) over the banks
__device__ __forceinline__ int slot(int row, int chunk)
{
    return row * 8 + (chunk ^ (row & 7));
}

struct TileArgs {
    DenseArgs d;
    uint8_t* wq;  // [units_n][G][16 KB]
    float* swt;   // [units_n][G][128]
    float* sat;   // [units_m][G][128]
    int32_t G, units_m, units_n;
};

// weight row of row r of unit u (clamped into the matrix); SwiGLU: 32 gate
// rows, their 32 up rows, and so on
__device__ __forceinline__ int64_t unit_weight_row(const DenseArgs& d, int64_t u, int r)
{
    if (d.act == W4A8_ACT_SWIGLU) {
        const int64_t n = u * (kUnit / 2) + (r >> 6) * 32 + (r & 31);
        return (r & 32 ? d.N : 0) + min(n, d.N - 1);
    }
    return min(u * kUnit + r, d.N - 1);
}

}  // namespace

// Blocks [0, 4 * units_n * ceil(G/2)): two groups (a row's 128 bytes) of a
// quarter of one unit of weights; then units_n * ceil(G/8) blocks: eight
// groups of weight scales of one unit; then units_m * ceil(G/8): of activation
// scales.  Short blocks: a pass this small is bound by latency.
__global__ __launch_bounds__(256) void dense_expand_kernel(const TileArgs t)
{
    const DenseArgs& d = t.d;
    const int tid = threadIdx.x;
    const int pairs = (t.G + 1) / 2, eights = (t.G + 7) / 8;
    int b = (int)blockIdx.x;
    if (b < 4 * t.units_n * pairs) {
        // 16 packed bytes a thread: eight of one row lie in one 128-byte line
        const int r = 32 * (b & 3) + (tid >> 3), g = (tid >> 2) & 1, q = tid & 3;
        const int64_t u = (b >> 2) / pairs;
        const int group = 2 * ((b >> 2) - (int)u * pairs) + g;
        if (group >= t.G)
            return;
        const int64_t n = unit_weight_row(d, u, r);
        const v8i c = int4_to_fp8(ldg16_nt(d.w + n * (d.K / 2) + (int64_t)group * (kGroup / 2) + 16 * q));
        uint8_t* dst = t.wq + (u * t.G + group) * kUnitCodes;
        *(v4i*)(dst + 16 * slot(r, 2 * q)) = v4i{c[0], c[1], c[2], c[3]};
        *(v4i*)(dst + 16 * slot(r, 2 * q + 1)) = v4i{c[4], c[5], c[6], c[7]};
        return;
    }
    b -= 4 * t.units_n * pairs;
    const bool weights = b < t.units_n * eights;
    if (!weights)
        b -= t.units_n * eights;
    const int64_t u = b / eights;
    const int g0 = 8 * (b - (int)u * eights) + 4 * (tid >> 7), r = tid & (kUnit - 1);
    const int64_t row = weights ? unit_weight_row(d, u, r) : min(u * kUnit + r, d.M - 1);
    const float* src = (weights ? d.sw : d.sa) + row * t.G;
    float* dst = (weights ? t.swt : t.sat) + u * t.G * kUnit + r;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = g0 + i < t.G ? src[g0 + i] : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (g0 + i < t.G)
            dst[(int64_t)(g0 + i) * kUnit] = v[i];
}

namespace {

// scales of ROWS rows of one group: 256 as one 16-byte load per lane, 128 as
// two 4-byte ones (each LDS side is linear in the lane)
template <int ROWS>
__device__ __forceinline__ void lds_scales(const v4i& r, uint32_t lds, uint32_t v16, int lane, uint32_t soff)
{
    if constexpr (ROWS == 256) {
        lds_load16(r, lds, v16, soff);
    } else {
        static_assert(ROWS == 128, "one or two units");
        lds_load4(r, lds, 4 * lane, soff);
        lds_load4(r, lds + 256, 256 + 4 * lane, soff);
    }
}

}  // namespace

// WM x WN waves of 16 SL rows x 64 weight rows each.
template <int WM, int WN, int SL>
struct Tile {
    static constexpr int kBM = WM * SL * 16, kBN = WN * 64;
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int kA = 0, kW = kBM * kGroup, kSw = kW + kBN * kGroup, kSa = kSw + kBN * 4;
    static constexpr int kStage = kSa + kBM * 4;
    static constexpr int kEpiStride = 68;  // floats; 64 columns and a pad against bank conflicts
    static constexpr int kEpiWave = 64 * kEpiStride * 4;
    static constexpr int kLds = 2 * kStage > WM * WN * kEpiWave ? 2 * kStage : WM * WN * kEpiWave;
    static_assert(kBM % kUnit == 0 && kBN % kUnit == 0 && SL % 4 == 0 && kLds <= 160 * 1024, "tile");
};

template <int WM, int WN, int SL>
__global__ __launch_bounds__(64 * WM * WN, 2) void dense_tile_kernel(const TileArgs t, const int32_t tiles_m,
                                                                     const int32_t tiles_n)
{
    using L = Tile<WM, WN, SL>;
    constexpr int kWaves = WM * WN;
    constexpr int kALoads = L::kBM / 8 / kWaves;  // 1 KB loads per wave and stage
    constexpr int kWLoads = L::kBN / 8 / kWaves;
    __shared__ __attribute__((aligned(16))) uint8_t smem[L::kLds];

    const DenseArgs& d = t.d;
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, c16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int G = t.G;

    // tile of this workgroup: an eighth of the numbering per XCD
    const int total = tiles_m * tiles_n;
    const int chunk = (total + 7) / 8;
    const int id = (int)(blockIdx.x & 7) * chunk + (int)(blockIdx.x >> 3);
    if (id >= total)
        return;
    const int band = id / (8 * tiles_n);
    const int bh = min(8, tiles_m - 8 * band);
    const int in_band = id - band * 8 * tiles_n;
    const int tm = 8 * band + in_band % bh, tn = in_band / bh;

    const int64_t m0 = (int64_t)tm * L::kBM;
    const int rows = (int)min((int64_t)L::kBM, d.M - m0);
    // the tile's operands; units past the end are not read (their loads
    // return zero: the resource ends with the last unit)
    const int un = min(L::kBN / kUnit, t.units_n - tn * (L::kBN / kUnit));
    const int um = min(L::kBM / kUnit, t.units_m - tm * (L::kBM / kUnit));
    const v4i ra = sgpr_rsrc(d.a + m0 * d.K, (uint32_t)(rows * d.K));
    const v4i rw = sgpr_rsrc(t.wq + (int64_t)tn * (L::kBN / kUnit) * G * kUnitCodes, (uint32_t)((int64_t)un * G * kUnitCodes));
    const v4i rsw = sgpr_rsrc(t.swt + (int64_t)tn * L::kBN * G, (uint32_t)((int64_t)un * G * kUnitScales));
    const v4i rsa = sgpr_rsrc(t.sat + (int64_t)tm * L::kBM * G, (uint32_t)((int64_t)um * G * kUnitScales));
    uint32_t va[kALoads];
#pragma unroll
    for (int j = 0; j < kALoads; ++j) {
        const int sl = (wave * kALoads + j) * 64 + lane;
        const int r = sl >> 3, c = (sl & 7) ^ (r & 7);
        va[j] = (uint32_t)(min(r, rows - 1) * d.K + 16 * c);
    }
    uint32_t vw[kWLoads];
#pragma unroll
    for (int j = 0; j < kWLoads; ++j) {
        const int piece = wave * kWLoads + j;  // of 16 per unit
        vw[j] = (uint32_t)((piece >> 4) * G * kUnitCodes + (piece & 15) * 1024 + lane * 16);
    }
    const uint32_t vs = (uint32_t)((lane >> 5) * G * kUnitScales + (lane & 31) * 16);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)smem;
    auto issue = [&](int g, int st) {
        const uint32_t base = lds0 + (uint32_t)(st * L::kStage);
#pragma unroll
        for (int j = 0; j < kALoads; ++j)
            lds_load16(ra, base + (uint32_t)((wave * kALoads + j) * 1024), va[j], (uint32_t)g * kGroup);
#pragma unroll
        for (int j = 0; j < kWLoads; ++j)
            lds_load16(rw, base + (uint32_t)(L::kW + (wave * kWLoads + j) * 1024), vw[j], (uint32_t)g * kUnitCodes);
        if (wave == 0)
            lds_scales<L::kBN>(rsw, base + L::kSw, vs, lane, (uint32_t)g * kUnitScales);
        if (wave == kWaves - 1)
            lds_scales<L::kBM>(rsa, base + L::kSa, vs, lane, (uint32_t)g * kUnitScales);
    };

    float acc[SL][4][4];
#pragma unroll
    for (int s = 0; s < SL; ++s)
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[s][f][i] = 0.0f;

    // LDS offsets of the lane's operands in a stage; slice s and fragment f lie
    // at constant distances (16 rows do not change the swizzle)
    const uint32_t oa0 = 16 * slot(16 * SL * wm + c16, q), oa1 = 16 * slot(16 * SL * wm + c16, 4 + q);
    const uint32_t ob0 = L::kW + 16 * slot(64 * wn + c16, q), ob1 = L::kW + 16 * slot(64 * wn + c16, 4 + q);
    const uint32_t osw = L::kSw + 4 * (64 * wn + 4 * q);
    const uint32_t osa = L::kSa + 4 * (16 * SL * wm + c16);
    constexpr int kFrag = 16 * kGroup;  // bytes of 16 rows

    issue(0, 0);
    for (int g = 0; g < G; ++g) {
        wait_vmcnt<0>();
        barrier();  // stage g is whole, and nobody reads stage g - 1 any more
        if (g + 1 < G)
            issue(g + 1, (g + 1) & 1);
        const uint8_t* st = smem + (g & 1) * L::kStage;
        const uint8_t *pa0 = st + oa0, *pa1 = st + oa1, *pb0 = st + ob0, *pb1 = st + ob1;
        const uint8_t *psw = st + osw, *psa = st + osa;
        auto read = [&](const uint8_t* p0, const uint8_t* p1, int i) {
            const v4i x0 = *(const v4i*)(p0 + i * kFrag), x1 = *(const v4i*)(p1 + i * kFrag);
            return v8i{x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
        };
        v8i av = read(pa0, pa1, 0);
        v8i b[4];
        float4 sw[4];
#pragma unroll
        for (int f = 0; f < 4; ++f)
            b[f] = read(pb0, pb1, f);
        float sa = *(const float*)psa;
#pragma unroll
        for (int f = 0; f < 4; ++f)
            sw[f] = *(const float4*)(psw + 64 * f);
        // slice s is multiplied while slice s - 1 gets its scales: the vector
        // unit works on results that are already there.  The scales meet first:
        // the largest activation scale has no room for the sum alone
        v4f raw[4];
        float sa_raw = 0.0f;  // scale of the rows in raw
        auto promote = [&](int s, int f) {
            acc[s][f][0] = fmaf(raw[f][0], sw[f].x * sa_raw, acc[s][f][0]);
            acc[s][f][1] = fmaf(raw[f][1], sw[f].y * sa_raw, acc[s][f][1]);
            acc[s][f][2] = fmaf(raw[f][2], sw[f].z * sa_raw, acc[s][f][2]);
            acc[s][f][3] = fmaf(raw[f][3], sw[f].w * sa_raw, acc[s][f][3]);
        };
#pragma unroll
        for (int s = 0; s < SL; ++s) {
            v8i next = av;
            float sa_next = sa;
            if (s + 1 < SL) {
                next = read(pa0, pa1, s + 1);
                sa_next = *(const float*)(psa + 64 * (s + 1));
            }
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const v4f r = mfma16x16x128(b[f], av, v4f{0.0f, 0.0f, 0.0f, 0.0f});
                if (s > 0)
                    promote(s - 1, f);
                raw[f] = r;
            }
            sa_raw = sa;
            av = next;
            sa = sa_next;
        }
#pragma unroll
        for (int f = 0; f < 4; ++f)
            promote(SL - 1, f);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // the first slice's MFMAs
#pragma unroll
        for (int i = 0; i < 4 * (SL - 1); ++i) {
            if (i % 4 == 0)
                __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);  // the next slice's reads
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);      // one MFMA
            __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);      // one promotion
        }
    }
    // Epilogue: each wave lays 64 of its rows at a time into its own part of
    // LDS and takes them out row by row, so that the stores of a row are one
    // contiguous piece and the epilogue's code stands here once.
    barrier();  // the last stage has been read by everyone
    const bool glu = d.act == W4A8_ACT_SWIGLU;
    float* const mine = (float*)(smem + wave * L::kEpiWave);
    const int cols = glu ? 8 : 16;  // float4 columns of outputs per wave
    const int c4 = lane & (cols - 1);
    const int64_t n0 = glu ? (int64_t)tn * (L::kBN / 2) + 32 * wn + 4 * c4 : (int64_t)tn * L::kBN + 64 * wn + 4 * c4;
#pragma unroll
    for (int p = 0; p < SL / 4; ++p) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const float* v = acc[4 * p + s][f];
                *(float4*)(mine + (16 * s + c16) * L::kEpiStride + 16 * f + 4 * q) = make_float4(v[0], v[1], v[2], v[3]);
            }
        __builtin_amdgcn_wave_barrier();  // one wave: LDS operations stay in order
        const int first = 16 * SL * wm + 64 * p;
#pragma unroll 1
        for (int r = lane / cols; r < 64; r += 64 / cols) {
            if (first + r >= rows)
                break;
            const float4 y = *(const float4*)(mine + r * L::kEpiStride + 4 * c4);
            const float yv[4] = {y.x, y.y, y.z, y.w};
            float uv[4] = {0, 0, 0, 0};
            if (glu) {
                const float4 u = *(const float4*)(mine + r * L::kEpiStride + 32 + 4 * c4);
                uv[0] = u.x, uv[1] = u.y, uv[2] = u.z, uv[3] = u.w;
            }
            epilogue4(d, m0 + first + r, n0, yv, uv, load_epilogue4(d, m0 + first + r, n0));
        }
        __builtin_amdgcn_wave_barrier();
    }
}

namespace {

TileArgs plan_tiles(void* ws, const DenseArgs& d, size_t* bytes)
{
    TileArgs t = {};
    t.d = d;
    t.G = (int32_t)(d.K / kGroup);
    t.units_m = (int32_t)api::ceil_div(d.M, kUnit);
    t.units_n = (int32_t)api::ceil_div(d.N, d.act == W4A8_ACT_SWIGLU ? kUnit / 2 : kUnit);
    api::Carve c(ws);
    t.wq = c.take<uint8_t>((size_t)t.units_n * t.G * kUnitCodes);
    t.swt = c.take<float>((size_t)t.units_n * t.G * kUnit);
    t.sat = c.take<float>((size_t)t.units_m * t.G * kUnit);
    *bytes = c.used;
    return t;
}

// workgroups of the first pass
int64_t expand_blocks(const TileArgs& t)
{
    return 4 * (int64_t)t.units_n * ((t.G + 1) / 2) + ((int64_t)t.units_n + t.units_m) * ((t.G + 7) / 8);
}

// tiles along both axes; their workgroups, a multiple of the 8 XCDs
template <typename L>
int64_t tile_blocks(const TileArgs& t, int64_t& tiles_m, int64_t& tiles_n)
{
    tiles_m = api::ceil_div(t.units_m, L::kBM / kUnit), tiles_n = api::ceil_div(t.units_n, L::kBN / kUnit);
    return (tiles_m * tiles_n + 7) / 8 * 8;
}

template <int WM, int WN, int SL>
hipError_t launch_tiles(const TileArgs& t, hipStream_t s)
{
    using L = Tile<WM, WN, SL>;
    int64_t tiles_m, tiles_n;
    const dim3 grid((unsigned)tile_blocks<L>(t, tiles_m, tiles_n));
    hipLaunchKernelGGL((dense_tile_kernel<WM, WN, SL>), grid, dim3(L::kThreads), 0, s, t, (int32_t)tiles_m,
                       (int32_t)tiles_n);
    return hipGetLastError();
}

}  // namespace

namespace {

// Predicted times (us), fitted on MI355X over M 256 to 8000, K 128 to 7168, R
// 1000 to 7168.
//
// A round of 256 x 256 tiles, one per CU, takes 16 + 0.0165 K; 128 x 128
// tiles, two per CU, 10.5 + 0.0096 K (up to 256 of them, one per CU: 7 +
// 0.0073 K).  4096 x 7168 x 4096: 138 us with the large ones, 163 with the
// small; 2048 x 7168 x 4096: 128 and 79; 4000 x 512 x 4000: 26 and 28.
struct TileCost {
    double us;
    bool large;
};
TileCost tile_cost(int64_t M, int64_t K, int64_t R)
{
    const double k = (double)K;
    const double t3 = (double)(api::ceil_div(M, 256) * api::ceil_div(R, 256));
    const double t1 = (double)(api::ceil_div(M, 128) * api::ceil_div(R, 128));
    const double large = ceil(t3 / 256) * (16 + 0.0165 * k);
    const double small = t1 <= 256 ? 7 + 0.0073 * k : fmax(1.0, t1 / 512) * (10.5 + 0.0096 * k);
    return TileCost{large <= small ? large : small, large <= small};
}
int64_t weight_rows(int64_t N, int act)
{
    return act == W4A8_ACT_SWIGLU ? 2 * N : N;
}

}  // namespace

// The tiles with their first pass (a launch, 5 us and 0.38 ps a weight)
// against the few-rows kernel, whose workgroups of 32 rows x 64 weight rows
// decode the weights again for every 32 rows (4.2 ns + 3.67 ps K each, over
// all CUs; the second is 4.5 on long K, which changes the choice only near the
// border: 2048 x 7168 x 2048 74 us and 79).  Both sides measured: 768 x 7168 x 4096
// 74 us and 60, 1024 x 2048 x 7168 41 and 46, 1500 x 2048 x 2048 31 and 23, 4096 x
// 128 x 4096 22 and 40.
bool use_dense_tiles(int64_t M, int64_t K, int64_t N, int act)
{
    const int64_t R = weight_rows(N, act);
    const double k = (double)K;
    const double rows = 4 + (double)api::ceil_div(M, 32) * (double)api::ceil_div(R, 64) * (4.2e-3 + 3.67e-6 * k);
    return tile_cost(M, K, R).us + 5 + 3.8e-7 * (double)R * k < rows;
}

size_t dense_tiles_workspace(int64_t M, int64_t K, int64_t N, int act)
{
    DenseArgs d = {};
    d.M = M, d.K = K, d.N = N, d.act = act;
    size_t bytes;
    plan_tiles(nullptr, d, &bytes);
    return bytes;
}

// the first pass has 256 threads a workgroup, the small tiles as many and
// four times the large ones' workgroups
bool dense_tiles_fit(int64_t M, int64_t K, int64_t N, int act)
{
    DenseArgs d = {};
    d.M = M, d.K = K, d.N = N, d.act = act;
    size_t bytes;
    int64_t m, n;
    const TileArgs t = plan_tiles(nullptr, d, &bytes);
    return expand_blocks(t) * 256 <= UINT32_MAX && tile_blocks<Tile<2, 2, 4>>(t, m, n) * 256 <= UINT32_MAX;
}

hipError_t launch_dense_tiles(const DenseArgs& d, void* ws, hipStream_t s)
{
    size_t bytes;
    const TileArgs t = plan_tiles(ws, d, &bytes);
    hipLaunchKernelGGL(dense_expand_kernel, dim3((unsigned)expand_blocks(t)), dim3(256), 0, s, t);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    return tile_cost(d.M, d.K, weight_rows(d.N, d.act)).large ? launch_tiles<2, 4, 8>(t, s)
                                                              : launch_tiles<2, 2, 4>(t, s);
}

}  // namespace w4a8
