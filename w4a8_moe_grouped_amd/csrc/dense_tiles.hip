// dense_tiles.hip -- w4a8_gemm_epilogue for many rows: tiles of BM activation
// rows x 256 weight rows.
//
// The product runs on the fp8 matrix instruction, whose operands are bytes,
// and what limits it is the vector work around it: two fp32 operations per
// output and 128-group apply the group's two scales.  So the int4 weights are
// not decoded in the K loop (17 vector operations per 8 weights, twice over,
// since two waves share each weight row): a first pass expands them once into
// e4m3 codes in the workspace, laid out as the stages of the K loop (a 32 KB
// block per 256 weight rows and group, swizzled as it lies in LDS), and
// transposes both scale matrices into one kilobyte per tile and group.
//
// A workgroup of 8 waves in a 2 x 4 grid holds a tile, each wave BM/2 x 64
// outputs; stage g + 1 loads straight into LDS while stage g is multiplied,
// with one barrier a group.  The weights are the first MFMA operand, so a lane
// holds four consecutive outputs of one row.  With SwiGLU a wave's 64 weight
// rows are 32 gate rows and their 32 up rows.
//
// Tiles are numbered in columns of 8 row tiles and cut into 8 contiguous
// ranges, one per XCD, so that the tiles that run at the same time on one XCD
// share their rows and weights in its L2.
#include "api_util.hpp"
#include "dense_common.hpp"
#include "lds_direct.hpp"

namespace w4a8 {

namespace {

constexpr int kBN = 256;                 // weight rows per tile
constexpr int kWStage = kBN * kGroup;    // 32 KB of codes
constexpr int kScaleStage = 1024;        // 256 floats

// 16-byte slot of (row, chunk 0..7 of its 128 bytes): the XOR spreads a
// column of chunks over the banks
__device__ __forceinline__ int slot(int row, int chunk)
{
    return row * 8 + (chunk ^ (row & 7));
}

struct TileArgs {
    DenseArgs d;
    uint8_t* wq;  // [tiles_n][G][32 KB]
    float* swt;   // [tiles_n][G][256]
    float* sat;   // [tiles_m][G][256] (BM of them used)
    int32_t G, tiles_m, tiles_n, bm;
};

// weight row of row r of column tile tn (clamped into the matrix)
__device__ __forceinline__ int64_t tile_weight_row(const DenseArgs& d, int64_t tn, int r)
{
    if (d.act == W4A8_ACT_SWIGLU) {
        const int64_t n = tn * (kBN / 2) + (r >> 6) * 32 + (r & 31);
        return (r & 32 ? d.N : 0) + min(n, d.N - 1);
    }
    return min(tn * kBN + r, d.N - 1);
}

}  // namespace

// Blocks [0, tiles_n * ceil(G/2)): two groups of one column tile; then
// tiles_m * ceil(G/8) blocks: eight groups of activation scales of one row
// tile.
__global__ __launch_bounds__(256) void dense_expand_kernel(const TileArgs t)
{
    const DenseArgs& d = t.d;
    const int tid = threadIdx.x;
    const int64_t pairs = (t.G + 1) / 2;
    int64_t b = blockIdx.x;
    if (b < t.tiles_n * pairs) {
        const int64_t tn = b / pairs;
        const int g0 = 2 * (int)(b - tn * pairs);
        const int ng = min(2, t.G - g0);
        // 16 packed bytes an item: eight of one row lie in one 128-byte line
#pragma unroll 4
        for (int i = 0; i < 8; ++i) {
            const int item = i * 256 + tid;
            const int r = item >> 3, g = (item >> 2) & 1, q = item & 3;
            if (g >= ng)
                continue;
            const int64_t n = tile_weight_row(d, tn, r);
            const v8i c = int4_to_fp8(ldg16_nt(d.w + n * (d.K / 2) + (int64_t)(g0 + g) * (kGroup / 2) + 16 * q));
            uint8_t* dst = t.wq + (tn * t.G + g0 + g) * kWStage;
            *(v4i*)(dst + 16 * slot(r, 2 * q)) = v4i{c[0], c[1], c[2], c[3]};
            *(v4i*)(dst + 16 * slot(r, 2 * q + 1)) = v4i{c[4], c[5], c[6], c[7]};
        }
        const int64_t n = tile_weight_row(d, tn, tid);
        for (int g = 0; g < ng; ++g)  // the codes count units of 2^-9
            t.swt[(tn * t.G + g0 + g) * 256 + tid] = 512.0f * d.sw[n * t.G + g0 + g];
        return;
    }
    b -= t.tiles_n * pairs;
    const int64_t chunks = (t.G + 7) / 8;
    const int64_t tm = b / chunks;
    const int g0 = 8 * (int)(b - tm * chunks);
    const int64_t m = min(tm * t.bm + min(tid, t.bm - 1), d.M - 1);
    for (int g = g0; g < min(g0 + 8, t.G); ++g)
        t.sat[(tm * t.G + g) * 256 + tid] = d.sa[m * t.G + g];
}

template <int BM>
__global__ __launch_bounds__(512, 2) void dense_tile_kernel(const TileArgs t)
{
    constexpr int kAStage = BM * kGroup;
    constexpr int kStage = kAStage + kWStage + 2 * kScaleStage;
    constexpr int kSl = BM / 2 / 16;     // 16-row slices per wave
    constexpr int kALoads = BM / 64;     // 1 KB loads per wave and stage
    constexpr int kEpiStride = 68;  // floats; 64 columns and a pad against bank conflicts
    constexpr int kEpiWave = 64 * kEpiStride * 4;
    __shared__ __attribute__((aligned(16))) uint8_t smem[2 * kStage > 8 * kEpiWave ? 2 * kStage : 8 * kEpiWave];

    const DenseArgs& d = t.d;
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, c16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int G = t.G;

    // tile of this workgroup: an eighth of the numbering per XCD
    const int total = t.tiles_m * t.tiles_n;
    const int chunk = (total + 7) / 8;
    const int id = (int)(blockIdx.x & 7) * chunk + (int)(blockIdx.x >> 3);
    if (id >= total || (int)(blockIdx.x >> 3) >= chunk)
        return;
    const int band = id / (8 * t.tiles_n);
    const int bh = min(8, t.tiles_m - 8 * band);
    const int in_band = id - band * 8 * t.tiles_n;
    const int tm = 8 * band + in_band % bh, tn = in_band / bh;

    const int64_t m0 = (int64_t)tm * BM;
    const int rows = (int)min((int64_t)BM, d.M - m0);
    const v4i ra = sgpr_rsrc(d.a + m0 * d.K, (uint32_t)(rows * d.K));
    const v4i rw = sgpr_rsrc(t.wq + (int64_t)tn * G * kWStage, (uint32_t)((int64_t)G * kWStage));
    const v4i rsw = sgpr_rsrc(t.swt + (int64_t)tn * G * 256, (uint32_t)((int64_t)G * kScaleStage));
    const v4i rsa = sgpr_rsrc(t.sat + (int64_t)tm * G * 256, (uint32_t)((int64_t)G * kScaleStage));
    uint32_t va[kALoads];
#pragma unroll
    for (int j = 0; j < kALoads; ++j) {
        const int sl = (wave * kALoads + j) * 64 + lane;
        const int r = sl >> 3, c = (sl & 7) ^ (r & 7);
        va[j] = (uint32_t)(min(r, rows - 1) * d.K + 16 * c);
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)smem;
    auto issue = [&](int g, int st) {
        const uint32_t base = lds0 + (uint32_t)(st * kStage);
#pragma unroll
        for (int j = 0; j < kALoads; ++j)
            lds_load16(ra, base + (uint32_t)((wave * kALoads + j) * 1024), va[j], (uint32_t)g * kGroup);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            lds_load16(rw, base + (uint32_t)(kAStage + (wave * 4 + j) * 1024), (uint32_t)((wave * 4 + j) * 1024 + lane * 16),
                       (uint32_t)g * kWStage);
        if (wave == 0)
            lds_load16(rsw, base + kAStage + kWStage, lane * 16, (uint32_t)g * kScaleStage);
        if (wave == 4)
            lds_load16(rsa, base + kAStage + kWStage + kScaleStage, lane * 16, (uint32_t)g * kScaleStage);
    };

    float acc[kSl][4][4];
#pragma unroll
    for (int s = 0; s < kSl; ++s)
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[s][f][i] = 0.0f;

    // LDS offsets of the lane's operands in a stage; slice s and fragment f lie
    // at constant distances (16 rows do not change the swizzle)
    const uint32_t oa0 = 16 * slot(BM / 2 * wm + c16, q), oa1 = 16 * slot(BM / 2 * wm + c16, 4 + q);
    const uint32_t ob0 = kAStage + 16 * slot(64 * wn + c16, q), ob1 = kAStage + 16 * slot(64 * wn + c16, 4 + q);
    const uint32_t osw = kAStage + kWStage + 4 * (64 * wn + 4 * q);
    const uint32_t osa = kAStage + kWStage + kScaleStage + 4 * (BM / 2 * wm + c16);
    constexpr int kFrag = 16 * kGroup;  // bytes of 16 rows

    issue(0, 0);
    for (int g = 0; g < G; ++g) {
        wait_vmcnt<0>();
        barrier();  // stage g is whole, and nobody reads stage g - 1 any more
        if (g + 1 < G)
            issue(g + 1, (g + 1) & 1);
        const uint8_t* st = smem + (g & 1) * kStage;
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
        // unit works on results that are already there
        v4f raw[4];
        float sa_raw = 0.0f;  // scale of the rows in raw
        auto promote = [&](int s, int f) {
            acc[s][f][0] = fmaf(sw[f].x, raw[f][0] * sa_raw, acc[s][f][0]);
            acc[s][f][1] = fmaf(sw[f].y, raw[f][1] * sa_raw, acc[s][f][1]);
            acc[s][f][2] = fmaf(sw[f].z, raw[f][2] * sa_raw, acc[s][f][2]);
            acc[s][f][3] = fmaf(sw[f].w, raw[f][3] * sa_raw, acc[s][f][3]);
        };
#pragma unroll
        for (int s = 0; s < kSl; ++s) {
            v8i next = av;
            float sa_next = sa;
            if (s + 1 < kSl) {
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
            promote(kSl - 1, f);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // the first slice's MFMAs
#pragma unroll
        for (int i = 0; i < 4 * (kSl - 1); ++i) {
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
    float* const mine = (float*)(smem + wave * kEpiWave);
    const int cols = glu ? 8 : 16;  // float4 columns of outputs per wave
    const int c4 = lane & (cols - 1);
    const int64_t n0 = glu ? (int64_t)tn * (kBN / 2) + 32 * wn + 4 * c4 : (int64_t)tn * kBN + 64 * wn + 4 * c4;
#pragma unroll
    for (int p = 0; p < kSl / 4; ++p) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const float* v = acc[4 * p + s][f];
                *(float4*)(mine + (16 * s + c16) * kEpiStride + 16 * f + 4 * q) = make_float4(v[0], v[1], v[2], v[3]);
            }
        __builtin_amdgcn_wave_barrier();  // one wave: LDS operations stay in order
        const int first = BM / 2 * wm + 64 * p;
#pragma unroll 1
        for (int r = lane / cols; r < 64; r += 64 / cols) {
            if (first + r >= rows)
                break;
            const float4 y = *(const float4*)(mine + r * kEpiStride + 4 * c4);
            const float yv[4] = {y.x, y.y, y.z, y.w};
            float uv[4] = {0, 0, 0, 0};
            if (glu) {
                const float4 u = *(const float4*)(mine + r * kEpiStride + 32 + 4 * c4);
                uv[0] = u.x, uv[1] = u.y, uv[2] = u.z, uv[3] = u.w;
            }
            epilogue4(d, m0 + first + r, n0, yv, uv);
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
    t.bm = 256;
    const int64_t per = d.act == W4A8_ACT_SWIGLU ? kBN / 2 : kBN;
    t.tiles_m = (int32_t)api::ceil_div(d.M, t.bm);
    t.tiles_n = (int32_t)api::ceil_div(d.N, per);
    api::Carve c(ws);
    t.wq = c.take<uint8_t>((size_t)t.tiles_n * t.G * kWStage);
    t.swt = c.take<float>((size_t)t.tiles_n * t.G * 256);
    t.sat = c.take<float>((size_t)t.tiles_m * t.G * 256);
    *bytes = c.used;
    return t;
}

template <int BM>
hipError_t launch_tiles(const TileArgs& t, hipStream_t s)
{
    const int64_t total = (int64_t)t.tiles_m * t.tiles_n;
    const dim3 grid((unsigned)((total + 7) / 8 * 8));
    hipLaunchKernelGGL(dense_tile_kernel<BM>, grid, dim3(512), 0, s, t);
    return hipGetLastError();
}

}  // namespace

bool use_dense_tiles(int64_t M, int64_t K, int64_t N, int act)
{
    return M >= 512;
}

size_t dense_tiles_workspace(int64_t M, int64_t K, int64_t N, int act)
{
    DenseArgs d = {};
    d.M = M, d.K = K, d.N = N, d.act = act;
    size_t bytes;
    plan_tiles(nullptr, d, &bytes);
    return bytes;
}

hipError_t launch_dense_tiles(const DenseArgs& d, void* ws, hipStream_t s)
{
    size_t bytes;
    const TileArgs t = plan_tiles(ws, d, &bytes);
    const int64_t blocks = (int64_t)t.tiles_n * ((t.G + 1) / 2) + (int64_t)t.tiles_m * ((t.G + 7) / 8);
    hipLaunchKernelGGL(dense_expand_kernel, dim3((unsigned)blocks), dim3(256), 0, s, t);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_tiles<256>(t, s);
}

}  // namespace w4a8
