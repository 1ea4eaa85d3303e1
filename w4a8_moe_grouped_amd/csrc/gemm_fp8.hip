// gemm_fp8.hip -- the dense linear on e4m3 weights with one scale per 128 x 128
// block (w4a8_gemm_fp8):
//   out[m, n] = bf16(act(sum_g sa[m, g] sw[n/128, g] sum_{k in g} a[m, k] w[n, k] + bias[n]) + residual[m, n]).
//
// Both operands are bytes of the fp8 matrix instruction as they lie in memory,
// so both come straight into LDS (buffer_load ... lds) in their own order and no
// first pass or workspace is needed.  One instruction covers a whole 128-group
// and its sums are promoted into fp32 with the product of the two scales, one
// multiply-add per output and group; the block scale is one value for
// all of a wave's weight rows (with SwiGLU one for its gate rows, one for its up
// rows), so the product of scales is a single multiplication for 16 rows.
//
// Few rows (fp8_rows_kernel): bound by the weight bytes and by latency.  1 x 7168 x
// 10240: 13.8 us (5.3 TB/s); 64 x 8192 x 7168: 13.7 (4.4 TB/s); 333 x 1664 x 2050: 7.6.
// Many (fp8_tile_kernel): by the matrix unit, the promotion beside it and power.
// 4096 x 7168 x 8192: 228 to 258 us by the box (1.9 to 2.1 PFLOP/s; the matrix
// unit busy 53% of the cycles, other vector instructions 44%), with operands of zero 180;
// torch's product with one scale per tensor 179.
#include "api_util.hpp"
#include "dense_common.hpp"
#include "lds_direct.hpp"

#include <math.h>

namespace w4a8 {

namespace {

constexpr int kBlock = 128;  // weight rows of a scale

// 16-byte slot of (row, chunk 0..7 of its 128 bytes): the XOR spreads what the
// lanes of one LDS cycle read (8 rows, two neighbouring chunks) over the banks
__device__ __forceinline__ int slot(int row, int chunk)
{
    return row * 8 + (chunk ^ (row & 7));
}
__device__ __forceinline__ v8i read32(const uint8_t* p0, const uint8_t* p1)
{
    const v4i x0 = *(const v4i*)p0, x1 = *(const v4i*)p1;
    return v8i{x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
}

template <int MF, int NF, int D, int WAVES>
struct RowsLds {
    static constexpr int kStage = (NF + MF) * 2048;  // weights, then activations
    static constexpr int kChunk = 8;                 // groups whose scales are staged at once
    static constexpr int kScales = 256 + MF * 16 * kChunk * 4;
    static constexpr int kWave = D * kStage + kScales;
    static_assert(NF * kChunk <= 64, "one load for the weight scales");
    static_assert(MF * NF * 1024 <= kWave, "a wave's sums fit its own part");
    static_assert(WAVES * kWave <= 160 * 1024, "LDS of a CU");
};

}  // namespace

// A workgroup owns NF fragments of 16 weight rows and MF slices of 16 rows; its
// waves split K, and each streams its groups through its own ring of D stages.
// AP: pieces of 8 activation rows that are loaded (1: up to 8 rows, whose
// partners in the slice are left as they are: a row of the product only
// depends on its own).
template <int MF, int NF, bool GLU, int D, int WAVES, int AP>
__global__ __launch_bounds__(64 * WAVES) void fp8_rows_kernel(const DenseArgs a, const int32_t col_blocks)
{
    static_assert(!GLU || NF % 2 == 0, "gate and up fragments come in pairs");
    using Lds = RowsLds<MF, NF, D, WAVES>;
    constexpr int kOut = GLU ? NF / 2 : NF;  // fragments of outputs
    constexpr int kLoads = 2 * NF + AP;      // per group
    constexpr int kChunk = Lds::kChunk;
    __shared__ __attribute__((aligned(16))) uint8_t smem[WAVES * Lds::kWave];

    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, c16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = (int)(a.K / kGroup);
    const int mb = (int)blockIdx.x / col_blocks;
    const int64_t n0 = (int64_t)((int)blockIdx.x - mb * col_blocks) * (16 * kOut);
    const int64_t m0 = (int64_t)mb * (16 * MF);
    if (n0 >= a.N)  // col_blocks may be rounded up
        return;

    // the first of this wave's items of the epilogue (slice, output fragment);
    // loads of all of them here cost more than they save (333 x 1664 x 2050: 9.8 -> 11.0 us)
    const int item_s = wave / kOut, item_f = wave - item_s * kOut;
    const int64_t item_m = m0 + 16 * item_s + c16, item_n = n0 + 16 * item_f + 4 * q;
    EpiOperands pre = {};
    if (wave < MF * kOut && item_m < a.M)
        pre = load_epilogue4(a, item_m, item_n);

    // rows past the last read the last valid one
    const int rows_a = (int)min((int64_t)(16 * MF), a.M - m0);
    const int rows_w = (int)min((int64_t)(16 * kOut), a.N - n0);
    const uint32_t krow = (uint32_t)a.K, srow = (uint32_t)G * 4;
    const v4i ra = sgpr_rsrc(a.a + m0 * a.K, rows_a * krow);
    const v4i rsa = sgpr_rsrc(a.sa + m0 * G, rows_a * srow);
    const v4i rw = sgpr_rsrc(a.w + n0 * a.K, rows_w * krow);
    const v4i ru = sgpr_rsrc(a.w + (n0 + (GLU ? a.N : 0)) * a.K, rows_w * krow);

    uint8_t* const mine = smem + wave * Lds::kWave;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)mine;
    uint32_t vw[2 * kOut], va[AP];
#pragma unroll
    for (int j = 0; j < 2 * kOut; ++j) {
        const int r = 8 * j + (lane >> 3), c = (lane & 7) ^ (r & 7);
        vw[j] = (uint32_t)min(r, rows_w - 1) * krow + 16 * c;
    }
#pragma unroll
    for (int j = 0; j < AP; ++j) {
        const int r = 8 * j + (lane >> 3), c = (lane & 7) ^ (r & 7);
        va[j] = (uint32_t)min(r, rows_a - 1) * krow + 16 * c;
    }
    auto issue = [&](int g, int st) {
        const uint32_t base = lds0 + (uint32_t)(st * Lds::kStage);
#pragma unroll
        for (int j = 0; j < 2 * NF; ++j)
            lds_load16(j < 2 * kOut ? rw : ru, base + 1024u * j, vw[j % (2 * kOut)], (uint32_t)g * kGroup);
#pragma unroll
        for (int j = 0; j < AP; ++j)
            lds_load16(ra, base + 1024u * (2 * NF + j), va[j], (uint32_t)g * kGroup);
    };
    // scales of groups c0 .. c0 + 7: of the weight fragments as [fragment][8],
    // then of the activation rows as [row][8]
    const int frag = min(lane >> 3, NF - 1);
    const int64_t frag_row = (GLU && frag >= kOut ? a.N + 16 * (frag - kOut) : 16 * frag) + n0;
    const int64_t last_row = (GLU ? 2 * a.N : a.N) - 1;
    const uint32_t block0 = (uint32_t)(n0 / kBlock);
    const v4i rsw = sgpr_rsrc(a.sw + (int64_t)block0 * G, (uint32_t)(((last_row / kBlock) + 1 - block0) * srow));
    const uint32_t vsw = (uint32_t)(min(frag_row, last_row) / kBlock - block0) * srow;
    auto issue_scales = [&](int c0) {
        const uint32_t base = lds0 + (uint32_t)(D * Lds::kStage);
        const uint32_t g = 4u * (uint32_t)min(c0 + (lane & 7), G - 1);
        lds_load4(rsw, base, vsw + g, 0);
#pragma unroll
        for (int j = 0; j < AP; ++j)
            lds_load4(rsa, base + 256u + 256u * j, (uint32_t)min(8 * j + (lane >> 3), rows_a - 1) * srow + g, 0);
    };

    v4f acc[MF][NF];
#pragma unroll
    for (int s = 0; s < MF; ++s)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            acc[s][f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const float* const sw_lds = (const float*)(mine + D * Lds::kStage);
    const float* const sa_lds = sw_lds + 64;
    auto multiply = [&](const uint8_t* st, int gi) {  // group gi of the chunk
        v8i b[NF];
        float sw[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const uint8_t* w = st + 2048 * f;
            b[f] = read32(w + 16 * slot(c16, q), w + 16 * slot(c16, 4 + q));
            sw[f] = sw_lds[f * kChunk + gi];
        }
#pragma unroll
        for (int s = 0; s < MF; ++s) {
            const uint8_t* x = st + 2048 * (NF + s);
            const v8i av = read32(x + 16 * slot(c16, q), x + 16 * slot(c16, 4 + q));
            const float sa = sa_lds[(16 * s + c16) * kChunk + gi];
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const v4f raw = mfma16x16x128(b[f], av, v4f{0.0f, 0.0f, 0.0f, 0.0f});
                const float both = sw[f] * sa;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[s][f][i] = fmaf(raw[i], both, acc[s][f][i]);
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
        int st = 0;
        for (int i = 0; i < n; ++i) {
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

// Tiles that a launch takes: `count` from number `first` on, of tiles_m x
// tiles_n whose height is `rows`, each as `split` parts along the rows.
struct TileGrid {
    int32_t tiles_m, tiles_n, rows, first, count, split;
};

// WM x WN waves of 16 SL rows x 64 weight rows each.  Scales: QUAD (K % 512
// == 0) four groups at once, which is one 16-byte load a row; else a group at
// a time.
template <int WM, int WN, int SL, bool QUAD>
struct Tile {
    static constexpr int kBM = WM * SL * 16, kBN = WN * 64;
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int kW = kBM * kGroup, kStage = kW + kBN * kGroup;
    static constexpr int kPer = QUAD ? 16 : 4;                      // bytes of a row's scales
    static constexpr int kSw = kBM * kPer, kScales = kSw + 64 * kPer;  // rows, then 64 lanes of weight scales
    static constexpr int kRing = 2 * (kStage + kScales);
    static constexpr int kLds = kRing > WM * WN * kTileWaveLds ? kRing : WM * WN * kTileWaveLds;
    static_assert(kBM % 64 == 0 && kBN % 64 == 0 && SL % 4 == 0 && kLds <= 160 * 1024, "tile");
    static_assert(kBM / 64 + 1 <= WM * WN, "one wave for each scale load");
};

}  // namespace

template <int WM, int WN, int SL, bool QUAD>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_tile_kernel(const DenseArgs d, const TileGrid t)
{
    using L = Tile<WM, WN, SL, QUAD>;
    constexpr int kWaves = WM * WN;
    constexpr int kALoads = L::kBM / 8 / kWaves;  // 1 KB loads per wave and stage
    constexpr int kWLoads = L::kBN / 8 / kWaves;
    __shared__ __attribute__((aligned(16))) uint8_t smem[L::kLds];

    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, c16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int G = (int)(d.K / kGroup);
    const bool glu = d.act == W4A8_ACT_SWIGLU;

    // tile of this workgroup: an eighth of the numbering per XCD, in columns of 8 row tiles
    const int total = t.count * t.split;
    const int chunk = (total + 7) / 8;
    const int part = (int)(blockIdx.x & 7) * chunk + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= chunk || part >= total)
        return;
    const int id = t.first + part / t.split;
    const int band = id / (8 * t.tiles_n);
    const int bh = min(8, t.tiles_m - 8 * band);
    const int in_band = id - band * 8 * t.tiles_n;
    const int tm = 8 * band + in_band % bh, tn = in_band / bh;

    const int64_t m0 = (int64_t)tm * t.rows + (part % t.split) * L::kBM;
    if (m0 >= d.M)
        return;
    const int rows = (int)min((int64_t)L::kBM, d.M - m0);
    // weight rows of the tile: kBN from n0; with SwiGLU runs of 32 gate rows and
    // their 32 up rows, kBN / 2 outputs from n0.  Rows past the last read the last.
    const int64_t n0 = (int64_t)tn * (glu ? L::kBN / 2 : L::kBN);
    const int rows_w = (int)min((int64_t)(glu ? L::kBN / 2 : L::kBN), d.N - n0);
    const v4i ra = sgpr_rsrc(d.a + m0 * d.K, (uint32_t)(rows * d.K));
    const v4i rw = sgpr_rsrc(d.w + n0 * d.K, (uint32_t)(rows_w * d.K));
    const v4i ru = sgpr_rsrc(d.w + (n0 + (glu ? d.N : 0)) * d.K, (uint32_t)(rows_w * d.K));
    uint32_t va[kALoads], vw[kWLoads];
#pragma unroll
    for (int j = 0; j < kALoads; ++j) {
        const int r = (wave * kALoads + j) * 8 + (lane >> 3), c = (lane & 7) ^ (r & 7);
        va[j] = (uint32_t)(min(r, rows - 1) * d.K + 16 * c);
    }
#pragma unroll
    for (int j = 0; j < kWLoads; ++j) {
        const int r = (wave * kWLoads + j) * 8 + (lane >> 3), c = (lane & 7) ^ (r & 7);
        const int n = glu ? (r >> 6) * 32 + (r & 31) : r;
        vw[j] = (uint32_t)(min(n, rows_w - 1) * d.K + 16 * c);
    }
    // scales: wave w < kBM / 64 those of 64 rows, the last wave those of the
    // weights, lane 2 wn + half the block of the wave's rows of that half
    const uint32_t srow = (uint32_t)G * 4;
    const int64_t rows_all = glu ? 2 * d.N : d.N;
    const int64_t lane_n = n0 + (glu ? 32 : 64) * min(lane >> 1, WN - 1);
    const int64_t lane_row = min(lane_n, d.N - 1) + (glu && (lane & 1) ? d.N : 0);
    const uint32_t block0 = (uint32_t)(n0 / kBlock);
    const v4i rsa = sgpr_rsrc(d.sa + m0 * G, (uint32_t)rows * srow);
    const v4i rsw = sgpr_rsrc(d.sw + (int64_t)block0 * G, (uint32_t)((rows_all - 1) / kBlock + 1 - block0) * srow);
    const uint32_t vsa = (uint32_t)min(wave * 64 + lane, rows - 1) * srow;
    const uint32_t vsw = (uint32_t)(lane_row / kBlock - block0) * srow;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)smem;
    // a quarter of the loads of stage g (past the last: the last again, which nobody reads)
    auto issue = [&](int g, int part) {
        const uint32_t base = lds0 + (uint32_t)((g & 1) * L::kStage), off = (uint32_t)min(g, G - 1) * kGroup;
#pragma unroll
        for (int j = part * kALoads / 4; j < (part + 1) * kALoads / 4; ++j)
            lds_load16(ra, base + (uint32_t)((wave * kALoads + j) * 1024), va[j], off);
#pragma unroll
        for (int j = part * kWLoads / 4; j < (part + 1) * kWLoads / 4; ++j) {
            const bool up = glu && ((wave * kWLoads + j) & 4);  // pieces of 8 rows
            lds_load16(up ? ru : rw, base + (uint32_t)(L::kW + (wave * kWLoads + j) * 1024), vw[j], off);
        }
    };
    // the scales of group g, with QUAD of groups g .. g + 3
    auto issue_scales = [&](int g) {
        const uint32_t sc = lds0 + (uint32_t)(2 * L::kStage + ((QUAD ? g >> 2 : g) & 1) * L::kScales);
        if (wave < L::kBM / 64) {
            if (QUAD)
                lds_load16(rsa, sc + (uint32_t)wave * 1024, vsa, 4u * (uint32_t)g);
            else
                lds_load4(rsa, sc + (uint32_t)wave * 256, vsa, 4u * (uint32_t)g);
        }
        if (wave == kWaves - 1) {
            if (QUAD)
                lds_load16(rsw, sc + L::kSw, vsw, 4u * (uint32_t)g);
            else
                lds_load4(rsw, sc + L::kSw, vsw, 4u * (uint32_t)g);
        }
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
    const uint32_t osa = L::kPer * (16 * SL * wm + c16), osw = L::kSw + L::kPer * 2 * wn;
    constexpr int kFrag = 16 * kGroup;  // bytes of 16 rows

    // The order of the loop's instructions is fixed here (the compiler's own put
    // each promotion right behind its product, with waits of 12 cycles in
    // between: 4096 x 7168 x 8192 took 314 us instead of 228).  A slice's products go out one by
    // one, each behind the promotion of the product four before it, and the next
    // slice's operands are read beneath them.  The barrier of a group stands before
    // its last slice, whose operands are in registers: behind it the next stage is whole, and
    // nobody reads this one any more, so the last slice's products cover the next
    // group's first reads (each b[f] is read as its last product is out) and the
    // loads of the stage after it.
    v4f raw[4];
    float both[2] = {0.0f, 0.0f};  // scales of the rows in raw
#pragma unroll
    for (int f = 0; f < 4; ++f)
        raw[f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    auto promote = [&](int s, int f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[s][f][i] = fmaf(raw[f][i], both[f >> 1], acc[s][f][i]);
    };
    auto stage_at = [&](int g) { return (const uint8_t*)smem + (g & 1) * L::kStage; };
    auto scales_at = [&](int g) {
        return (const uint8_t*)smem + 2 * L::kStage + ((QUAD ? g >> 2 : g) & 1) * L::kScales + (QUAD ? 4 * (g & 3) : 0);
    };
#pragma unroll
    for (int part = 0; part < 4; ++part)
        issue(0, part);
    issue_scales(0);
    wait_vmcnt<0>();
    barrier();
#pragma unroll
    for (int part = 0; part < 4; ++part)
        issue(1, part);
    const uint8_t *st = stage_at(0), *sc = scales_at(0);
    v8i av = read32(st + oa0, st + oa1), b[4];
#pragma unroll
    for (int f = 0; f < 4; ++f)
        b[f] = read32(st + ob0 + f * kFrag, st + ob1 + f * kFrag);
    float sw[2] = {*(const float*)(sc + osw), *(const float*)(sc + osw + L::kPer)};
    float sa = *(const float*)(sc + osa);
    auto multiply = [&](int g, bool more) {
#pragma unroll
        for (int s = 0; s < SL; ++s) {
            v8i next = av;
            float sa_next = sa, sw_next[2] = {sw[0], sw[1]};
            if (s + 1 < SL) {
                next = read32(st + oa0 + (s + 1) * kFrag, st + oa1 + (s + 1) * kFrag);
                sa_next = *(const float*)(sc + osa + 16 * L::kPer * (s + 1));
            } else if (more) {
                wait_vmcnt<0>();
                barrier();
                st = stage_at(g + 1);
                sc = scales_at(g + 1);
                next = read32(st + oa0, st + oa1);
                sa_next = *(const float*)(sc + osa);
                sw_next[0] = *(const float*)(sc + osw);
                sw_next[1] = *(const float*)(sc + osw + L::kPer);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                promote(s > 0 ? s - 1 : SL - 1, f);
                __builtin_amdgcn_sched_barrier(0);
                raw[f] = mfma16x16x128(b[f], av, v4f{0.0f, 0.0f, 0.0f, 0.0f});
                __builtin_amdgcn_sched_barrier(0);
                if (s + 1 == SL && more) {
                    b[f] = read32(st + ob0 + f * kFrag, st + ob1 + f * kFrag);
                    issue(g + 2, f);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            both[0] = sw[0] * sa;
            both[1] = sw[1] * sa;
            av = next;
            sa = sa_next;
            sw[0] = sw_next[0];
            sw[1] = sw_next[1];
        }
    };
    for (int g = 0; g + 1 < G; ++g) {
        // the scales that the group after the next barrier needs first
        if (!QUAD)
            issue_scales(g + 1);
        else if ((g & 3) == 2 && g + 2 < G)
            issue_scales(g + 2);
        multiply(g, true);
    }
    multiply(G - 1, false);
#pragma unroll
    for (int f = 0; f < 4; ++f)
        promote(SL - 1, f);
    wait_vmcnt<0>();
    barrier();  // the last stage has been read by everyone
    store_tile<SL>(d, acc, (float*)(smem + wave * kTileWaveLds), lane, rows, 16 * SL * wm, m0, n0 + (glu ? 32 : 64) * wn);
}

namespace {

int64_t weight_rows(const DenseArgs& d)
{
    return d.act == W4A8_ACT_SWIGLU ? 2 * d.N : d.N;
}

enum Kernel { kRows12, kRows14, kRows22, kRows24, kRows44, kRows44Two, kTiles128, kTiles128x256, kTiles256, kKernels };

// Predicted times (us), fitted on MI355X (over 1071 sizes, M 1 to 4096, K 512 to
// 8192, R 256 to 10240, the kernel they choose takes 3% more than the best on
// average, 14% at the 95th percentile).  Few rows, blocks of 16 mf rows x 16 nf
// weight rows: the latency of one block and the throughput of all, per_cu of
// them a CU at a time, joined as the fourth root of the sum of fourth powers.  Tiles: rounds.
struct Cost {
    int mf, nf, per_cu;
    double latency, latency_k, round, round_k;
};
constexpr Cost kCost[kKernels] = {
    {1, 2, 2, 8.0, 0.00004, 1.3, 0.00197},  {1, 4, 1, 6.8, 0.0005, 2.3, 0.00149},  {2, 2, 2, 7.3, 0.00028, 2.6, 0.00192},
    {2, 4, 1, 6.7, 0.00069, 3.7, 0.00143},  {4, 4, 1, 6.5, 0.0011, 4.2, 0.00186},  {4, 4, 2, 6.4, 0.00166, 4.9, 0.00348},
    {8, 8, 2, 7.4, 0.00485, 10.3, 0.0083},  {8, 16, 1, 0.0, 0.0, 8.1, 0.0064},     {16, 16, 1, 0.0, 0.0, 11.4, 0.0101},
};

double cost(const DenseArgs& d, int kernel)
{
    const Cost& c = kCost[kernel];
    const double k = (double)d.K, cus = 256.0;
    const double blocks = (double)api::ceil_div(d.M, 16 * c.mf) * (double)api::ceil_div(weight_rows(d), 16 * c.nf);
    const double rounds = blocks / (cus * c.per_cu), latency = c.latency + c.latency_k * k, round = c.round + c.round_k * k;
    switch (kernel) {
    case kTiles128: return blocks <= cus ? latency : fmax(1.0, rounds) * round;
    case kTiles128x256: return ceil(rounds) * round;
    case kTiles256: {
        const double full = floor(rounds), rest = rounds - full;
        const Cost& half = kCost[kTiles128x256];
        return full * round + (rest == 0.0 ? 0.0 : full > 0 && rest <= 0.5 ? half.round + half.round_k * k : round);
    }
    default: {
        const double a = latency * latency, b = rounds * round * rounds * round;
        return sqrt(sqrt(a * a + b * b));
    }
    }
}

int choose(const DenseArgs& d)
{
    int best = 0;
    double least = INFINITY;
    // more than 128 rows would read the weights many times over
    for (int i = d.M > 128 ? kRows22 : kRows12; i < kKernels; ++i) {
        const double t = cost(d, i);
        if (t < least)
            best = i, least = t;
    }
    return best;
}

// Columns of blocks as fp8_rows_kernel numbers them.  Of several row blocks those
// of one column share weight rows: with a multiple of 8 columns they run on one
// XCD, whose L2 then serves all but the first (96 x 8192 x 5000: 21.7 -> 13.4 us,
// 200 x 4096 x 1500: 12.4 -> 9.4, 333 x 1664 x 2050: 9.1 -> 7.6).
int64_t numbered_columns(int64_t row_blocks, int64_t cols)
{
    return row_blocks > 1 && cols >= 16 ? (cols + 7) / 8 * 8 : cols;
}

template <int MF, int NF, int D, int WAVES, int AP>
hipError_t launch_rows(const DenseArgs& a, hipStream_t s)
{
    const bool glu = a.act == W4A8_ACT_SWIGLU;
    const int64_t row_blocks = api::ceil_div(a.M, 16 * MF);
    const int64_t col_blocks = numbered_columns(row_blocks, api::ceil_div(a.N, 16 * (glu ? NF / 2 : NF)));
    const dim3 grid((unsigned)(col_blocks * row_blocks)), block(64 * WAVES);
    if (glu)
        hipLaunchKernelGGL((fp8_rows_kernel<MF, NF, true, D, WAVES, AP>), grid, block, 0, s, a, (int32_t)col_blocks);
    else
        hipLaunchKernelGGL((fp8_rows_kernel<MF, NF, false, D, WAVES, AP>), grid, block, 0, s, a, (int32_t)col_blocks);
    return hipGetLastError();
}

template <int WM, int WN, int SL>
hipError_t launch_tiles(const DenseArgs& d, const TileGrid& t, hipStream_t s)
{
    using L = Tile<WM, WN, SL, true>;
    const dim3 grid((unsigned)((t.count * t.split + 7) / 8 * 8));  // a multiple of the 8 XCDs
    if (d.K % (4 * kGroup) == 0)
        hipLaunchKernelGGL((fp8_tile_kernel<WM, WN, SL, true>), grid, dim3(L::kThreads), 0, s, d, t);
    else
        hipLaunchKernelGGL((fp8_tile_kernel<WM, WN, SL, false>), grid, dim3(L::kThreads), 0, s, d, t);
    return hipGetLastError();
}

TileGrid all_tiles(const DenseArgs& d, int bm, int bn)
{
    TileGrid t = {};
    t.tiles_m = (int32_t)api::ceil_div(d.M, bm);
    t.tiles_n = (int32_t)api::ceil_div(weight_rows(d), bn);
    t.rows = bm;
    t.count = t.tiles_m * t.tiles_n;
    t.split = 1;
    return t;
}

}  // namespace

size_t gemm_fp8_workspace(int64_t, int64_t, int64_t, int)
{
    return 0;
}

// whether every launch of the call stays below 2^32 threads (and its count of
// workgroups, twice that of the tiles at most, below 2^31)
bool gemm_fp8_fits(int64_t M, int64_t K, int64_t N, int act)
{
    DenseArgs d = {};
    d.M = M, d.K = K, d.N = N, d.act = act;
    const int kernel = choose(d);
    const Cost& c = kCost[kernel];
    // workgroups have 512 threads at most
    const int64_t row_blocks = api::ceil_div(M, 16 * c.mf);
    const int64_t blocks = row_blocks * numbered_columns(row_blocks, api::ceil_div(weight_rows(d), 16 * c.nf));
    return blocks < ((int64_t)1 << 23) - 8;
}

hipError_t launch_gemm_fp8(const DenseArgs& d, void*, hipStream_t s)
{
    switch (choose(d)) {
    case kRows12: return d.M <= 8 ? launch_rows<1, 2, 1, 8, 1>(d, s) : launch_rows<1, 2, 1, 8, 2>(d, s);
    case kRows14: return d.M <= 8 ? launch_rows<1, 4, 2, 4, 1>(d, s) : launch_rows<1, 4, 2, 4, 2>(d, s);
    case kRows22: return launch_rows<2, 2, 1, 8, 4>(d, s);
    case kRows24: return launch_rows<2, 4, 1, 8, 4>(d, s);
    case kRows44: return launch_rows<4, 4, 1, 8, 8>(d, s);
    case kRows44Two: return launch_rows<4, 4, 1, 4, 8>(d, s);
    case kTiles128: return launch_tiles<2, 2, 4>(d, all_tiles(d, 128, 128), s);
    case kTiles128x256: return launch_tiles<2, 4, 4>(d, all_tiles(d, 128, 256), s);
    default: {
        // A last round that is at most half full goes out as tiles of half the
        // size, twice as many: 4096 x 2048 x 5000 (320 tiles) 75 -> 67 us,
        // 4000 x 4096 x 9000 185 -> 172, 4096 x 7168 x 10240 346 -> 338.
        TileGrid t = all_tiles(d, 256, 256);
        const int32_t rest = t.count % 256;
        if (t.count < 256 || rest == 0 || rest > 128)
            return launch_tiles<2, 4, 8>(d, t, s);
        t.count -= rest;
        const hipError_t e = launch_tiles<2, 4, 8>(d, t, s);
        if (e != hipSuccess)
            return e;
        t.first = t.count;
        t.count = rest;
        t.split = 2;
        return launch_tiles<2, 4, 4>(d, t, s);
    }
    }
}

}  // namespace w4a8
