// rope.hip -- rotary positions (w4a8_rope) and the append to a paged cache that
// rotates on the way (w4a8_kv_append).
//
// Bound by bytes: each element is read once and written once.  A wave takes
// one token and some of its rows (the heads of q, then k, then v).  Its lanes
// first make the token's cosines and sines, one pair each, into the wave's own
// part of LDS, so that their 40 operations are done once for all the wave's
// rows; then 8 lanes (16 for D > 128) hold a row in chunks of 16 bytes,
// neighbouring lanes' chunks side by side; for pairs of halves a lane holds both
// partners, so that no element crosses lanes.
//
// The angle's turns are reduced in twice 64 bits (at position 10^6 an fp32 angle is
// off by 0.03, at 2^31 one of 64 bits by more than sine and cosine are), sine and cosine of what is left, at most an eighth of a turn,
// by their Taylor series in fp32.
//
// 16384 tokens x 40 heads of 128, fp32: 127 us (5.3 TB/s, a copy 5.1; with 32
// contiguous bytes a lane 154); append of 16384 tokens, 64 + 2 x 8 heads, to
// e4m3: 124 us (5.1 TB/s); 64 tokens: 3.6 and 4.4 us, two memory latencies.
// Halves that are no whole chunks read partners one by one (16384 x 72 x 80, bf16,
// 20 of it turned: 144 us, interleaved 77).
#include "common.hpp"
#include "internal.hpp"
#include "w4a8.h"

namespace w4a8 {

namespace {

constexpr int kWaves = 4;       // per workgroup
constexpr int kMaxPairs = 128;  // D <= 256
enum Layout { kPairs = 0, kHalves = 1, kHalvesAny = 2 };

// cos and sin of the angle pos * f, times m.  The product and its turns are kept as
// two numbers of 64 bits each, of which whole turns go first: one would be off by
// 2^-53 of the angle, 2.4e-7 for each radian a position at position 2^31.
__device__ __forceinline__ float2 cos_sin(double pos, double f, float m)
{
#pragma clang fp contract(off)  // turns - rint(turns) as one operation on the product would hold `rest` already
    constexpr double kTurn = 0.15915494309189535, kTurnRest = -9.839338337591243e-18;  // 1 / (2 pi)
    const double angle = pos * f, angle_rest = fma(pos, f, -angle);
    double turns = angle * kTurn;
    double rest = fma(angle, kTurn, -turns) + fma(angle, kTurnRest, angle_rest * kTurn);
    turns -= rint(turns);
    rest -= rint(rest);
    turns += rest;
    const double quarter = rint(4.0 * turns);
    const float x = (float)((turns - 0.25 * quarter) * 6.283185307179586477);
    const int n = (int)quarter & 3;
    const float z = x * x;
    // |x| <= pi/4: the first terms left out are below 2e-9
    float s = fmaf(z, 1.0f / 362880, -1.0f / 5040);
    s = fmaf(z, s, 1.0f / 120);
    s = fmaf(z, s, -1.0f / 6);
    s = fmaf(z * x, s, x);
    float c = fmaf(z, -1.0f / 3628800, 1.0f / 40320);
    c = fmaf(z, c, -1.0f / 720);
    c = fmaf(z, c, 1.0f / 24);
    c = fmaf(z, c, -0.5f);
    c = fmaf(z, c, 1.0f);
    const float cq = n & 1 ? s : c, sq = n & 1 ? c : s;
    return make_float2(m * (n == 1 || n == 2 ? -cq : cq), m * (n >= 2 ? -sq : sq));
}

// 16 bytes of a row
template <int TYPE>
struct Elem;
template <>
struct Elem<W4A8_TYPE_FP32> {
    typedef float T;
    static __device__ __forceinline__ float get(const v4i& r, int i) { return __int_as_float(r[i]); }
    static __device__ __forceinline__ v4i pack(const float* f)
    {
        return v4i{__float_as_int(f[0]), __float_as_int(f[1]), __float_as_int(f[2]), __float_as_int(f[3])};
    }
};
template <>
struct Elem<W4A8_TYPE_BF16> {
    typedef __bf16 T;
    static __device__ __forceinline__ float get(const v4i& r, int i)
    {
        const uint32_t d = (uint32_t)r[i >> 1];
        return __uint_as_float(i & 1 ? d & 0xFFFF0000u : d << 16);
    }
    static __device__ __forceinline__ v4i pack(const float* f)
    {
        return v4i{(int)f32x2_to_bf16x2(f[0], f[1]), (int)f32x2_to_bf16x2(f[2], f[3]), (int)f32x2_to_bf16x2(f[4], f[5]),
                   (int)f32x2_to_bf16x2(f[6], f[7])};
    }
};
template <>
struct Elem<W4A8_TYPE_FP16> {
    typedef _Float16 T;
    static __device__ __forceinline__ float get(const v4i& r, int i) { return (float)__builtin_bit_cast(v8h, r)[i]; }
    static __device__ __forceinline__ v4i pack(const float* f)
    {
        v8h h;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h[i] = (_Float16)f[i];
        return __builtin_bit_cast(v4i, h);
    }
};

}  // namespace

// LANES lanes a row (at least D / 16), PASSES rows for each of a wave's 64 / LANES groups.
template <int TYPE, int LAYOUT, int LANES, int PASSES, bool QUANT>
__global__ __launch_bounds__(64 * kWaves) void rope_kernel(const RopeArgs a, const int32_t parts)
{
    using E = Elem<TYPE>;
    typedef typename E::T T;
    constexpr int kGroups = 64 / LANES;
    constexpr int kChunk = 16 / sizeof(T), kChunks = 16 / kChunk;  // elements of 16 bytes, and their number in a lane
    __shared__ float2 table[kWaves][kMaxPairs];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t item = blockIdx.x * kWaves + wave;  // below 2^26
    const int64_t t = item / (uint32_t)parts;
    if (t >= a.T)
        return;
    const int c = lane & (LANES - 1);
    const int first = (int)(item - (uint32_t)t * parts) * (kGroups * PASSES);  // of the wave's rows
    const int row0 = first + lane / LANES;
    const int rows = a.q_heads + 2 * a.kv_heads;
    const int half = a.R / 2;

    // this lane's chunks of a row, neighbouring lanes' side by side; the last may lie past its end
    int e[kChunks];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        e[j] = kChunk * (c + LANES * j);
        if (LAYOUT == kHalves) {  // two by two: partners, then what is not turned
            const int pair = c + LANES * (j / 2), turned = half / kChunk;
            e[j] = pair < turned ? kChunk * pair + (j & 1) * half : a.R + kChunk * (2 * (pair - turned) + (j & 1));
        }
    }

    auto source = [&](int row) {
        const bool is_q = row < a.q_heads, is_k = row < a.q_heads + a.kv_heads;
        const Rows& r = is_q ? a.q : is_k ? a.k : a.v;
        const int head = is_q ? row : is_k ? row - a.q_heads : row - a.q_heads - a.kv_heads;
        return (const T*)r.p + t * r.ts + head * r.hs;
    };
    v4i raw[PASSES][kChunks];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int row = row0 + p * kGroups;
        if (row < rows) {
            const T* src = source(row);
#pragma unroll
            for (int j = 0; j < kChunks; ++j)
                if (e[j] < a.D)
                    raw[p][j] = ldg16(src + e[j]);
        }
    }
    int64_t slot = -1;
    if (a.kv_heads > 0)
        slot = a.slots[t];
    if (half > 0) {
        const double pos = (double)a.positions[t];
        for (int i = lane; i < half; i += 64)
            table[wave][i] = cos_sin(pos, a.frequencies[i], a.magnitude);
    }
    __builtin_amdgcn_wave_barrier();  // one wave: LDS operations stay in order
    const float2* cs = table[wave];
    const bool kept = slot >= 0 && slot < a.num_slots;
    const bool narrow = (uint64_t)(slot | a.page_size) <= UINT32_MAX;  // a division in 64 bits is a long one
    const int64_t page = !kept ? 0 : narrow ? (uint32_t)slot / (uint32_t)a.page_size : slot / a.page_size;
    const int64_t place = kept ? slot - page * a.page_size : 0;

#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        if (first + p * kGroups >= rows)
            break;
        const int row = row0 + p * kGroups;
        const bool is_q = row < a.q_heads, is_k = !is_q && row < a.q_heads + a.kv_heads;
        const bool live = row < rows && (is_q || kept);
        float f[16];
#pragma unroll
        for (int j = 0; j < kChunks; ++j)
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
                f[kChunk * j + i] = live && e[j] < a.D ? E::get(raw[p][j], i) : 0.0f;
        if (live && (is_q || is_k) && half > 0) {
            if (LAYOUT == kHalves) {
#pragma unroll
                for (int j = 0; j < kChunks; j += 2) {
                    if (e[j] < half) {
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) {
                            const float2 w = cs[e[j] + i];
                            const float x = f[kChunk * j + i], y = f[kChunk * (j + 1) + i];
                            f[kChunk * j + i] = x * w.x - y * w.y;
                            f[kChunk * (j + 1) + i] = fmaf(x, w.y, y * w.x);
                        }
                    }
                }
            } else if (LAYOUT == kPairs) {
#pragma unroll
                for (int j = 0; j < kChunks; ++j)
#pragma unroll
                    for (int i = 0; i < kChunk; i += 2) {
                        if (e[j] + i < a.R) {
                            const float2 w = cs[(e[j] + i) / 2];
                            const float x = f[kChunk * j + i], y = f[kChunk * j + i + 1];
                            f[kChunk * j + i] = x * w.x - y * w.y;
                            f[kChunk * j + i + 1] = fmaf(x, w.y, y * w.x);
                        }
                    }
            } else {
                // halves that are no whole chunks: the partner, element by element
                const T* src = source(row);
#pragma unroll
                for (int j = 0; j < kChunks; ++j)
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) {
                        const int at = e[j] + i;
                        if (at < a.R) {
                            const bool first = at < half;
                            const float2 w = cs[first ? at : at - half];
                            const float x = f[kChunk * j + i], y = (float)src[first ? at + half : at - half];
                            f[kChunk * j + i] = first ? x * w.x - y * w.y : fmaf(y, w.y, x * w.x);
                        }
                    }
            }
        }
        if (is_q && live) {
            T* dst = (T*)a.q_out + t * a.qo_ts + row * a.qo_hs;
#pragma unroll
            for (int j = 0; j < kChunks; ++j)
                if (e[j] < a.D)
                    *(v4i*)(dst + e[j]) = E::pack(f + kChunk * j);
        }
        if (a.kv_heads == 0)
            continue;
        const CacheRows& out = is_k ? a.kc : a.vc;
        const int head = is_k ? row - a.q_heads : row - a.q_heads - a.kv_heads;
        const int64_t at = page * out.ps + place * out.ts + head * out.hs;
        static_assert(!QUANT || kChunks == 2, "codes come from 2-byte types");
        if constexpr (!QUANT) {
            if (!is_q && live) {
#pragma unroll
                for (int j = 0; j < kChunks; ++j)
                    if (e[j] < a.D)
                        *(v4i*)((T*)out.p + at + e[j]) = E::pack(f + kChunk * j);
            }
        } else {
            // the row's maximum; a NaN stays one
            float amax = 0.0f;
            bool nan = false;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                amax = fmaxf(amax, fabsf(f[i]));
                nan |= f[i] != f[i];
            }
            amax = group_max<LANES>(nan ? __builtin_inff() : amax);
            float bad = group_max<LANES>(nan ? 1.0f : 0.0f);
            const float amax_c = clamp_amax(amax);
            const float inv = recip448(amax_c);
            const bool far = __any(amax == __builtin_inff());
            if (!is_q && live) {
                uint8_t* dst = (uint8_t*)out.p + at;
                uint32_t q[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    q[i] = cvt_e4m3x2(f[2 * i] * inv, f[2 * i + 1] * inv);
                // infinity times 0 and NaN, which the conversion's clamp takes for -448: their code is NaN's
                if (__builtin_expect(far, 0)) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (!(fabsf(f[2 * i]) < __builtin_inff()))
                            q[i] = (q[i] & 0xFF00u) | 0x7Fu;
                        if (!(fabsf(f[2 * i + 1]) < __builtin_inff()))
                            q[i] = (q[i] & 0xFFu) | 0x7F00u;
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (e[j] < a.D)
                        *(uint2*)(dst + e[j]) =
                            make_uint2(q[4 * j] | q[4 * j + 1] << 16, q[4 * j + 2] | q[4 * j + 3] << 16);
                if (c == 0)
                    out.scales[(page * a.kv_heads + head) * a.page_size + place] =
                        bad > 0.0f ? __builtin_nanf("") : scale_of(amax_c);
            }
        }
    }
}

__global__ __launch_bounds__(kMaxPairs) void rope_frequencies_kernel(const FrequencyArgs a, double* out)
{
    const int i = threadIdx.x;
    if (i >= a.R / 2)
        return;
    const double f = pow(a.base, -2.0 * i / a.R);
    double y = f;
    if (a.scaling == W4A8_ROPE_LINEAR) {
        y = f / a.factor;
    } else if (a.scaling == W4A8_ROPE_YARN) {
        const double r = fmin(fmax((i - a.lo) / fmax(a.hi - a.lo, 0.001), 0.0), 1.0);
        y = f / a.factor * r + f * (1.0 - r);
    }
    out[i] = y;
}

namespace {

int lanes_of(const RopeArgs& a)
{
    return a.D <= 128 ? 8 : 16;
}
// Many rows: four a lane group, so that a wave's angles serve more of them and
// its loads are in flight together; few: one, for more waves.
int passes_of(const RopeArgs& a)
{
    const int64_t rows = a.q_heads + 2 * (int64_t)a.kv_heads;
    return a.T * ((rows * lanes_of(a) + 63) / 64) <= 8192 ? 1 : 4;
}
int64_t parts_of(const RopeArgs& a)
{
    const int64_t rows = a.q_heads + 2 * (int64_t)a.kv_heads, step = 64 / lanes_of(a) * passes_of(a);
    return (rows + step - 1) / step;
}

template <int TYPE, int LAYOUT, int LANES, bool QUANT>
hipError_t launch4(const RopeArgs& a, hipStream_t s)
{
    const int64_t parts = parts_of(a);
    const dim3 grid((unsigned)((a.T * parts + kWaves - 1) / kWaves)), block(64 * kWaves);
    if (passes_of(a) == 1)
        hipLaunchKernelGGL((rope_kernel<TYPE, LAYOUT, LANES, 1, QUANT>), grid, block, 0, s, a, (int32_t)parts);
    else
        hipLaunchKernelGGL((rope_kernel<TYPE, LAYOUT, LANES, 4, QUANT>), grid, block, 0, s, a, (int32_t)parts);
    return hipGetLastError();
}
template <int TYPE, int LAYOUT, bool QUANT>
hipError_t launch3(const RopeArgs& a, hipStream_t s)
{
    return lanes_of(a) == 8 ? launch4<TYPE, LAYOUT, 8, QUANT>(a, s) : launch4<TYPE, LAYOUT, 16, QUANT>(a, s);
}
template <int TYPE, bool QUANT>
hipError_t launch2(const RopeArgs& a, hipStream_t s)
{
    if (a.interleaved)
        return launch3<TYPE, kPairs, QUANT>(a, s);
    return a.R % 16 == 0 && a.D % 16 == 0 ? launch3<TYPE, kHalves, QUANT>(a, s) : launch3<TYPE, kHalvesAny, QUANT>(a, s);
}

}  // namespace

// whether the launch stays below 2^32 threads
bool rope_fits(const RopeArgs& a)
{
    return (a.T * parts_of(a) + kWaves - 1) / kWaves * (64 * kWaves) <= (int64_t)UINT32_MAX;
}

hipError_t launch_rope(const RopeArgs& a, hipStream_t s)
{
    if (a.kv_heads > 0 && a.cache_type == W4A8_TYPE_E4M3)
        return a.type == W4A8_TYPE_BF16 ? launch2<W4A8_TYPE_BF16, true>(a, s) : launch2<W4A8_TYPE_FP16, true>(a, s);
    switch (a.type) {
    case W4A8_TYPE_BF16: return launch2<W4A8_TYPE_BF16, false>(a, s);
    case W4A8_TYPE_FP16: return launch2<W4A8_TYPE_FP16, false>(a, s);
    default: return launch2<W4A8_TYPE_FP32, false>(a, s);
    }
}

hipError_t launch_rope_frequencies(const FrequencyArgs& a, double* out, hipStream_t s)
{
    hipLaunchKernelGGL(rope_frequencies_kernel, dim3(1), dim3(kMaxPairs), 0, s, a, out);
    return hipGetLastError();
}

}  // namespace w4a8
