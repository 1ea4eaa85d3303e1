// rope.hip -- rotary positions (w4a8_rope) and the append to a paged cache that
// rotates on the way (w4a8_kv_append).
//
// Bound by bytes: each element is read once and written once.  A wave takes
// one token and some of its rows (the heads of q, then k, then v).  Its lanes
// first make the token's cosines and sines, one pair each, into the wave's own
// part of LDS, so that their 40 operations are done once for all the wave's
// rows; then 8 lanes (16 for D > 128) hold a row, two chunks of 8 elements
// each, which for pairs of halves are the two partners, so that all accesses
// are 16 bytes and no element crosses lanes.
//
// The angle's turns are reduced in 64 bits (at position 10^6 an fp32 angle is
// off by 0.03), sine and cosine of what is left, at most an eighth of a turn,
// by their Taylor series in fp32.
#include "common.hpp"
#include "internal.hpp"
#include "w4a8.h"

namespace w4a8 {

namespace {

constexpr int kWaves = 4;       // per workgroup
constexpr int kMaxPairs = 128;  // D <= 256
enum Layout { kPairs = 0, kHalves = 1, kHalvesAny = 2 };

// cos and sin of 2 pi `turns`, times m
__device__ __forceinline__ float2 cos_sin(double turns, float m)
{
    const double quarter = rint(4.0 * turns);
    const float x = (float)((turns - 0.25 * quarter) * 6.283185307179586477);
    const int n = (int)(quarter - 4.0 * floor(0.25 * quarter));
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

template <int TYPE>
struct Elem;
template <>
struct Elem<W4A8_TYPE_FP32> {
    typedef float T;
    struct Raw {
        v4i a, b;
    };
    static __device__ __forceinline__ Raw load(const T* p) { return Raw{ldg16(p), ldg16(p + 4)}; }
    static __device__ __forceinline__ float get(const Raw& r, int i)
    {
        return __int_as_float(i < 4 ? r.a[i & 3] : r.b[i & 3]);
    }
    static __device__ __forceinline__ float one(const T* p) { return *p; }
    static __device__ __forceinline__ void store(T* p, const float* f)
    {
        *(float4*)p = make_float4(f[0], f[1], f[2], f[3]);
        *(float4*)(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
};
template <>
struct Elem<W4A8_TYPE_BF16> {
    typedef uint16_t T;
    struct Raw {
        v4i a;
    };
    static __device__ __forceinline__ Raw load(const T* p) { return Raw{ldg16(p)}; }
    static __device__ __forceinline__ float get(const Raw& r, int i)
    {
        const uint32_t d = (uint32_t)r.a[i >> 1];
        return __uint_as_float(i & 1 ? d & 0xFFFF0000u : d << 16);
    }
    static __device__ __forceinline__ float one(const T* p) { return bf16_to_f32(*p); }
    static __device__ __forceinline__ void store(T* p, const float* f)
    {
        *(v4i*)p = v4i{(int)f32x2_to_bf16x2(f[0], f[1]), (int)f32x2_to_bf16x2(f[2], f[3]),
                       (int)f32x2_to_bf16x2(f[4], f[5]), (int)f32x2_to_bf16x2(f[6], f[7])};
    }
};
template <>
struct Elem<W4A8_TYPE_FP16> {
    typedef _Float16 T;
    struct Raw {
        v8h a;
    };
    static __device__ __forceinline__ Raw load(const T* p) { return Raw{__builtin_bit_cast(v8h, ldg16(p))}; }
    static __device__ __forceinline__ float get(const Raw& r, int i) { return (float)r.a[i]; }
    static __device__ __forceinline__ float one(const T* p) { return (float)*p; }
    static __device__ __forceinline__ void store(T* p, const float* f)
    {
        v8h h;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h[i] = (_Float16)f[i];
        *(v8h*)p = h;
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
    __shared__ float2 table[kWaves][kMaxPairs];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t item = (int64_t)blockIdx.x * kWaves + wave;
    const int64_t t = item / parts;
    if (t >= a.T)
        return;
    const int c = lane & (LANES - 1);
    const int row0 = (int)(item - t * parts) * (kGroups * PASSES) + lane / LANES;
    const int rows = a.q_heads + 2 * a.kv_heads;
    const int half = a.R / 2;

    // this lane's two chunks of a row; the second may lie past its end
    int e0 = 16 * c, e1 = 16 * c + 8;
    if (LAYOUT == kHalves) {
        const int turned = a.R / 16;  // lanes that hold partners
        e0 = c < turned ? 8 * c : a.R + 16 * (c - turned);
        e1 = c < turned ? 8 * c + half : e0 + 8;
    }
    const bool has0 = e0 < a.D, has1 = e1 < a.D;

    auto source = [&](int row) {
        const bool is_q = row < a.q_heads, is_k = row < a.q_heads + a.kv_heads;
        const Rows& r = is_q ? a.q : is_k ? a.k : a.v;
        const int head = is_q ? row : is_k ? row - a.q_heads : row - a.q_heads - a.kv_heads;
        return (const T*)r.p + t * r.ts + head * r.hs;
    };
    typename E::Raw raw[PASSES][2];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int row = row0 + p * kGroups;
        if (row < rows) {
            const T* src = source(row);
            if (has0)
                raw[p][0] = E::load(src + e0);
            if (has1)
                raw[p][1] = E::load(src + e1);
        }
    }
    int64_t slot = -1;
    if (a.kv_heads > 0)
        slot = a.slots[t];
    if (half > 0) {
        const double turns_per = 0.15915494309189533577;
        const double pos = (double)a.positions[t];
        for (int i = lane; i < half; i += 64)
            table[wave][i] = cos_sin(pos * a.frequencies[i] * turns_per, a.magnitude);
    }
    __builtin_amdgcn_wave_barrier();  // one wave: LDS operations stay in order
    const float2* cs = table[wave];
    const bool kept = slot >= 0 && slot < a.num_slots;
    const int64_t page = kept ? slot / a.page_size : 0;
    const int64_t place = kept ? slot - page * a.page_size : 0;

#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int row = row0 + p * kGroups;
        const bool is_q = row < a.q_heads, is_k = !is_q && row < a.q_heads + a.kv_heads;
        const bool live = row < rows && (is_q || kept);
        float f[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = live && has0 ? E::get(raw[p][0], i) : 0.0f;
            f[8 + i] = live && has1 ? E::get(raw[p][1], i) : 0.0f;
        }
        if (live && (is_q || is_k) && half > 0) {
            if (LAYOUT == kHalves) {
                if (e0 < half) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 w = cs[e0 + i];
                        const float x = f[i], y = f[8 + i];
                        f[i] = x * w.x - y * w.y;
                        f[8 + i] = fmaf(x, w.y, y * w.x);
                    }
                }
            } else if (LAYOUT == kPairs) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int pair = 8 * c + i;
                    if (pair < half) {
                        const float2 w = cs[pair];
                        const float x = f[2 * i], y = f[2 * i + 1];
                        f[2 * i] = x * w.x - y * w.y;
                        f[2 * i + 1] = fmaf(x, w.y, y * w.x);
                    }
                }
            } else {
                // halves that are no whole chunks: the partner, element by element
                const T* src = source(row);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int e = 16 * c + i;
                    if (e < a.R) {
                        const bool first = e < half;
                        const float2 w = cs[first ? e : e - half];
                        const float y = E::one(src + (first ? e + half : e - half));
                        f[i] = first ? f[i] * w.x - y * w.y : fmaf(y, w.y, f[i] * w.x);
                    }
                }
            }
        }
        if (is_q && live) {
            T* dst = (T*)a.q_out + t * a.qo_ts + row * a.qo_hs;
            if (has0)
                E::store(dst + e0, f);
            if (has1)
                E::store(dst + e1, f + 8);
        }
        if (a.kv_heads == 0)
            continue;
        const CacheRows& out = is_k ? a.kc : a.vc;
        const int head = is_k ? row - a.q_heads : row - a.q_heads - a.kv_heads;
        const int64_t at = page * out.ps + place * out.ts + head * out.hs;
        if (!QUANT) {
            if (!is_q && live) {
                if (has0)
                    E::store((T*)out.p + at + e0, f);
                if (has1)
                    E::store((T*)out.p + at + e1, f + 8);
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
            if (!is_q && live) {
                uint8_t* dst = (uint8_t*)out.p + at;
                uint32_t q[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    q[i] = cvt_e4m3x2(f[2 * i] * inv, f[2 * i + 1] * inv);
                if (has0)
                    *(uint2*)(dst + e0) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
                if (has1)
                    *(uint2*)(dst + e1) = make_uint2(q[4] | q[5] << 16, q[6] | q[7] << 16);
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
    return a.T * ((rows * lanes_of(a) + 63) / 64) <= 4096 ? 1 : 4;
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
