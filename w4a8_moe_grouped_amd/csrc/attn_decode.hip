// attn_decode.hip -- attention of one new token per sequence over the paged
// cache (w4a8_attn_decode).
//
// Bound by the cache's bytes, each read once for all the query heads of its kv
// head.  A wave takes tiles of 32 keys and keeps everything in registers:
//   S[key, head] = K Q^T and O[d, head] += V^T P^T are MFMA 16x16x32 with the
//   heads (up to 16) as columns, so a lane holds one head's scores and sums
//   and the softmax needs no exchange but the maximum's.
// Which key is which row of S is free: rows 4g + r of its two products are
// keys 8g + r and 8g + 4 + r, so the 8 scores a lane of quarter g ends up with
// are those of keys 8g.. + 7, which are the K positions of the second product's
// operand in that lane.  The operand's other side, element d of 8 keys in one lane,
// comes from 8 loads of a key's 16 bytes each (16 lanes read a row of 256
// contiguous bytes) and byte permutations: product i takes the elements d = 8c + i of
// the chunks c that the lanes hold.  So the cache goes straight into
// registers, whole rows at a time, and LDS only joins the 4 waves at the end.
//
// The maximum is taken lazily: sums are rescaled only when a score passes the
// reference by 2^8, which a vote of the wave finds out.
//
// Work: the batch's tiles are numbered (sequence, kv head, unit of 128 keys)
// and cut evenly over the workgroups, from the lengths on the device.  A sequence and kv
// head that falls into several workgroups leaves partial results, at most two
// per workgroup, which a second launch joins in order; one that falls into one is
// finished there.
#include "api_util.hpp"
#include "common.hpp"
#include "internal.hpp"
#include "w4a8.h"

namespace w4a8 {

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kTile = 32;                // keys a wave takes at a time
constexpr int kUnit = kTile * kWaves;    // keys a workgroup takes at a time
constexpr int kHeads = 16;               // columns of a product
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

struct Plan {
    AttnArgs a;
    int32_t group, blocks;  // query heads per kv head; blocks of 16 of them
    int32_t items;          // kv heads x blocks
    int32_t workgroups;
    int32_t cut;            // whether sequences are cut over workgroups
    uint32_t page_mul;      // floor(n / page_size) = (2 n page_mul) >> (32 + page_shift), n < 2^30
    int32_t page_shift;
    int64_t* header;        // total units, workgroups in use; then the first unit of each sequence
    float* part_o;          // [2 workgroups][16][D]
    float2* part_ml;        // [2 workgroups][16]: reference, sum
};

__device__ __forceinline__ int page_of(const Plan& p, int key)
{
    return (int)(__umulhi((uint32_t)key << 1, p.page_mul) >> p.page_shift);
}

// keys [start, end) that sequence b sees
__device__ __forceinline__ void span_of(const AttnArgs& a, int b, int& start, int& end)
{
    const int64_t len = a.lens[b];
    const int64_t table = (int64_t)a.max_pages * a.page_size;
    end = (int)min(max(len, (int64_t)0), table);
    start = a.window > 0 ? (int)min(max(len - a.window, (int64_t)0), table) : 0;
}
__device__ __forceinline__ int units_of(int start, int end)
{
    return start < end ? (end + kUnit - 1) / kUnit - start / kUnit : 0;
}

// a value that is the same in all lanes, in scalar registers
__device__ __forceinline__ int64_t uniform(int64_t v)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ float exp2_(float x)
{
    return __builtin_amdgcn_exp2f(x);
}

// the operand types of one kind of cache
template <int CT>
struct Kind;
template <>
struct Kind<W4A8_TYPE_BF16> {
    static __device__ __forceinline__ v4f mfma(const v4i& a, const v4i& b, const v4f& c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) { return f32x2_to_bf16x2(a, b); }
};
template <>
struct Kind<W4A8_TYPE_FP16> {
    static __device__ __forceinline__ v4f mfma(const v4i& a, const v4i& b, const v4f& c)
    {
        return mfma16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        return __builtin_bit_cast(uint32_t, v2h{(_Float16)a, (_Float16)b});
    }
};
template <>
struct Kind<W4A8_TYPE_E4M3> : Kind<W4A8_TYPE_BF16> {};

// two of a dword's four e4m3 codes -> two bf16 (exact)
template <bool HIGH>
__device__ __forceinline__ uint32_t fp8x2_to_bf16(uint32_t d)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, HIGH));
}

template <int BYTES>
struct Chunk;
template <>
struct Chunk<4> {
    typedef uint32_t T;
};
template <>
struct Chunk<8> {
    typedef uint2 T;
};
template <>
struct Chunk<16> {
    typedef v4i T;
};

}  // namespace

// CT: type of the cache.  DP: D rounded up to 64, 128 or 256.  PAD: D < DP (or
// rows of codes that are not 16-byte aligned): chunks past D are not read.
// RUNS: pages hold whole runs of 8 keys, so a lane's 8 keys share a page.
template <int CT, int DP, bool PAD, bool RUNS>
__global__ __launch_bounds__(kThreads, DP == 256 ? 1 : 2) void attn_decode_kernel(const Plan p)
{
    using K = Kind<CT>;
    constexpr bool FP8 = CT == W4A8_TYPE_E4M3;
    constexpr int kElem = FP8 ? 1 : 2;
    constexpr int kSteps = DP / 32;                       // MFMA steps over d
    constexpr int kKLoads = FP8 ? DP / 64 : DP / 32;      // 16-byte loads of a lane's key row
    constexpr int kPer = DP == 64 ? 4 : 8;                // elements of a lane's chunk of a value row
    constexpr int kHalves = DP == 256 ? 2 : 1;            // chunks of a lane
    constexpr int kOut = kPer * kHalves;                  // products over d
    using VChunk = typename Chunk<kPer * kElem>::T;
    constexpr int kVWords = kPer * kElem / 4;

    const AttnArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, c16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    __shared__ float sh_o[kWaves][kOut * 4][64];
    __shared__ float2 sh_ml[kWaves][kHeads];
    __shared__ int64_t sh_sum[kThreads];
    __shared__ int64_t sh_at[2];  // sequence, its first unit

    // where this workgroup's work begins
    int64_t u = 0, u_end = 0;  // in units of the whole batch
    int b = 0;
    int64_t b_first = 0;       // first unit of sequence b
    if (p.cut) {
        // thread i sums the units of an equal part of the sequences
        const int per = (a.B + kThreads - 1) / kThreads;
        const int first = tid * per, last = min(first + per, a.B);
        int64_t mine = 0;
        for (int i = first; i < last; ++i) {
            int s, e;
            span_of(a, i, s, e);
            mine += units_of(s, e);
        }
        mine *= p.items;
        sh_sum[tid] = mine;
        __syncthreads();
        for (int o = 1; o < kThreads; o <<= 1) {
            const int64_t v = tid >= o ? sh_sum[tid - o] : 0;
            __syncthreads();
            sh_sum[tid] += v;
            __syncthreads();
        }
        const int64_t total = uniform(sh_sum[kThreads - 1]);
        const int in_use = (int)min((int64_t)p.workgroups, total);
        const int64_t before = sh_sum[tid] - mine;
        if (blockIdx.x == 0) {  // for the join
            if (tid == 0) {
                p.header[0] = total;
                p.header[1] = in_use;
            }
            int64_t at = before;
            for (int i = first; i < last; ++i) {
                p.header[2 + i] = at;
                int s, e;
                span_of(a, i, s, e);
                at += (int64_t)units_of(s, e) * p.items;
            }
            if (last == a.B && first < last)
                p.header[2 + a.B] = at;
        }
        if ((int)blockIdx.x >= in_use)
            return;
        u = total * (int)blockIdx.x / in_use;
        u_end = total * ((int)blockIdx.x + 1) / in_use;
        if (before <= u && u < before + mine) {
            int64_t at = before;
            for (int i = first; i < last; ++i) {
                int s, e;
                span_of(a, i, s, e);
                const int64_t n = (int64_t)units_of(s, e) * p.items;
                if (u < at + n) {
                    sh_at[0] = i;
                    sh_at[1] = at;
                    break;
                }
                at += n;
            }
        }
        __syncthreads();
        b = (int)uniform(sh_at[0]);
        b_first = uniform(sh_at[1]);
    }

    const float c = a.scale * kLog2e;
    for (int segment = 0;; ++segment) {
        int start, end, item, unit0, unit1, units;
        if (p.cut) {
            if (u >= u_end)
                break;
            span_of(a, b, start, end);
            units = units_of(start, end);
            if (u >= b_first + (int64_t)units * p.items) {
                b_first += (int64_t)units * p.items;
                ++b;
                --segment;
                continue;
            }
            item = (int)((u - b_first) / units);
            unit0 = (int)(u - b_first - (int64_t)item * units);
            unit1 = (int)min((int64_t)units, unit0 + (u_end - u));
            u += unit1 - unit0;
        } else {
            if (segment > 0)
                break;
            b = (int)blockIdx.x / p.items;
            item = (int)blockIdx.x - b * p.items;
            span_of(a, b, start, end);
            units = units_of(start, end);
            unit0 = 0;
            unit1 = units;
        }
        const int kv = item / p.blocks, head0 = kv * p.group + (item - kv * p.blocks) * kHeads;
        const int heads = min(kHeads, (kv + 1) * p.group - head0);
        const int tile_base = start / kUnit * kWaves + wave;
        const int32_t* table = a.table + b * a.ld_table;

        // the queries: column c16, positions of d as the keys' loads give them
        v4i q[kSteps];
        {
            const uint16_t* src = (const uint16_t*)a.q + b * a.q_bs + (head0 + min(c16, heads - 1)) * a.q_hs;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int d = FP8 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
                const bool in = c16 < heads && (!PAD || d < a.D);
                q[s] = in ? ldg16(src + d) : v4i{0, 0, 0, 0};
            }
        }
        v4f o[kOut];
#pragma unroll
        for (int i = 0; i < kOut; ++i)
            o[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        float m = -__builtin_inff(), ref = 0.0f, l = 0.0f;

        const char* const kbase = (const char*)a.kc.p + kv * a.kc.hs * kElem;
        const char* const vbase = (const char*)a.vc.p + kv * a.vc.hs * kElem;
        const int64_t kts = a.kc.ts * kElem, kps = a.kc.ps * kElem, vts = a.vc.ts * kElem, vps = a.vc.ps * kElem;

        v4i kreg[2][kKLoads];
        VChunk vreg[8][kHalves];
        float ksc[8], vsc[8];
        uint32_t mask = 0;  // which of the lane's 8 keys 8g.. of the tile are there

        // the page of the key `key`, or -1
        auto lookup = [&](int key) {
            if (key < start || key >= end)
                return -1;
            const int id = table[page_of(p, key)];
            return id >= 0 && id < a.num_pages ? id : -1;
        };
        // the page of the run of 8 keys from `key`, or -1
        auto lookup_run = [&](int key) {
            if (key + 8 <= start || key >= end)
                return -1;
            const int id = table[page_of(p, key)];
            return id >= 0 && id < a.num_pages ? id : -1;
        };
        auto load_k_row = [&](int t, const char* row) {
#pragma unroll
            for (int i = 0; i < kKLoads; ++i) {
                if (!FP8) {
                    const int d = 32 * i + 8 * g;
                    kreg[t][i] = !PAD || d < a.D ? ldg16(row + 2 * d) : v4i{0, 0, 0, 0};
                } else if (!PAD) {
                    kreg[t][i] = ldg16(row + 64 * i + 16 * g);
                } else {
                    const int d = 64 * i + 16 * g;
                    const uint2 x = d < a.D ? *(const uint2*)(row + d) : make_uint2(0, 0);
                    const uint2 y = d + 8 < a.D ? *(const uint2*)(row + d + 8) : make_uint2(0, 0);
                    kreg[t][i] = v4i{(int)x.x, (int)x.y, (int)y.x, (int)y.y};
                }
            }
        };
        auto load_v_row = [&](int j, const char* row) {
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                const int d = 128 * h + kPer * c16;
                if (!PAD || d < a.D)
                    vreg[j][h] = *(const VChunk*)(row + d * kElem);
                else
                    vreg[j][h] = VChunk{};
            }
        };
        const int krun = 8 * (c16 >> 2);  // this lane's key row in a tile is in the run of that key
        auto load_k = [&](int tile, int idk) {
            const int key0 = tile * kTile;
            if (RUNS) {
                const int key = key0 + krun;
                const int off = idk >= 0 ? key - page_of(p, key) * a.page_size : 0;
                const char* row = kbase + max(idk, 0) * kps + (off + (c16 & 3)) * kts;
                load_k_row(0, row);
                load_k_row(1, row + 4 * kts);
            } else {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int key = key0 + krun + 4 * t + (c16 & 3);
                    const int id = lookup(key);
                    const int off = id >= 0 ? key - page_of(p, key) * a.page_size : 0;
                    load_k_row(t, kbase + max(id, 0) * kps + off * kts);
                }
            }
        };
        auto load_v = [&](int tile, int idv) {
            const int key = tile * kTile + 8 * g;
            mask = 0;
            if (RUNS) {
                const int off = idv >= 0 ? key - page_of(p, key) * a.page_size : 0;
                const char* row = vbase + max(idv, 0) * vps + off * vts;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    load_v_row(j, row + j * vts);
                if (idv >= 0) {
                    const int lo = max(start - key, 0), hi = min(end - key, 8);
                    mask = (0xFFu << lo) & (0xFFu >> (8 - hi)) & 0xFFu;
                }
                if (FP8) {
                    const int64_t at = ((int64_t)max(idv, 0) * a.kv_heads + kv) * a.page_size + off;
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        const float4 x = *(const float4*)(a.kc.scales + at + j), y = *(const float4*)(a.vc.scales + at + j);
                        ksc[j] = x.x, ksc[j + 1] = x.y, ksc[j + 2] = x.z, ksc[j + 3] = x.w;
                        vsc[j] = y.x, vsc[j + 1] = y.y, vsc[j + 2] = y.z, vsc[j + 3] = y.w;
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int id = lookup(key + j);
                    const int off = id >= 0 ? key + j - page_of(p, key + j) * a.page_size : 0;
                    load_v_row(j, vbase + max(id, 0) * vps + off * vts);
                    if (FP8) {
                        const int64_t at = ((int64_t)max(id, 0) * a.kv_heads + kv) * a.page_size + off;
                        ksc[j] = a.kc.scales[at];
                        vsc[j] = a.vc.scales[at];
                    }
                    mask |= (id >= 0 ? 1u : 0u) << j;
                }
            }
        };

        // this wave's tiles, those that hold a key that is seen
        int tile = tile_base + unit0 * kWaves;
        const int tile_end = min(tile_base - wave + unit1 * kWaves, (end + kTile - 1) / kTile);
        while (tile < tile_end && (tile + 1) * kTile <= start)
            tile += kWaves;
        int idk = -1, idv = -1;
        if (tile < tile_end) {
            if (RUNS) {
                idk = lookup_run(tile * kTile + krun);
                idv = lookup_run(tile * kTile + 8 * g);
            }
            load_k(tile, idk);
            load_v(tile, idv);
            if (RUNS && tile + kWaves < tile_end) {
                idk = lookup_run((tile + kWaves) * kTile + krun);
                idv = lookup_run((tile + kWaves) * kTile + 8 * g);
            }
        }
        for (; tile < tile_end; tile += kWaves) {
            const bool more = tile + kWaves < tile_end;
            v4f s[2] = {v4f{0.0f, 0.0f, 0.0f, 0.0f}, v4f{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    v4i x;
                    if (FP8) {
                        const uint32_t d0 = (uint32_t)kreg[t][k >> 1][2 * (k & 1)], d1 = (uint32_t)kreg[t][k >> 1][2 * (k & 1) + 1];
                        x = v4i{(int)fp8x2_to_bf16<false>(d0), (int)fp8x2_to_bf16<true>(d0), (int)fp8x2_to_bf16<false>(d1),
                                (int)fp8x2_to_bf16<true>(d1)};
                    } else {
                        x = kreg[t][FP8 ? 0 : k];
                    }
                    s[t] = K::mfma(x, q[k], s[t]);
                }
            int idv_next = idv;
            if (more) {
                const int idk_now = idk;
                if (RUNS && tile + 2 * kWaves < tile_end) {
                    idk = lookup_run((tile + 2 * kWaves) * kTile + krun);
                    idv_next = lookup_run((tile + 2 * kWaves) * kTile + 8 * g);
                }
                load_k(tile + kWaves, idk_now);
            }
            // scores in powers of two; those that are not there are -inf
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = s[j >> 2][j & 3] * (FP8 ? c * ksc[j] : c);
            const bool whole = __all(mask == 0xFFu);
            if (!whole) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = mask >> j & 1 ? x[j] : -__builtin_inff();
            }
            float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
            if (__any(top > m + 8.0f)) {
                top = fmaxf(top, __shfl_xor(top, 16, 64));
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                const float next = fmaxf(m, top);
                const float next_ref = next == -__builtin_inff() ? 0.0f : next;
                const float f = exp2_(m - next_ref);
                l *= f;
#pragma unroll
                for (int i = 0; i < kOut; ++i)
                    o[i] *= f;
                m = next;
                ref = next_ref;
            }
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                w[j] = exp2_(x[j] - ref);
                l += w[j];
                if (FP8)
                    w[j] *= vsc[j];
            }
            if (!whole) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool in = mask >> j & 1;
                    w[j] = in ? w[j] : 0.0f;
#pragma unroll
                    for (int h = 0; h < kHalves; ++h)
                        if (!in)
                            vreg[j][h] = VChunk{};
                }
            }
            const v4i pw = {(int)K::pack(w[0], w[1]), (int)K::pack(w[2], w[3]), (int)K::pack(w[4], w[5]),
                            (int)K::pack(w[6], w[7])};
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int d = 0; d < kVWords; ++d) {
                    uint32_t word[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        word[j] = ((const uint32_t*)&vreg[j][h])[d];
                    if (!FP8) {  // two elements of eight keys
                        v4i lo, hi;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            lo[j] = (int)__builtin_amdgcn_perm(word[2 * j + 1], word[2 * j], 0x05040100u);
                            hi[j] = (int)__builtin_amdgcn_perm(word[2 * j + 1], word[2 * j], 0x07060302u);
                        }
                        o[kPer * h + 2 * d] = K::mfma(lo, pw, o[kPer * h + 2 * d]);
                        o[kPer * h + 2 * d + 1] = K::mfma(hi, pw, o[kPer * h + 2 * d + 1]);
                    } else {  // four elements of eight keys
                        v4i e[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t lo = __builtin_amdgcn_perm(word[2 * j + 1], word[2 * j], 0x05010400u);
                            const uint32_t hi = __builtin_amdgcn_perm(word[2 * j + 1], word[2 * j], 0x07030602u);
                            e[0][j] = (int)fp8x2_to_bf16<false>(lo);
                            e[1][j] = (int)fp8x2_to_bf16<true>(lo);
                            e[2][j] = (int)fp8x2_to_bf16<false>(hi);
                            e[3][j] = (int)fp8x2_to_bf16<true>(hi);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[kPer * h + 4 * d + i] = K::mfma(e[i], pw, o[kPer * h + 4 * d + i]);
                    }
                }
            if (more) {
                load_v(tile + kWaves, idv);
                idv = idv_next;
            }
        }

        // join the waves
        l += __shfl_xor(l, 16, 64);
        l += __shfl_xor(l, 32, 64);
        if (g == 0)
            sh_ml[wave][c16] = make_float2(m, l);
#pragma unroll
        for (int i = 0; i < kOut; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                sh_o[wave][4 * i + r][lane] = o[i][r];
        __syncthreads();
        float2 ml[kWaves];
        float all_m = -__builtin_inff(), all_l = 0.0f, f[kWaves];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            ml[w] = sh_ml[w][c16];
            all_m = fmaxf(all_m, ml[w].x);
        }
        const float all_ref = all_m == -__builtin_inff() ? 0.0f : all_m;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            f[w] = exp2_(ml[w].x - all_ref);
            all_l += ml[w].y * f[w];
        }
        const bool done = !p.cut || (unit0 == 0 && unit1 == units);
        const int64_t slot = 2 * (int64_t)blockIdx.x + (segment > 0);
        const float inv = all_l == 0.0f ? 0.0f : 1.0f / all_l;  // NaN stays
        // this wave takes register `wave` of each product: elements kPer * (4 g + wave) .. of column c16
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            float y[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                y[i] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w)
                    y[i] += sh_o[w][4 * (kPer * h + i) + wave][lane] * f[w];
            }
            const int d = 128 * h + kPer * (4 * g + wave);
            if (c16 < heads && d < a.D) {
                if (done) {
                    uint32_t* dst = (uint32_t*)((uint16_t*)a.out + b * a.o_bs + (head0 + c16) * a.o_hs + d);
#pragma unroll
                    for (int i = 0; i < kPer; i += 2)
                        dst[i / 2] = K::pack(y[i] * inv, y[i + 1] * inv);
                } else {
                    float* dst = p.part_o + (slot * kHeads + c16) * a.D + d;
#pragma unroll
                    for (int i = 0; i < kPer; i += 4)
                        *(float4*)(dst + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                }
            }
        }
        if (wave == 0 && g == 0 && c16 < heads) {
            if (!done)
                p.part_ml[slot * kHeads + c16] = make_float2(all_m, all_l);
            else if (a.lse != nullptr)
                a.lse[(int64_t)b * a.q_heads + head0 + c16] = (all_m + __builtin_amdgcn_logf(all_l)) * kLn2;
        }
        __syncthreads();  // before the next segment writes into LDS
    }
}

// One wave per (sequence, query head): nothing to do where the head's work lay
// in one workgroup; zeros where there was none.
template <bool F16>
__global__ __launch_bounds__(256) void attn_join_kernel(const Plan p)
{
    const AttnArgs& a = p.a;
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= (int64_t)a.B * a.q_heads)
        return;
    const int b = (int)(row / a.q_heads), head = (int)(row - (int64_t)b * a.q_heads);
    const int kv = head / p.group, in_group = head - kv * p.group;
    const int item = kv * p.blocks + in_group / kHeads, col = in_group % kHeads;
    uint16_t* out = (uint16_t*)a.out + b * a.o_bs + head * a.o_hs;
    const int64_t total = p.header[0], in_use = p.header[1];
    const int64_t b0 = p.header[2 + b], units = (p.header[3 + b] - b0) / p.items;
    if (units == 0) {
        for (int d = lane; d < a.D; d += 64)
            out[d] = 0;
        if (lane == 0 && a.lse != nullptr)
            a.lse[row] = -__builtin_inff();
        return;
    }
    // workgroup w begins at floor(total * w / in_use)
    const int64_t u0 = b0 + item * units, u1 = u0 + units;
    const int64_t w0 = ((u0 + 1) * in_use + total - 1) / total - 1, w1 = (u1 * in_use + total - 1) / total - 1;
    if (w0 == w1)
        return;
    auto slot_of = [&](int64_t w) {  // the work is the workgroup's first, or for w0 perhaps a later one
        return 2 * w + (w == w0 && total * w / in_use < u0);
    };
    float m = -__builtin_inff();
    for (int64_t w = w0 + lane; w <= w1; w += 64)
        m = fmaxf(m, p.part_ml[slot_of(w) * kHeads + col].x);
    m = group_max<64>(m);
    const float ref = m == -__builtin_inff() ? 0.0f : m;
    float l = 0.0f;
    for (int64_t w = w0 + lane; w <= w1; w += 64) {
        const float2 ml = p.part_ml[slot_of(w) * kHeads + col];
        l += ml.y * exp2_(ml.x - ref);
    }
    l = group_sum<64>(l);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    for (int d = lane; d < a.D; d += 64) {
        float y = 0.0f;
        for (int64_t w = w0; w <= w1; ++w) {
            const int64_t at = slot_of(w) * kHeads + col;
            y += p.part_o[at * a.D + d] * exp2_(p.part_ml[at].x - ref);
        }
        y *= inv;
        out[d] = F16 ? __builtin_bit_cast(uint16_t, (_Float16)y) : (uint16_t)f32x2_to_bf16x2(y, 0.0f);
    }
    if (lane == 0 && a.lse != nullptr)
        a.lse[row] = (m + __builtin_amdgcn_logf(l)) * kLn2;
}

namespace {

constexpr int64_t kWorkgroups = 512;  // two for each CU

// Cut over workgroups unless no sequence can be longer than one unit.
bool cuts(int64_t max_len)
{
    return max_len > kUnit;
}

Plan plan(void* ws, const AttnArgs& a, size_t* bytes)
{
    Plan p = {};
    p.a = a;
    p.group = a.q_heads / a.kv_heads;
    p.blocks = (p.group + kHeads - 1) / kHeads;
    p.items = a.kv_heads * p.blocks;
    int64_t longest = (int64_t)a.max_pages * a.page_size;
    p.cut = cuts(longest);
    p.workgroups = (int32_t)(p.cut ? kWorkgroups : (int64_t)a.B * p.items);
    // 2^l >= s > 2^(l - 1): m = ceil(2^(31 + l) / s) is below 2^32, and m s exceeds
    // 2^(31 + l) by less than s, so n m / 2^(31 + l) exceeds n / s by less than
    // n / 2^(31 + l) <= n 2^-31 / s, which is below 1 / s and carries over no integer
    int l = 0;
    while (((int64_t)1 << l) < a.page_size)
        ++l;
    p.page_mul = (uint32_t)((((uint64_t)1 << (31 + l)) + a.page_size - 1) / a.page_size);
    p.page_shift = l;
    api::Carve c(ws);
    if (p.cut) {
        p.header = c.take<int64_t>((size_t)a.B + 3);
        p.part_o = c.take<float>((size_t)(2 * kWorkgroups) * kHeads * a.D);
        p.part_ml = c.take<float2>((size_t)(2 * kWorkgroups) * kHeads);
    }
    *bytes = c.used;
    return p;
}

template <int CT, int DP, bool PAD>
void launch3(const Plan& p, hipStream_t s)
{
    const dim3 grid((unsigned)p.workgroups);
    if (p.a.page_size % 8 == 0)
        hipLaunchKernelGGL((attn_decode_kernel<CT, DP, PAD, true>), grid, dim3(kThreads), 0, s, p);
    else
        hipLaunchKernelGGL((attn_decode_kernel<CT, DP, PAD, false>), grid, dim3(kThreads), 0, s, p);
}
template <int CT, int DP>
void launch2(const Plan& p, hipStream_t s)
{
    const AttnArgs& a = p.a;
    const bool apart = CT == W4A8_TYPE_E4M3 &&  // code rows that are not 16-byte aligned
                       (((uintptr_t)a.kc.p | (uintptr_t)a.vc.p | (uintptr_t)(a.kc.ps | a.kc.ts | a.kc.hs) |
                         (uintptr_t)(a.vc.ps | a.vc.ts | a.vc.hs)) & 15) != 0;
    if (a.D != DP || apart)
        launch3<CT, DP, true>(p, s);
    else
        launch3<CT, DP, false>(p, s);
}
template <int CT>
void launch1(const Plan& p, hipStream_t s)
{
    if (p.a.D <= 64)
        launch2<CT, 64>(p, s);
    else if (p.a.D <= 128)
        launch2<CT, 128>(p, s);
    else
        launch2<CT, 256>(p, s);
}

}  // namespace

size_t attn_decode_workspace(int64_t B, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_len)
{
    AttnArgs a = {};
    a.B = (int32_t)B, a.q_heads = (int32_t)q_heads, a.kv_heads = (int32_t)kv_heads, a.D = (int32_t)D;
    a.page_size = 1, a.max_pages = (int32_t)max_len;
    size_t bytes;
    plan(nullptr, a, &bytes);
    return bytes;
}

hipError_t launch_attn_decode(const AttnArgs& a, void* ws, hipStream_t s)
{
    size_t bytes;
    const Plan p = plan(ws, a, &bytes);
    switch (a.cache_type) {
    case W4A8_TYPE_BF16: launch1<W4A8_TYPE_BF16>(p, s); break;
    case W4A8_TYPE_FP16: launch1<W4A8_TYPE_FP16>(p, s); break;
    default: launch1<W4A8_TYPE_E4M3>(p, s);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.cut)
        return e;
    const dim3 grid((unsigned)(((int64_t)a.B * a.q_heads + 3) / 4));
    if (a.q_type == W4A8_TYPE_FP16)
        hipLaunchKernelGGL((attn_join_kernel<true>), grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((attn_join_kernel<false>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace w4a8
