// attn_decode.hip -- attention of one new token per sequence over the paged
// cache (w4a8_attn_decode).
//
// Bound by the cache's bytes, each read once for up to 16 query heads of its kv
// head (each 16 more read them again: 64 x 4096 keys, one kv head of 128, bf16,
// 16 query heads 32 us, 32 52, 128 154).  A wave takes tiles of 32 keys and keeps
// everything in registers:
//   S[key, head] = K Q^T and O[d, head] += V^T P^T are MFMA 16x16x32 with the
//   heads (up to 16) as columns, so a lane holds one head's scores and sums
//   and the softmax needs no exchange but the maximum's.
// Which key is which row of S is free: rows 4g + r of its two products are
// keys 8g + r and 8g + 4 + r, so the 8 scores a lane of quarter g ends up with
// are those of keys 8g.. + 7, which are the K positions of the second product's
// operand in that lane.  The operand's other side, element d of 8 keys in one
// lane, comes from 8 loads of a key's 16 bytes each (16 lanes read a row of 256
// contiguous bytes) and byte permutations: product i takes the elements d = 8c +
// i of the chunks c that the lanes hold.  So the cache goes straight into
// registers, whole rows at a time, and LDS only joins the waves at the end.
//
// The maximum is taken lazily: sums are rescaled only when a score passes the
// reference by 2^8 (fp16: 2), which a vote of the wave finds out.
//
// Work: the batch's tiles are numbered (sequence, kv head, unit of 128 keys) and
// cut evenly over the workgroups, from the lengths on the device.  A sequence
// and kv head that falls into several workgroups leaves partial results, at most
// two per workgroup, which a second launch joins in order; one that falls into
// one is finished there.  Where sequences are short by the table or the window (`cuts`),
// a workgroup takes one sequence and kv head whole, and there is no second launch.
//
// 64 x 4096 keys, 64 / 8 heads of 128, bf16: 192 us (5.6 TB/s; a reduction reads
// 6.1) and 4.9 for the second launch, which finds nothing to join; 655 MB of e4m3
// in 16 sequences: 133 + 7.0 (rows of 128 bytes, 1 KB apart); one sequence of
// 1000: 7.2 + 4.8.
#include "api_util.hpp"
#include "common.hpp"
#include "internal.hpp"
#include "w4a8.h"

#include <type_traits>

namespace w4a8 {

namespace {

constexpr int kJoinWaves = 4;
constexpr int kUnit = 128;               // keys: what work is counted and cut in
constexpr int kHeads = 16;               // columns of a product
enum Pad { kWhole, kShort, kApart };     // rows of the cache
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

typedef __bf16 v8b __attribute__((ext_vector_type(8)));

struct Plan {
    AttnArgs a;
    int32_t group, blocks;  // query heads per kv head; blocks of 16 of them
    int32_t items;          // kv heads x blocks
    int32_t workgroups;
    int32_t cut;            // whether sequences are cut over workgroups
    int32_t pair;           // whether two kv heads of 64 are taken together: group and items count pairs
    uint32_t page_mul;      // floor(n / page_size) = (2 n page_mul) >> (32 + page_shift), n < 2^30
    int32_t page_shift;
    int64_t* header;        // total units, workgroups in use; then the first unit of each sequence
    float* part_o;          // [2 workgroups][16][D]
    float2* part_ml;        // [2 workgroups][16]: maximum, sum
};

__device__ __forceinline__ int page_of(const Plan& p, int key)
{
    return (int)(__umulhi((uint32_t)key << 1, p.page_mul) >> p.page_shift);
}

// keys [start, end) that a sequence of this length sees
__device__ __forceinline__ void span_of(const AttnArgs& a, int64_t len, int& start, int& end)
{
    const int64_t table = (int64_t)a.max_pages * a.page_size;
    end = (int)min(max(len, (int64_t)0), table);
    start = a.window > 0 ? (int)min(max(len - a.window, (int64_t)0), table) : 0;
}
__device__ __forceinline__ int units_of(int start, int end)
{
    return start < end ? (end + kUnit - 1) / kUnit - start / kUnit : 0;
}

// The i-th of n pieces of work such that XCD i % 8 takes an eighth of them in
// order.  Neighbours are heads of one sequence, whose rows lie side by side in the
// usual layout: of 128 bytes and less they share lines or the memory's own rows (uncut,
// 64 x 4096 keys, 8 kv heads of 64, e4m3: 95 -> 82 us; cut, 64 x 16384: 344 -> 308, of 128
// 144 -> 141; 37 sequences under a window: 14.9 -> 13.6).  Cut, rows of 256 bytes lose
// (bf16, 64 x 4096 keys of 128: 200 -> 203), and stay as they are.
__device__ __forceinline__ int eighths(int i, int n)
{
    return (i & 7) * (n >> 3) + min(i & 7, n & 7) + (i >> 3);
}

// lane l's value, in scalar registers
__device__ __forceinline__ int64_t uniform(int64_t v, int l)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)v >> 32), l);
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// floor(x / y) of values below 2^52 (a call has less than 2^46 units)
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y)
{
    int64_t q = (int64_t)((double)x / (double)y);
    const int64_t r = x - q * y;
    q += r >= y ? 1 : 0;
    return q - (r < 0 ? 1 : 0);
}

// the first unit of workgroup w of n, which share `total` units: the first
// total % n of them have one more
__device__ __forceinline__ int64_t begin_of(int64_t total, int n, int w)
{
    const int64_t each = quotient(total, n), more = total - each * n;
    return each * w + min((int64_t)w, more);
}
// the workgroup that holds unit u
__device__ __forceinline__ int holder_of(int64_t total, int n, int64_t u)
{
    const int64_t each = quotient(total, n), more = total - each * n, big = (each + 1) * more;
    return (int)(u < big ? quotient(u, each + 1) : more + quotient(u - big, max(each, (int64_t)1)));
}

// inclusive sums over the lanes
__device__ __forceinline__ int64_t wave_scan(int64_t v, int lane)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t x = __shfl_up(v, o, 64);
        v += lane >= o ? x : 0;
    }
    return v;
}

__device__ __forceinline__ float exp2_(float x)
{
    return __builtin_amdgcn_exp2f(x);
}

typedef unsigned short v2us __attribute__((ext_vector_type(2)));
// whether one of n numbers is NaN or infinite, without a comparison for each, whose
// results would go through scalar registers
template <int N>
__device__ __forceinline__ bool not_finite(const float (&x)[N])
{
    float zero[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i)
        zero[i & 1] = fmaf(x[i], 0.0f, zero[i & 1]);
    return zero[0] != zero[1];
}
// two 16-bit values, not negative, each not below its half of `least`: their bits
// order as they do, NaN above all
__device__ __forceinline__ int raised(uint32_t d, uint32_t least)
{
    return __builtin_bit_cast(int, __builtin_elementwise_max(__builtin_bit_cast(v2us, d), __builtin_bit_cast(v2us, least)));
}

// The operand types of one kind of cache.  split: weights as a value cut to the
// type and what the cut left, each not below `least` (two of them in its halves).
// The weights are held times 2^kShift.  kLazy: the scores' lead over the reference, as a
// power of two, that moves it: weights stay below 2^(kLazy + kShift).  fp16, whose
// least part is 2^-24, holds them as large as it can, below 2^15; else they stay
// below 2^-30: of 2^30 values of the type's largest size the sum is finite.
// Zero times an infinite value is NaN, though a weight is above zero however it
// rounds.  So where joined sums show NaN (of 16-bit caches; e4m3 has no infinity),
// the workgroup goes over the segment's keys again with no part below kLeast and no
// sum scaled by less than kLeastFactor, and takes from that what was NaN; nothing else
// sees it.  (Looked for in each tile: one sequence of 1000 keys 11.8 -> 13.1 us.)
constexpr float kLeastFactor = 0x1p-120f;
template <int CT>
struct Kind;
template <>
struct Kind<W4A8_TYPE_BF16> {
    static __device__ __forceinline__ v4f mfma(const v4i& a, const v4i& b, const v4f& c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) { return f32x2_to_bf16x2(a, b); }
    static constexpr float kShift = -38.0f, kLazy = 8.0f;
    static constexpr uint32_t kLeast = 0x00800080;  // 2^-126
    static __device__ __forceinline__ void split(float a, float b, uint32_t least, int& hi, int& lo)
    {
        hi = raised(cut(a, b), least);
        lo = raised(pack(a, b), least);
    }
    // the values cut to the type; a and b become the rest
    static __device__ __forceinline__ uint32_t cut(float& a, float& b)
    {
        const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
        a -= __uint_as_float(__float_as_uint(a) & 0xFFFF0000u);
        b -= __uint_as_float(__float_as_uint(b) & 0xFFFF0000u);
        return hi;
    }
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
    static constexpr float kShift = 14.0f, kLazy = 1.0f;
    static constexpr uint32_t kLeast = 0x00010001;  // 2^-24
    static __device__ __forceinline__ void split(float a, float b, uint32_t least, int& hi, int& lo)
    {
        const auto h = __builtin_amdgcn_cvt_pkrtz(a, b);
        hi = raised(__builtin_bit_cast(uint32_t, h), least);
        lo = raised(pack(a - (float)h[0], b - (float)h[1]), least);
    }
};
template <>
struct Kind<W4A8_TYPE_E4M3> : Kind<W4A8_TYPE_BF16> {
    static __device__ __forceinline__ void split(float a, float b, uint32_t, int& hi, int& lo)
    {
        hi = (int)cut(a, b);
        lo = (int)pack(fmaxf(a, 0.0f), fmaxf(b, 0.0f));  // under an infinite scale the rest is NaN
    }
};

// ln of a sum l of weights times 2^kShift, whose reference is m
template <class K>
__device__ __forceinline__ float lse_of(float m, float l)
{
    return (m + __builtin_amdgcn_logf(__builtin_amdgcn_ldexpf(l, -(int)K::kShift))) * kLn2;
}

// two of a dword's four e4m3 codes -> two bf16 (exact)
template <bool HIGH>
__device__ __forceinline__ uint32_t fp8x2_to_bf16(uint32_t d)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, HIGH));
}

// tiles of 32 keys that a wave takes at a time: 16 KB of cache where registers
// hold it (e4m3, D 128: 148 us with one, 142 with two; D 64: 185 and 179; pages
// without whole runs need registers for their places: 48 with one, 50 with two)
constexpr int tiles_of(int ct, int dp, bool runs)
{
    return runs && dp != 256 && (ct == W4A8_TYPE_E4M3 || dp == 64) ? 2 : 1;
}
// waves of a workgroup (uncut, 37 sequences under a window of 1000: 4 waves 21 us,
// 8 waves 14.6; with D 256 a wave's registers leave room for 4)
constexpr int waves_of(int dp, bool cut)
{
    return cut || dp == 256 ? 4 : 8;
}

template <typename T>
__device__ __forceinline__ T load(const char* p)
{
    return *(const T*)p;
}
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
template <int BYTES>
struct Chunk;
template <>
struct Chunk<4> {
    typedef uint32_t T;
};
template <>
struct Chunk<8> {
    typedef v2u T;
};
template <>
struct Chunk<16> {
    typedef v4i T;
};

}  // namespace

// CT: type of the cache.  DP: D rounded up to 64, 128 or 256.  PAD: kShort if D <
// DP, whose chunks past D are not read; kApart where rows of codes are not whole
// pieces of 16 aligned bytes and go 8 by 8 (64 x 4096 keys, 8 heads of 96: 119 us, kShort 107).
// RUNS: pages hold whole runs of 8 keys, so a lane's 8 keys share a page.  Else
// each lane looks up one key of the tile, ahead as for runs, and hands its page
// round (64 x 4096 keys, bf16, pages of 60: 195 us; each lane looking up its own keys,
// a load behind a load, 288).
// PAIR: two neighbouring kv heads of 64 whose rows lie side by side are read as
// rows of 128.  Each has its own scores, of which a lane keeps those of its
// column's head; the sums are of both, and its head's are stored.
template <int CT, int DP, int PAD, bool RUNS, bool CUT, bool PAIR>
__global__ __launch_bounds__(64 * waves_of(DP, CUT), DP == 256 ? 1 : 2) void attn_decode_kernel(const Plan p)
{
    constexpr int kWaves = waves_of(DP, CUT);
    constexpr int NT = tiles_of(CT, DP, RUNS);  // tiles of 32 keys that a wave takes at a time
    constexpr int kTile = 32 * NT;
    using K = Kind<CT>;
    constexpr bool FP8 = CT == W4A8_TYPE_E4M3;
    constexpr int kElem = FP8 ? 1 : 2;
    static_assert(!PAIR || (DP == 128 && !PAD), "pairs of heads of 64");
    constexpr int kSteps = DP / 32;                       // MFMA steps over d
    constexpr int kQSteps = PAIR ? kSteps / 2 : kSteps;   // of one head
    constexpr int kKLoads = FP8 ? DP / 64 : DP / 32;      // 16-byte loads of a lane's key row
    constexpr int kPer = DP == 64 ? 4 : 8;                // elements of a lane's chunk of a value row
    constexpr int kHalves = DP == 256 ? 2 : 1;            // chunks of a lane
    constexpr int kOut = kPer * kHalves;                  // products over d
    using VChunk = typename Chunk<kPer * kElem>::T;
    constexpr int kVWords = kPer * kElem / 4;

    int me = (int)blockIdx.x;
    const AttnArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, c16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    __shared__ float sh_o[kWaves][kOut * 4][64];
    __shared__ float2 sh_ml[kWaves][kHeads];
    __shared__ int sh_nan;  // whether a sum of the segment is
    if (tid == 0)
        sh_nan = 0;
    // where this workgroup's work begins
    int64_t u = 0, u_end = 0;  // in units of the whole batch
    int b = 0;
    int64_t b_first = 0;       // first unit of sequence b
    const int lens0 = CUT && lane < a.B ? a.lens[lane] : 0;  // of the first 64
    auto units_at = [&](int i) {  // of sequence i, i % 64 == lane if it is below 64
        int s, e;
        span_of(a, i < 64 ? lens0 : i < a.B ? a.lens[i] : 0, s, e);
        return (int64_t)units_of(s, e);
    };
    if (CUT) {
        // every wave for itself, 64 sequences at a time: no barrier, and one load for a batch of up to 64
        const int64_t first = units_at(lane);
        int64_t total = first;
#pragma unroll 4
        for (int at = 64; at < a.B; at += 64)
            total += units_at(at + lane);
        total = uniform(wave_scan(total, lane), 63) * p.items;
        const int in_use = (int)min((int64_t)p.workgroups, total);
        if (blockIdx.x == 0 && wave == 0) {  // for the join
            if (lane == 0) {
                p.header[0] = total;
                p.header[1] = in_use;
            }
            int64_t before = 0;
            for (int at = 0; at < a.B; at += 64) {
                const int64_t n = at ? units_at(at + lane) : first, sum = wave_scan(n, lane);
                if (at + lane < a.B)
                    p.header[3 + at + lane] = (before + sum) * p.items;
                if (at + lane == 0)
                    p.header[2] = 0;
                before += uniform(sum, 63);
            }
        }
        if (me >= in_use)
            return;
        if (FP8 || DP == 64 || PAIR)
            me = eighths(me, in_use);
        u = begin_of(total, in_use, me);
        u_end = begin_of(total, in_use, me + 1);
        int64_t before = 0;
        for (int at = 0; at < a.B; at += 64) {
            const int64_t n = at ? units_at(at + lane) : first, sum = wave_scan(n, lane);
            const uint64_t behind = __ballot((before + sum) * p.items > u);
            if (behind != 0) {
                const int l = __builtin_ctzll(behind);
                b = at + l;
                b_first = (before + uniform(sum - n, l)) * p.items;
                break;
            }
            before += uniform(sum, 63);
        }
    }

    const float c = a.scale * kLog2e;
    for (int segment = 0;; ++segment) {
        int start, end, item, unit0, unit1, units;
        if (CUT) {
            if (u >= u_end)
                break;
            span_of(a, b < 64 ? __builtin_amdgcn_readlane(lens0, b) : a.lens[b], start, end);
            units = units_of(start, end);
            if (u >= b_first + (int64_t)units * p.items) {
                b_first += (int64_t)units * p.items;
                // the next sequence with something in it: there is one, as u < u_end
                // (the bound ends the loop if the lengths change under it)
                uint64_t some = 0;
                for (int at = (b + 1) & ~63; some == 0 && at < a.B; at += 64) {
                    some = __ballot(at + lane > b && at + lane < a.B && units_at(at + lane) > 0);
                    if (some != 0)
                        b = at + __builtin_ctzll(some);
                }
                if (some == 0)
                    break;
                --segment;
                continue;
            }
            item = (int)quotient(u - b_first, units);
            unit0 = (int)(u - b_first - (int64_t)item * units);
            unit1 = (int)min((int64_t)units, unit0 + (u_end - u));
            u += unit1 - unit0;
        } else {
            if (segment > 0)
                break;
            const int id = eighths(me, p.workgroups);
            b = id / p.items;
            item = id - b * p.items;
            span_of(a, a.lens[b], start, end);
            units = units_of(start, end);
            unit0 = 0;
            unit1 = units;
        }
        const int kv = item / p.blocks, head0 = kv * p.group + (item - kv * p.blocks) * kHeads;
        const int heads = min(kHeads, (kv + 1) * p.group - head0);
        const int32_t* table = a.table + b * a.ld_table;

        // the queries: column c16, positions of d as the keys' loads give them
        v4i q[kQSteps];
        {
            const uint16_t* src = (const uint16_t*)a.q + b * a.q_bs + (head0 + min(c16, heads - 1)) * a.q_hs;
#pragma unroll
            for (int s = 0; s < kQSteps; ++s) {
                const int d = FP8 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
                const bool in = c16 < heads && (!PAD || d < a.D);
                q[s] = in ? ldg16(src + d) : v4i{0, 0, 0, 0};
            }
        }
        v4f o[kOut];
        float m, ref, l;

        const int first_kv = PAIR ? 2 * kv : kv, second = PAIR && c16 >= p.group / 2;  // which of a pair is this column's
        const char* const kbase = (const char*)a.kc.p + first_kv * a.kc.hs * kElem;
        const char* const vbase = (const char*)a.vc.p + first_kv * a.vc.hs * kElem;
        const int64_t kts = a.kc.ts * kElem, kps = a.kc.ps * kElem, vts = a.vc.ts * kElem, vps = a.vc.ps * kElem;

        v4i kreg[NT][2][kKLoads];
        VChunk vreg[NT][8][kHalves];
        float ksc[NT][8], vsc[NT][8];
        uint32_t mask = 0;  // which of the lane's keys 32 n + 8 g + j of the tile are there, bit 8 n + j
        constexpr uint32_t kAll = (1u << 8 * NT) - 1;

        // the page of key `key`, or of the run of keys from `key`, as the table has it; -1:
        // nothing of it is seen.  `held` checks it where it is used: here the wave would
        // wait for the table, and with it for all that it has asked for before.
        auto held = [&](int id) { return id >= 0 && id < a.num_pages ? id : -1; };
        auto lookup = [&](int key, int run) {
            if (key + run <= start || key >= end)
                return -1;
            return table[page_of(p, key)];
        };
        auto load_k_row = [&](int n, int t, const char* row) {
#pragma unroll
            for (int i = 0; i < kKLoads; ++i) {
                if (!FP8) {
                    const int d = 32 * i + 8 * g;
                    kreg[n][t][i] = !PAD || d < a.D ? load<v4i>(row + 2 * d) : v4i{0, 0, 0, 0};
                } else if (PAD != kApart) {
                    const int d = 64 * i + 16 * g;
                    kreg[n][t][i] = !PAD || d < a.D ? load<v4i>(row + d) : v4i{0, 0, 0, 0};
                } else {
                    const int d = 64 * i + 16 * g;
                    const uint2 x = d < a.D ? *(const uint2*)(row + d) : make_uint2(0, 0);
                    const uint2 y = d + 8 < a.D ? *(const uint2*)(row + d + 8) : make_uint2(0, 0);
                    kreg[n][t][i] = v4i{(int)x.x, (int)x.y, (int)y.x, (int)y.y};
                }
            }
        };
        auto load_v_row = [&](int n, int j, const char* row) {
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                const int d = 128 * h + kPer * c16;
                if (!PAD || d < a.D)
                    vreg[n][j][h] = load<VChunk>(row + d * kElem);
                else
                    vreg[n][j][h] = VChunk{};
            }
        };
        // a lane's key row of tile t of a pair is key krun + 4 t + c16 % 4; its run of values is from key 8 g
        const int krun = 8 * (c16 >> 2), vrun = 8 * g;
        // the pages of a tile: of the lane's runs, or without whole runs of the
        // tile's key `lane`, which the lanes then ask each other for
        struct Ids {
            int k[NT], v[NT];
        };
        auto lookup_all = [&](int key0) {
            Ids id;
            if (!RUNS)
                id.k[0] = lane < kTile ? lookup(key0 + lane, 1) : -1;
#pragma unroll
            for (int n = 0; RUNS && n < NT; ++n) {
                id.k[n] = lookup(key0 + 32 * n + krun, 8);
                id.v[n] = lookup(key0 + 32 * n + vrun, 8);
            }
            return id;
        };
        auto load_k = [&](int key0, const Ids& id) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (RUNS) {
                    const int key = key0 + 32 * n + krun, page = held(id.k[n]);
                    const int off = page >= 0 ? key - page_of(p, key) * a.page_size : 0;
                    const char* row = kbase + max(page, 0) * kps + (off + (c16 & 3)) * kts;
                    load_k_row(n, 0, row);
                    load_k_row(n, 1, row + 4 * kts);
                } else {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int in = 32 * n + krun + 4 * t + (c16 & 3), key = key0 + in;
                        const int one = held(__shfl(id.k[0], in, 64));
                        const int off = one >= 0 ? key - page_of(p, key) * a.page_size : 0;
                        load_k_row(n, t, kbase + max(one, 0) * kps + off * kts);
                    }
                }
            }
        };
        auto load_v = [&](int key0, const Ids& id) {
            mask = 0;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int key = key0 + 32 * n + vrun;
                if (RUNS) {
                    const int id_v = held(id.v[n]), page = max(id_v, 0);
                    const int off = id_v >= 0 ? key - page_of(p, key) * a.page_size : 0;
                    const char* row = vbase + page * vps + off * vts;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        load_v_row(n, j, row + j * vts);
                    const int lo = max(start - key, 0), hi = min(end - key, 8);
                    if (id_v >= 0)
                        mask |= ((0xFFu << lo) & (0xFFu >> (8 - hi)) & 0xFFu) << (8 * n);
                    if (FP8) {
                        const int64_t at = ((int64_t)page * a.kv_heads + first_kv + second) * a.page_size + off;
#pragma unroll
                        for (int j = 0; j < 8; j += 4) {
                            const float4 x = *(const float4*)(a.kc.scales + at + j), y = *(const float4*)(a.vc.scales + at + j);
                            ksc[n][j] = x.x, ksc[n][j + 1] = x.y, ksc[n][j + 2] = x.z, ksc[n][j + 3] = x.w;
                            vsc[n][j] = y.x, vsc[n][j + 1] = y.y, vsc[n][j + 2] = y.z, vsc[n][j + 3] = y.w;
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int one = held(__shfl(id.k[0], 32 * n + vrun + j, 64));
                        const int off = one >= 0 ? key + j - page_of(p, key + j) * a.page_size : 0;
                        load_v_row(n, j, vbase + max(one, 0) * vps + off * vts);
                        if (FP8) {
                            const int64_t at = ((int64_t)max(one, 0) * a.kv_heads + first_kv + second) * a.page_size + off;
                            ksc[n][j] = a.kc.scales[at];
                            vsc[n][j] = a.vc.scales[at];
                        }
                        mask |= (one >= 0 ? 1u : 0u) << (8 * n + j);
                    }
                }
            }
        };

        // the segment's keys, in tiles that the waves take in turn
        constexpr int kStep = kTile * kWaves;
        const int seg0 = (start / kUnit + unit0) * kUnit, seg1 = min((start / kUnit + unit1) * kUnit, end);
        uint32_t nan = 0;  // which of the lane's joined sums are
        // careful: again, for those
        auto attend = [&](auto careful) {
            constexpr bool kCareful = decltype(careful)::value;
            constexpr uint32_t least = kCareful ? K::kLeast : 0;
            constexpr float least_factor = kCareful ? kLeastFactor : 0.0f;
#pragma unroll
            for (int i = 0; i < kOut; ++i)
                o[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            m = -__builtin_inff(), ref = -K::kShift, l = 0.0f;
            int key0 = seg0 + wave * kTile;
            while (key0 < seg1 && key0 + kTile <= start)
                key0 += kStep;
            Ids ids;
            if (!CUT && RUNS && a.window == 0) {
                // the first tile's place is known without the length: its pages are
                // looked up while the length is on its way
                auto early = [&](int key) {
                    const int id = table[min(page_of(p, key), a.max_pages - 1)];
                    return key < end ? id : -1;
                };
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    ids.k[n] = early(wave * kTile + 32 * n + krun);
                    ids.v[n] = early(wave * kTile + 32 * n + vrun);
                }
            } else {
                ids = lookup_all(key0 < seg1 ? key0 : end);
            }
            // a tile; more: whether the wave has another behind it
            auto tile = [&](auto is_more) {
                const bool more = is_more;
                v4f s[NT][2], s1[PAIR ? NT : 1][2];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        s[n][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
                        if (PAIR)
                            s1[PAIR ? n : 0][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
                    }
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            v4i x;
                            if (FP8) {
                                const v4i& r = kreg[n][t][k >> 1];
                                const uint32_t d0 = (uint32_t)r[2 * (k & 1)], d1 = (uint32_t)r[2 * (k & 1) + 1];
                                x = v4i{(int)fp8x2_to_bf16<false>(d0), (int)fp8x2_to_bf16<true>(d0), (int)fp8x2_to_bf16<false>(d1),
                                        (int)fp8x2_to_bf16<true>(d1)};
                            } else {
                                x = kreg[n][t][FP8 ? 0 : k];
                            }
                            v4f& sum = k < kQSteps ? s[n][t] : s1[PAIR ? n : 0][t];
                            sum = K::mfma(x, q[k % kQSteps], sum);
                        }
                Ids next = ids;
                if (more) {
                    if (key0 + 2 * kStep < seg1)
                        next = lookup_all(key0 + 2 * kStep);
                    load_k(key0 + kStep, ids);
                }
                // scores in powers of two; those that are not there are -inf
                float x[NT][8];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[n][j] = (PAIR && second ? s1[PAIR ? n : 0][j >> 2][j & 3] : s[n][j >> 2][j & 3]) *
                                  (FP8 ? c * ksc[n][j] : c);
                const bool whole = __all(mask == kAll);
                if (!whole) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            x[n][j] = mask >> (8 * n + j) & 1 ? x[n][j] : -__builtin_inff();
                }
                float top = x[0][0];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        top = fmaxf(top, x[n][j]);
                if (__any(top > m + K::kLazy)) {
                    top = fmaxf(top, __shfl_xor(top, 16, 64));
                    top = fmaxf(top, __shfl_xor(top, 32, 64));
                    const float high = fmaxf(m, top);
                    const float next_ref = high == -__builtin_inff() ? 0.0f : high;
                    const float f = fmaxf(exp2_(m - next_ref), least_factor);
                    l *= f;
#pragma unroll
                    for (int i = 0; i < kOut; ++i)
                        o[i] *= f;
                    m = high;
                    ref = next_ref - K::kShift;
                }
                if (!whole) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (!(mask >> (8 * n + j) & 1)) {
                                vsc[n][j] = 0.0f;
#pragma unroll
                                for (int h = 0; h < kHalves; ++h)
                                    vreg[n][j][h] = VChunk{};
                            }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    // the weights as a value of the type and the rest: the products'
                    // error is that of their sums (one rounding alone would add an
                    // error as large as the result's)
                    v4i ph, pl;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float w0 = exp2_(x[n][2 * j] - ref), w1 = exp2_(x[n][2 * j + 1] - ref);
                        l += w0 + w1;
                        if (FP8) {
                            w0 *= vsc[n][2 * j];
                            w1 *= vsc[n][2 * j + 1];
                        }
                        int hi, lo;
                        K::split(w0, w1, least, hi, lo);
                        ph[j] = hi;
                        pl[j] = lo;
                    }
                    auto add = [&](int i, const v4i& e) {
                        o[i] = K::mfma(e, ph, o[i]);
                        o[i] = K::mfma(e, pl, o[i]);
                    };
#pragma unroll
                    for (int h = 0; h < kHalves; ++h)
#pragma unroll
                        for (int d = 0; d < kVWords; ++d) {
                            uint32_t word[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                word[j] = ((const uint32_t*)&vreg[n][j][h])[d];
                            if (!FP8) {  // two elements of eight keys
                                v4i lo, hi;
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    lo[j] = (int)__builtin_amdgcn_perm(word[2 * j + 1], word[2 * j], 0x05040100u);
                                    hi[j] = (int)__builtin_amdgcn_perm(word[2 * j + 1], word[2 * j], 0x07060302u);
                                }
                                add(kPer * h + 2 * d, lo);
                                add(kPer * h + 2 * d + 1, hi);
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
                                    add(kPer * h + 4 * d + i, e[i]);
                            }
                        }
                }
                if (more) {
                    load_v(key0 + kStep, ids);
                    ids = next;
                }
            };
            if (key0 < seg1) {
                load_k(key0, ids);
                load_v(key0, ids);
                if (key0 + kStep < seg1)
                    ids = lookup_all(key0 + kStep);
                if (FP8) {
                    for (; key0 < seg1; key0 += kStep)
                        tile(key0 + kStep < seg1);
                } else {
                    // The last tile stands by itself: with the loads of the next under a condition
                    // there are ways round the loop, never taken, for which the first product
                    // would wait for the values too (128 x 120 keys: 23.4 us, so 21.4)
                    for (; key0 + kStep < seg1; key0 += kStep)
                        tile(std::true_type{});
                    tile(std::false_type{});
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
                f[w] = fmaxf(exp2_(ml[w].x - all_ref), least_factor);
                all_l += ml[w].y * f[w];
            }
            const bool done = !CUT || (unit0 == 0 && unit1 == units);
            const int64_t slot = 2 * (int64_t)me + (segment > 0);
            const float inv = all_l == 0.0f ? 0.0f : 1.0f / all_l;  // NaN stays
            // register r of the products of a half: elements kPer * (4 g + r) .. of column c16
            for (int it = wave; it < 4 * kHalves; it += kWaves) {
                const int r = it & 3, h = it >> 2;
                float y[kPer];
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    y[i] = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWaves; ++w)
                        y[i] += sh_o[w][4 * (kPer * h + i) + r][lane] * f[w];
                }
                const int row_d = 128 * h + kPer * (4 * g + r), d = PAIR ? row_d & 63 : row_d;
                if (c16 < heads && (PAIR ? row_d >> 6 == second : d < a.D)) {
                    if (!FP8 && !kCareful && __builtin_expect(not_finite(y), 0)) {
#pragma unroll
                        for (int i = 0; i < kPer; ++i)
                            nan |= (y[i] != y[i] ? 1u : 0u) << (it / kWaves * kPer + i);
                        if (nan != 0)
                            sh_nan = 1;
                    }
                    if (kCareful) {
#pragma unroll
                        for (int i = 0; i < kPer; ++i) {
                            if (nan >> (it / kWaves * kPer + i) & 1) {
                                if (done)
                                    ((uint16_t*)a.out)[b * a.o_bs + (head0 + c16) * a.o_hs + d + i] =
                                        (uint16_t)K::pack(y[i] * inv, 0.0f);
                                else
                                    p.part_o[(slot * kHeads + c16) * a.D + d + i] = y[i];
                            }
                        }
                        continue;
                    }
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
            if (!kCareful && wave == 0 && g == 0 && c16 < heads) {
                if (!done)
                    p.part_ml[slot * kHeads + c16] = make_float2(all_m, all_l);
                else if (a.lse != nullptr)
                    a.lse[(int64_t)b * a.q_heads + head0 + c16] = lse_of<K>(all_m, all_l);
            }
            __syncthreads();  // before the next segment writes into LDS
        };
        attend(std::false_type{});
        if (!FP8 && __builtin_expect(__builtin_amdgcn_readfirstlane(sh_nan) != 0, 0)) {
            attend(std::true_type{});
            if (tid == 0)
                sh_nan = 0;
            __syncthreads();
        }
    }
}

// Joins what was cut: a workgroup takes ROWS query heads of one (sequence, kv
// head, block of 16).  ROWS 16: a wave takes a head at a time; 1: the waves split its parts.  Nothing
// to do where the work lay in one workgroup; zeros where there was none.
template <bool F16, int ROWS>
__global__ __launch_bounds__(64 * kJoinWaves) void attn_join_kernel(const Plan p, const int32_t parts)
{
    using K = Kind<F16 ? W4A8_TYPE_FP16 : W4A8_TYPE_BF16>;
    constexpr int kSplit = ROWS == 1 ? kJoinWaves : 1;  // waves that share a row
    constexpr int kMost = 4;                        // elements of a lane
    __shared__ float sh[kSplit][64 * kMost];
    const AttnArgs& a = p.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = (int64_t)blockIdx.x / parts;  // sequence and item
    const int b = (int)(id / p.items), item = (int)(id - (int64_t)b * p.items);
    const int kv = item / p.blocks, head0 = kv * p.group + (item - kv * p.blocks) * kHeads;
    const int heads = min(kHeads, (kv + 1) * p.group - head0);
    const int64_t total = p.header[0];
    const int in_use = (int)p.header[1];
    const int64_t b0 = p.header[2 + b], units = quotient(p.header[3 + b] - b0, p.items);
    const int64_t u0 = b0 + item * units, u1 = u0 + units;
    int w0 = 0, w1 = -1, later = 0;  // workgroups that hold a part; w0's may not be its first
    if (units > 0) {
        w0 = holder_of(total, in_use, u0);
        w1 = holder_of(total, in_use, u1 - 1);
        later = begin_of(total, in_use, w0) < u0;
        if (w0 == w1)
            return;
    }
    auto slot_of = [&](int w) { return (2 * (int64_t)w + (w == w0 ? later : 0)) * kHeads; };
    const int first = (int)((int64_t)blockIdx.x - id * parts) * ROWS + (ROWS == 1 ? 0 : wave);
    for (int row = first; row < heads && row < first + ROWS; row += ROWS == 1 ? 1 : kJoinWaves) {
        float m = -__builtin_inff(), l, y[kMost];
        for (int w = w0 + lane; w <= w1; w += 64)
            m = fmaxf(m, p.part_ml[slot_of(w) + row].x);
        m = group_max<64>(m);
        const float ref = m == -__builtin_inff() ? 0.0f : m;
        // the parts' sums, each times its factor, but no less than `least`
        auto sums = [&](float least, float (&sum)[kMost]) {
            l = 0.0f;
#pragma unroll
            for (int k = 0; k < kMost; ++k)
                sum[k] = 0.0f;
            for (int at = w0; at <= w1; at += 64) {
                float f = 0.0f;
                if (at + lane <= w1) {
                    const float2 ml = p.part_ml[slot_of(at + lane) + row];
                    f = exp2_(ml.x - ref);
                    l += ml.y * f;
                    f = fmaxf(f, least);
                }
                const int n = min(64, w1 - at + 1);
                for (int i0 = ROWS == 1 ? wave : 0; i0 < n; i0 += 4 * kSplit) {
                    float v[4][kMost];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float* src = p.part_o + (slot_of(at + min(i0 + j * kSplit, n - 1)) + row) * a.D;
#pragma unroll
                        for (int k = 0; k < kMost; ++k)
                            v[j][k] = lane + 64 * k < a.D ? src[lane + 64 * k] : 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int i = i0 + j * kSplit;
                        if (i < n) {
                            const float g = __shfl(f, i, 64);
#pragma unroll
                            for (int k = 0; k < kMost; ++k)
                                sum[k] = fmaf(v[j][k], g, sum[k]);
                        }
                    }
                }
            }
        };
        sums(0.0f, y);
        if (__builtin_expect(__any(not_finite(y)), 0)) {  // perhaps an infinite sum times 0
            float z[kMost];
            sums(kLeastFactor, z);
#pragma unroll
            for (int k = 0; k < kMost; ++k)
                y[k] = y[k] != y[k] ? z[k] : y[k];
        }
        l = group_sum<64>(l);
        if (ROWS == 1) {
#pragma unroll
            for (int k = 0; k < kMost; ++k)
                sh[wave][64 * k + lane] = y[k];
            __syncthreads();
            if (wave != 0)
                return;
#pragma unroll
            for (int k = 0; k < kMost; ++k) {
                y[k] = 0.0f;
#pragma unroll
                for (int w = 0; w < kSplit; ++w)
                    y[k] += sh[w][64 * k + lane];
            }
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t* out = (uint16_t*)a.out + b * a.o_bs + (head0 + row) * a.o_hs;
#pragma unroll
        for (int k = 0; k < kMost; ++k)
            if (lane + 64 * k < a.D)
                out[lane + 64 * k] = (uint16_t)K::pack(y[k] * inv, 0.0f);
        if (lane == 0 && a.lse != nullptr)
            a.lse[(int64_t)b * a.q_heads + head0 + row] = lse_of<K>(m, l);
    }
}

namespace {

// workgroups that share what is cut: one or two for each CU, as their registers allow
int64_t workgroups_of(int64_t D)
{
    return D > 128 ? 256 : 512;
}

// Whether sequences are cut over workgroups, by what one of the n (sequence, kv
// head) can hold at most.  Uncut, one CU streams 45 GB/s of it after 7 us; cut,
// all share it, but the partial results and their join take 12 us and more.
// Measured (bf16, D 128, 8 kv heads; uncut / cut, us): 1 sequence of 500
// keys 9.1 / 12.5, of 1000 14.5 / 12.3; 8 of 1000 15.7 / 17.5, of 2000 26.8 /
// 21.8; 32 of 2000 50.8 / 60.5, of 125 to 4000 65.9 / 45.5.
bool cuts(int64_t n, int64_t bytes)
{
    return bytes > (n >= 256 ? 1 << 20 : n >= 64 ? 1 << 19 : 1 << 18);
}

// Whether kv heads of 64 are taken two by two, which reads rows of twice the bytes
// and shares the softmax's instructions: where there are enough for all CUs, or
// where they are cut and enough that the join does not get longer.  `placed`: by where the cache
// lies too.  8 kv heads, single / paired, us: 64 x 4096 keys, e4m3 82 / 62, bf16 114 /
// 112, up to 4096 55 / 42; 64 x 16384 308 / 226 and 434 / 397; 4 x 20000 37 / 29
// and 41.6 / 39.1; but 32 x 4096 uncut 37 / 48 and 60 / 70; 2 x 20000 bf16 26 / 29.
bool pairs(const AttnArgs& a, int32_t group, bool cut, bool placed)
{
    const int64_t n = (int64_t)a.B * a.kv_heads;
    if (a.D != 64 || a.kv_heads % 2 != 0 || group > kHeads / 2 || n < (cut ? 32 : 512))
        return false;
    const uint64_t strides = a.kc.ps | a.kc.ts | a.vc.ps | a.vc.ts;
    return !placed || (a.kc.hs == 64 && a.vc.hs == 64 && (strides & 15) == 0 &&
                       (((uintptr_t)a.kc.p | (uintptr_t)a.vc.p) & 15) == 0);
}

Plan plan(void* ws, const AttnArgs& a, size_t* bytes)
{
    Plan p = {};
    p.a = a;
    p.group = a.q_heads / a.kv_heads;
    p.blocks = (p.group + kHeads - 1) / kHeads;
    p.items = a.kv_heads * p.blocks;
    const int64_t longest = (int64_t)a.max_pages * a.page_size;
    const int64_t row = 2 * a.D * (a.cache_type == W4A8_TYPE_E4M3 ? 1 : 2), n = (int64_t)a.B * p.items;
    const int64_t most = row * (a.window > 0 && a.window < longest ? a.window : longest);
    p.cut = cuts(n, most);
    const bool paired_cut = p.cut || (pairs(a, p.group, false, false) && cuts(n / 2, 2 * most));
    if (pairs(a, p.group, p.cut, true)) {
        p.pair = 1;
        p.cut = paired_cut;
        p.group *= 2, p.items /= 2;
    }
    p.workgroups = (int32_t)(p.cut ? workgroups_of(a.D) : (int64_t)a.B * p.items);
    // 2^l >= s > 2^(l - 1): m = ceil(2^(31 + l) / s) is below 2^32, and m s exceeds
    // 2^(31 + l) by less than s, so n m / 2^(31 + l) exceeds n / s by less than
    // n / 2^(31 + l) <= n 2^-31 / s, which is below 1 / s and carries over no integer
    int l = 0;
    while (((int64_t)1 << l) < a.page_size)
        ++l;
    p.page_mul = (uint32_t)((((uint64_t)1 << (31 + l)) + a.page_size - 1) / a.page_size);
    p.page_shift = l;
    api::Carve c(ws);
    if (paired_cut) {  // what a cache of any layout needs
        p.header = c.take<int64_t>((size_t)a.B + 3);
        p.part_o = c.take<float>((size_t)(2 * workgroups_of(a.D)) * kHeads * a.D);
        p.part_ml = c.take<float2>((size_t)(2 * workgroups_of(a.D)) * kHeads);
    }
    *bytes = c.used;
    return p;
}

template <int CT, int DP, int PAD, bool RUNS, bool PAIR>
void launch4(const Plan& p, hipStream_t s)
{
    const dim3 grid((unsigned)p.workgroups);
    if (p.cut)
        hipLaunchKernelGGL((attn_decode_kernel<CT, DP, PAD, RUNS, true, PAIR>), grid, dim3(64 * waves_of(DP, true)), 0, s, p);
    else
        hipLaunchKernelGGL((attn_decode_kernel<CT, DP, PAD, RUNS, false, PAIR>), grid, dim3(64 * waves_of(DP, false)), 0, s, p);
}
template <int CT, int DP, int PAD, bool PAIR = false>
void launch3(const Plan& p, hipStream_t s)
{
    if (p.a.page_size % 8 == 0)
        launch4<CT, DP, PAD, true, PAIR>(p, s);
    else
        launch4<CT, DP, PAD, false, PAIR>(p, s);
}
template <int CT, int DP>
void launch2(const Plan& p, hipStream_t s)
{
    const AttnArgs& a = p.a;
    const bool apart = ((((uintptr_t)a.kc.p | (uintptr_t)a.vc.p | (uintptr_t)(a.kc.ps | a.kc.ts | a.kc.hs) |
                          (uintptr_t)(a.vc.ps | a.vc.ts | a.vc.hs)) | (uintptr_t)a.D) & 15) != 0;
    if (CT == W4A8_TYPE_E4M3 && apart)
        launch3<CT, DP, CT == W4A8_TYPE_E4M3 ? kApart : kShort>(p, s);
    else if (a.D != DP)
        launch3<CT, DP, kShort>(p, s);
    else
        launch3<CT, DP, kWhole>(p, s);
}
template <int CT>
void launch1(const Plan& p, hipStream_t s)
{
    if (p.pair)
        launch3<CT, 128, kWhole, true>(p, s);
    else if (p.a.D <= 64)
        launch2<CT, 64>(p, s);
    else if (p.a.D <= 128)
        launch2<CT, 128>(p, s);
    else
        launch2<CT, 256>(p, s);
}

template <bool F16>
hipError_t launch_join(const Plan& p, hipStream_t s)
{
    // few: a workgroup for each head, for whose parts many waves can ask at once
    const int64_t n = (int64_t)p.a.B * p.items;
    const int32_t rows = p.group < kHeads ? p.group : kHeads;
    if (n >= 256)
        hipLaunchKernelGGL((attn_join_kernel<F16, kHeads>), dim3((unsigned)n), dim3(64 * kJoinWaves), 0, s, p, 1);
    else
        hipLaunchKernelGGL((attn_join_kernel<F16, 1>), dim3((unsigned)(n * rows)), dim3(64 * kJoinWaves), 0, s, p, rows);
    return hipGetLastError();
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
    return a.q_type == W4A8_TYPE_FP16 ? launch_join<true>(p, s) : launch_join<false>(p, s);
}

}  // namespace w4a8
