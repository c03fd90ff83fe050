// kv4_prompt_impl.h -- attention over the 4-bit cache for many rows a key head
// (prompts, and chunks of them): bound by the matrix cores and the vector
// ALU beside them, where kv4_attn_impl.h is bound by what it reads.
//
// A work-group of 8 waves takes 256 rows, a wave 32 of them, and walks the keys
// 64 at a time (32 where the head has 256 dimensions).  Four waves turn the keys'
// codes into operands and four the values', once for all 256 rows, into LDS (one
// barrier a tile, two buffers for keys, three for values) in the order in which
// the products read them: 16 bytes a lane, lane after lane.  With two waves on a
// SIMD there is little to hide one wave's waits, so the exponentials of 32 keys
// stand among the products for the scores of the next 32.
//
// Measured: a prompt of 8192 tokens, 32 heads of 128 on 8 key heads, groups of 64,
// bfloat16: 670 to 700 us in a warm loop, 785 to 820 TFLOP/s, where a library matrix
// product reaches 1209.  The matrix cores are busy 38 % of the cycles and the vector
// ALU 56 %, 15 % both at once: a barrier a tile holds the waves together, and they do
// the same things at the same time.  Setting half the waves half a tile off, or a
// priority for those at the products, changed nothing (1 %).  Turning the codes
// costs a sixth.  Keys of rounded numbers instead of exact scores took the same
// time, with scores off by 2^-12 each.  Groups of 32 and 128: 716 and 657 where 64
// take 670; heads of 64 491; float16 940 (groups of 32 2080, of 128 910; heads of 64
// 650).  What is spilled: of float16 at 128, 1 register in groups of 128, 15 of 64
// and 60 of 32; at 256, 8 to 39.
//
//   S^T[key, row] = K Q^T,  O^T[dim, row] += V^T P:  v_mfma_32x32x16, where the
//   probabilities that a lane computes are the operand it needs (as in
//   kv4_attn_impl.h), the values' tokens being put into that order.
//
// A code c becomes an operand from the bits of the float16 number c 2^-18 or
// 16 + c, which is exact, in one multiply-add.  Queries are float16, brought under
// 2^15 by a power of two a row (exact, but for what is under 2^-29 of the row's
// largest and keeps 2^-40 of it).
//
// Keys of bfloat16 scales: s (c - 8) has 8 + 3 bits, so float16 holds it exactly,
// the block of 16 tokens brought under 2^14 by a power of two that goes into the
// softmax scale (what is under 2^-28 of the block's largest keeps 2^-39 of it).  A
// block whose tokens are more than 2^8 apart has a power a token, which the scores
// are multiplied by: another token's keys, seen or not, cost none of a key's
// digits.  What is left, b + 8 s, times the sums of the queries is a first step of
// the product: b and s by the sums in three bfloat16 pieces each, which hold 24
// bits.  Keys of float16 scales (11 bits) stay codes, and a group's product is
// multiplied by the token's scale in 32 bits.  Either way scores are as exact as
// their 32-bit sums.
//
// Values become c s + b divided by a power of two: one for the tile where its
// tokens are within 2^5 of each other, else one a token.  A row's sums have a power
// of their own, the largest of the tokens that it sees; what is left goes to the
// probability.  So a token that a row does not see costs it no digits, however
// large.  As long as a tile has the power of all rows' sums, as nearly always,
// that is one comparison of scalars.  Values and probabilities are rounded to
// float16, half a step 2^-11, as the matrix cores need (bfloat16 would cost eight
// times that); values also to 2^-18 of their token's largest, and a probability
// times a value to 2^-26 of the largest that the row sees.  All sums are float32.
// One power of two for all values so far, seen or not, took 1 to 4 % less time.
//
// Where the output is float16 too, both roundings show beside its own: off by
// 3.2e-4 of the exact result where float32 products are off by 2.1e-4.  So there
// what a probability loses enters as a second float16 number: 2.8e-4, for half as
// many products again and 24 vector instructions per 32 keys (12 requests over
// 4000 keys, heads of 256: 184 -> 201 us; 8192 tokens, heads of 128: 725 -> 940).
// bfloat16 outputs are off by 1.7e-3 either way.
//
// 0 * NaN is NaN in a product, so values that are not finite are entered as 0
// and added afterwards to the rows that see them (a tile that holds one is rare
// and says so).
#pragma once

#include "kv4_attn_impl.h"

namespace qmx {
namespace kv4 {

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

// The product of biases, in the cache's type.
template <int DT>
__device__ __forceinline__ f32x16 mfma32_type(u32x4 a, u32x4 b, f32x16 c) {
    if constexpr (DT == DT_F16) return mfma32(a, b, c);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

constexpr int PROMPT_WAVES = 8, PROMPT_ROWS = 256;

// Products and reads of LDS stay in the order of the source, so that operands
// are read a few products ahead; everything else may move.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0x676); }

// The largest of the wave's numbers, none below 0, without a trip through LDS:
// over rows of 16 lanes, then the four rows as integers, which order alike.
__device__ __forceinline__ float wave_max(float v) {
    int x = __float_as_int(v);
#define QMX_ROW_TURN(K) x = max(x, __builtin_amdgcn_mov_dpp(x, 0x120 + K, 0xf, 0xf, true))
    QMX_ROW_TURN(8);
    QMX_ROW_TURN(4);
    QMX_ROW_TURN(2);
    QMX_ROW_TURN(1);
#undef QMX_ROW_TURN
    return __int_as_float(max(max(__builtin_amdgcn_readlane(x, 0), __builtin_amdgcn_readlane(x, 16)),
                              max(__builtin_amdgcn_readlane(x, 32), __builtin_amdgcn_readlane(x, 48))));
}

// The lane.  SHORT of registers: as if not known before, so that what is worked
// out from it in a loop is worked out there, and not spilled from before the loop
// on: a spilled number comes back behind the loads that are on their way.
template <bool SHORT>
__device__ __forceinline__ int lane_of() {
    int lane = threadIdx.x & 63;
    if constexpr (SHORT) asm volatile("" : "+v"(lane));
    return lane;
}

// What the rows need to know of a tile beside its operands.
struct alignas(16) TileInfo {
    static constexpr int MISSING = -1001, OWN = 1000, ZEROS = -1000, NONE = 1001;
    int block[4];   // the keys' exponent; MISSING: no page; OWN: each token has one
    int value_exponent;   // or OWN, or ZEROS
    int bad;        // tile + 1, where it holds values that are not finite
    int unused[2];
};

// What a lane takes of one block of 16 tokens to turn it into operands: codes of
// the D / SPLIT dimensions that fall to its wave, the pairs of one token, and a
// share of the pairs of the four tokens 4h .. 4h + 3, h = lane / 16, as in
// kv4_attn_impl.h.  Keys: the token is the block's lane % 16, whose codes the lane
// has.  Values: the lane has codes of the four tokens; the one token, of all the
// tile's, is for the largest value.
template <int D, int GS, int DT>
struct Raw {
    static constexpr int KEYS = 64 * 128 / (D < 128 ? 128 : D);   // of a tile
    static constexpr int SPLIT = 64 / KEYS;                       // waves that share a block
    static constexpr int NJ = D / 32, G = D / GS, KS = D / 16, DB = D / 32;
    static constexpr int NW = NJ / SPLIT, GW = G / SPLIT;         // words and groups of a wave
    static constexpr bool SCALED = DT == DT_BF16;                 // keys enter the product with their scales
    static constexpr int SLOTS = SCALED ? 8 : 4;                  // of a group in the product of biases
    static constexpr int BK = (SLOTS * G + 15) / 16;              // its steps
    static constexpr int SHARE = (4 * G + 15) / 16;               // a lane's share of a block's pairs
    // Where lane_of is to hide what it knows: 8192 tokens, heads of 128, float16 in
    // groups of 32 2384 us without and 2079 with; heads of 256, 12 requests over 4000
    // keys, float16 220 and 203, bfloat16 166 and 154.  Where little or nothing is
    // spilled it costs 1 to 4 %.
    static constexpr bool SHORT = D == 256 || (DT == DT_F16 && D == 128 && GS == 32);
    // Powers of two that keys, queries and the queries' sums are brought to, and
    // what a score is multiplied by in all.
    static constexpr int KEY_UP = 14, QUERY_UP = 15, SUM_UP = SCALED ? QUERY_UP : 8;
    static constexpr int SCORE_UP = SCALED ? KEY_UP + QUERY_UP : SUM_UP;
    // The same loads for either kind of wave, and no branch about them: where two
    // met in a register, a copy behind them would wait for memory.
    uint32_t w[NW], token_pairs[G], share[SHARE];
    bool there;    // the block's page is in the cache
    bool live;     // the lane's token is there
    int tokens;    // of the block, from its first on, that are there

    // `pages`: entries of 64 blocks of 16 tokens, one a lane, from a tile's start
    // on; the tile's are from `first` on, `key` its first key.
    __device__ __forceinline__ void load(const Kv4View& c, int pages, int first, int head, int key, int my_blk,
                                         int part, int end, bool value) {
        const int lane = lane_of<SHORT>();
        const int page = __builtin_amdgcn_readlane(pages, first + my_blk), blk = (key >> 4) + my_blk;
        const int own = value ? lane % KEYS : 16 * my_blk + (lane & 15);   // the lane's token of the tile
        const int its = __shfl(pages, first + own / 16, 64);
        tokens = end - 16 * blk;
        there = tokens > 0 && page >= 0 && page < c.num_pages;
        live = key + own < end && its >= 0 && its < c.num_pages;
        // what is not there is read from page 0 and not used
        const uint32_t at = block_number(c, there ? page : 0, head, blk);
        const uint32_t row = block_number(c, live ? its : 0, head, (key + own) >> 4);
        const uint32_t* codes = (value ? c.vc : c.kc) + lane * NJ + part * NW;
        const uint32_t* pairs = value ? c.vs : c.ks;
        const uint32_t* own_pairs = pairs + (own & 15) * G;
        const uint32_t* shared = pairs + (lane >> 4) * (4 * G);
        load_words(w, codes + (uint64_t)at * (64 * NJ));
#pragma unroll
        for (int g = 0; g < G; ++g) token_pairs[g] = own_pairs[(uint64_t)row * (16 * G) + g];
#pragma unroll
        for (int r = 0; r < SHARE; ++r)
            share[r] = shared[(uint64_t)at * (16 * G) + ((16 * r + (lane & 15)) & (4 * G - 1))];
    }

    // Keys to `k` [blocks of 32][BK + KS][2][32] of 16 bytes; `blk` counts in the
    // tile.  SCALED: divided by 2^(what is returned), `exponent`, or, where that is
    // OWN, each token by 2^(its `powers` [KEYS]).  Else: the scales to `factor`
    // [G][KEYS].
    __device__ __forceinline__ int keys(u32x4* k, float* factor, int& exponent, int* powers, int blk,
                                        int part) const {
        const int lane = lane_of<SHORT>(), n = lane & 15, h = lane >> 4;
        u32x4* to = k + (blk >> 1) * (BK + KS) * 64 + (blk & 1) * 16 + n;
        int e = 0, result = 0;
        if constexpr (SCALED) {
            float most = 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float x = fmaxf(fabsf(8.0f * half_lo<DT>(token_pairs[g])), fabsf(half_hi<DT>(token_pairs[g])));
                most = x < INFINITY ? fmaxf(most, x) : most;
            }
            const bool zeros = !live || most == 0.0f;
            const int own = power(most);
            auto far = [&] { return __any(!zeros && (uint32_t)(exponent - own) > 8u); };
            result = e = exponent;
            if (far()) {   // not the last block's power: this one's, or one a token
                result = e = exponent = power(wave_max(zeros ? 0.0f : most));
                if (far()) {
                    e = zeros ? e : own;
                    result = TileInfo::OWN;
                    if (part == 0 && h == 0) powers[16 * blk + n] = e;
                }
            }
        }
#pragma unroll
        for (int g = 0; g < GW; ++g) {
            const int group = part * GW + g;
            const uint32_t pair = live ? (SPLIT == 2 && part ? token_pairs[GW + g < G ? GW + g : 0] : token_pairs[g]) : 0u;
            const float s = half_lo<DT>(pair);
            f16x2 s2, b2;
            if constexpr (SCALED) {
                const float x = ldexpf(s, KEY_UP - e);
                s2 = half2_of(x, x);
                b2 = half2_of(-24.0f * x, -24.0f * x);
                if (h == g % 4) {   // 8 slots: three times b, and three times s for 8 s
                    const uint32_t z = Half<DT>::pack(ldexpf(half_hi<DT>(pair), KEY_UP - e), x);
                    const uint32_t b = z & 0xffffu, y = z >> 16;
                    to[(group / 2) * 64 + (group % 2) * 32] = u32x4{b | (b << 16), b, y | (y << 16), y};
                }
            } else if (h == g % 4) {   // 4 slots: three times b
                const uint32_t b = pair >> 16;
                reinterpret_cast<u32x2*>(to + (group / 4) * 64 + (group / 2 % 2) * 32)[group % 2] =
                    u32x2{b | (b << 16), b};
                factor[KEYS * group + 16 * blk + n] = ldexpf(s, 18 - QUERY_UP + SUM_UP);
            }
#pragma unroll
            for (int j = g * (GS / 32); j < (g + 1) * (GS / 32); ++j) {
                u32x4 x;
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const uint32_t y = tiny_codes(w[j], f);
                    x[f] = SCALED ? __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(
                                                                     __builtin_bit_cast(f16x2, y | 0x4c004c00u), s2, b2))
                                  : y;
                }
                to[(BK + 2 * (part * NW + j) + (h >> 1)) * 64 + (h & 1) * 32] = x;
            }
        }
        return result;
    }
    // The power of two above x.  Not under 2^-95: bfloat16 has no digits below
    // 2^-133, which KEY_UP takes to float16's.
    static __device__ __forceinline__ int power(float x) { return max(__builtin_amdgcn_frexp_expf(x), -95); }

    // Values to `v` [blocks of 16][DB][2][32] of 16 bytes, divided by 2^(what is
    // returned), `exponent` or, where the tile holds zeros only, ZEROS; where that
    // is OWN, each token by 2^(its `powers` [KEYS]).  `good`: the tile is finite.
    __device__ __forceinline__ int values(u32x4* v, int& exponent, int* powers, int blk, int part, bool& good) const {
        const int lane = lane_of<SHORT>(), n = lane & 15, h = lane >> 4;
        u32x2* to = reinterpret_cast<u32x2*>(v + ((blk * DB + part * (DB / SPLIT)) * 2 + (h & 1)) * 32 + n) + (h >> 1);
        float most = 0.0f;
        good = true;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float x = half_lo<DT>(token_pairs[g]), y = half_hi<DT>(token_pairs[g]);
            const bool finite = (x - x) + (y - y) == 0.0f;
            good = good && (finite || !live);
            const float z = fmaxf(fabsf(y), fabsf(fmaf(15.0f, x, y)));
            most = live && finite ? fmaxf(most, z) : most;
        }
        const int own = most > 0.0f ? __builtin_amdgcn_frexp_expf(fminf(most, 0x1.fffffep127f)) : TileInfo::ZEROS;
        auto far = [&] { return __any(live && (uint32_t)(exponent - own) > 5u); };
        int result = exponent;
        if (far()) {   // not the last tile's power: this one's, or one a token
            const float all = wave_max(most);
            if (all > 0.0f) exponent = __builtin_amdgcn_frexp_expf(fminf(all, 0x1.fffffep127f));
            result = all == 0.0f ? TileInfo::ZEROS : far() ? TileInfo::OWN : exponent;
            if (result == TileInfo::OWN && blk == 0 && part == 0 && lane < KEYS) powers[lane] = own;
        }
        uint32_t pair[SHARE];   // scale 2^18 and bias, float16
#pragma unroll
        for (int r = 0; r < SHARE; ++r) {
            const float x = half_lo<DT>(share[r]), y = half_hi<DT>(share[r]);
            const int token = 4 * h + ((16 * r + n) & (4 * G - 1)) / G;
            const bool use = there && token < tokens && (x - x) + (y - y) == 0.0f;
            const int e = result == TileInfo::OWN ? __shfl(own, 16 * blk + token, 64) : exponent;
            pair[r] = use ? __builtin_bit_cast(uint32_t, half2_of(ldexpf(x, 18 - e), ldexpf(y, -e))) : 0u;
        }
#pragma unroll
        for (int g = 0; g < GW; ++g) {
            f16x2 s2[2], b2[2];   // of two tokens
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint32_t x[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int at = (2 * p + i) * G + g;
                    x[i] = pair_at(pair, at);
                    if constexpr (SPLIT == 2) x[i] = part ? pair_at(pair, at + GW) : x[i];
                }
                s2[p] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(x[1], x[0], 0x05040100u));
                b2[p] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(x[1], x[0], 0x07060302u));
            }
#pragma unroll
            for (int cb = g * (GS / 16); cb < (g + 1) * (GS / 16); ++cb) {   // 16 dims
                const int a = cb / 4, f = cb % 4;
                u32x2 x;
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    x[p] = __builtin_bit_cast(
                        uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2, tiny_codes(w[2 * a + p], f)),
                                                            s2[p], b2[p]));
                to[2 * ((cb >> 1) * 64 + (cb & 1) * 16)] = x;
            }
        }
        return result;
    }
    static __device__ __forceinline__ uint32_t pair_at(const uint32_t (&pair)[SHARE], int at) {
        return (uint32_t)__float_as_int(row_lane(__int_as_float((int)pair[at / 16]), at % 16));
    }
};

template <int D, int GS, int DT>
__global__ __launch_bounds__(64 * PROMPT_WAVES, 2) void kv4_prompt_kernel(Kv4AttnArgs a) {
    using W = Raw<D, GS, DT>;
    using H = Half<DT>;
    constexpr int KS = D / 16, DB = D / 32, G = D / GS, BK = W::BK, KEYS = W::KEYS, NT = KEYS / 32;
    constexpr int KQ = D == 256 ? KS / 2 : KS;   // steps whose queries stay in registers; the others' in LDS
    constexpr int AHEAD = D == 256 ? 2 : 4;      // operands read ahead
    // The largest score has a probability of 2^8, later ones may reach 2^15: float16
    // holds what is down to 2^-33 of the largest.
    constexpr float kUp = 8.0f, kSlack = 7.0f;
    constexpr float kLeast = -0x1.8p127f;   // under every score
    __shared__ u32x4 s_k[2][NT * (BK + KS) * 64], s_v[3][2 * NT * DB * 64];
    __shared__ u32x4 s_q[PROMPT_WAVES][KS > KQ ? (KS - KQ) * 64 : 1];
    __shared__ float s_factor[2][W::SCALED ? 1 : G * KEYS];
    __shared__ int s_key_power[3][W::SCALED ? KEYS : 1], s_value_power[3][KEYS];
    __shared__ TileInfo s_info[3];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, n = lane & 31, hh = lane >> 5;
    const Kv4View& c = a.c;
    const int head = blockIdx.x % c.heads;
    const bool value = wave >= 4;   // which codes this wave turns into operands
    const int my_blk = (wave & 3) / W::SPLIT, my_part = (wave & 3) % W::SPLIT;

    if (clears(a, blockIdx.x / c.heads, head)) return;
    for (int i = threadIdx.x; i < 2 * NT * BK * 64; i += 64 * PROMPT_WAVES)   // slots that no group has
        s_k[i / (NT * BK * 64)][i / (BK * 64) % NT * (BK + KS) * 64 + i % (BK * 64)] = u32x4{0, 0, 0, 0};

    Units<64 * PROMPT_WAVES> units(a, blockIdx.x / c.heads, head);
    for (Unit u; units.next(a, u);) {
        // this wave's rows
        const int row0 = u.row0 + 32 * wave;
        const int rows = min(u.row0 + u.rows - row0, 32);
        const bool mine = rows > 0;
        const int row = row0 + (mine ? min(n, rows - 1) : 0);
        const int i = mine ? row / a.each : 0;
        const long long token = (long long)u.start + i;
        const int qhead = head * a.each + (mine ? row - i * a.each : 0);
        const int key0 = u.step * 32, part_end = min(u.end, (u.step + u.steps) * 32);
        int lo = a.window ? u.back + i - a.window + 1 : 0, reach = min(u.back + i, part_end - 1) - lo;
        if (reach < 0) {   // none: no key is that far
            lo = 0x7fffffff;
            reach = 0;
        }
        const int pos0 = u.back + row0 / a.each, pos1 = mine ? u.back + (row0 + rows - 1) / a.each : 0;
        const int full_lo = a.window ? pos1 - a.window + 1 : 0, full_hi = min(pos0, part_end - 1);
        const int any_lo = a.window ? pos0 - a.window + 1 : 0, any_hi = mine ? min(pos1, part_end - 1) : -1;

        u32x4 q[KQ], qb[BK];
        int shift;   // the queries' power of two, over that of the products
        {
            const uint16_t* from = static_cast<const uint16_t*>(a.q) + token * a.q_ts + qhead * a.q_hs + 8 * hh;
            const bool vec = (((uintptr_t)a.q & 15) | ((a.q_ts | a.q_hs) & 7)) == 0;
            auto load = [&](int j) {
                u32x4 x;
                if (vec) {
                    x = *reinterpret_cast<const u32x4*>(from + 16 * j);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[e] = (uint32_t)from[16 * j + 2 * e] | ((uint32_t)from[16 * j + 2 * e + 1] << 16);
                }
                return x;
            };
            float most = 0.0f, sum[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                sum[g] = 0.0f;
#pragma unroll
                for (int j = g * (GS / 16); j < (g + 1) * (GS / 16); ++j) {
                    const u32x4 x = load(j);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y = half_lo<DT>(x[e]), z = half_hi<DT>(x[e]);
                        most = fmaxf(most, fmaxf(fabsf(y), fabsf(z)));
                        sum[g] += y + z;
                    }
                }
            }
            most = fmaxf(most, __shfl_xor(most, 32, 64));
            const int e = max(min(__builtin_amdgcn_frexp_expf(most), 127), -94);   // as in kv4_attn_impl.h
            shift = e - W::SCORE_UP;
            u32x4 sums[2 * BK] = {};   // a group's slots: the sum's pieces, and those of 8 times it
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float rest = ldexpf(sum[g] + __shfl_xor(sum[g], 32, 64), W::SUM_UP - e);
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const uint32_t piece = H::pack(rest, 0.0f) & 0xffffu;
                    rest -= half_lo<DT>(piece);
                    const int slot = W::SLOTS * g + i;
                    sums[slot / 8][slot % 8 / 2] |= piece << (16 * (slot % 2));
                    if constexpr (W::SCALED)
                        sums[slot / 8][2 + i / 2] |= (H::pack(8.0f * half_lo<DT>(piece), 0.0f) & 0xffffu)
                                                     << (16 * (i % 2));
                }
            }
#pragma unroll
            for (int y = 0; y < BK; ++y)
#pragma unroll
                for (int w = 0; w < 4; ++w) qb[y][w] = hh ? sums[2 * y + 1][w] : sums[2 * y][w];
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                u32x4 x = load(j);
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    x[w] = __builtin_bit_cast(uint32_t, half2_of(ldexpf(half_lo<DT>(x[w]), W::QUERY_UP - e),
                                                                 ldexpf(half_hi<DT>(x[w]), W::QUERY_UP - e)));
                if (j < KQ) q[j < KQ ? j : 0] = x;
                else s_q[wave][(j - KQ) * 64 + lane] = x;   // read by the same lane
            }
        }

        float top = kLeast, l = 0.0f;   // what a score may reach, and the sum of probabilities
        int power = TileInfo::ZEROS, common = power;   // the row's sums o are divided by 2^power; all rows', or NONE
        f32x16 o[DB];
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;

        const int* table = a.table + u.req * a.table_stride;
        const int blocks = min((part_end + 15) >> 4, a.columns << c.page_shift);
        const int tiles = (part_end - key0 + KEYS - 1) / KEYS;
        // Block table entries of 64 blocks, one a lane: read by the scalar unit, each
        // would hold up the next read of LDS.
        constexpr int BLOCKS = KEYS / 16, FETCH = 64 / BLOCKS;   // of a tile; tiles an entry read goes for
        int pages = -1;
        auto fetch = [&](int tile) {   // for the tile that is loaded next
            if (tile % FETCH == 0) {
                const int blk = ((key0 + KEYS * tile) >> 4) + lane;
                pages = blk < blocks ? table[blk >> c.page_shift] : -1;
            }
        };
        // Keys' powers that take the wave's rows' rf neither to 0 nor to infinity.
        const float rf = W::SCALED ? ldexpf(a.scale_log2, shift) : score_scale(a, shift);
        int lowest = TileInfo::ZEROS, highest = TileInfo::OWN - 1;
        if constexpr (W::SCALED) {
            const int e = shift + __builtin_amdgcn_frexp_expf(a.scale_log2);
            const int most = (int)wave_max((float)(4096 + e)) - 4096, least = 4096 - (int)wave_max((float)(4096 - e));
            if (least > -125 && most < 127) lowest = max(lowest, -125 - least), highest = min(highest, 127 - most);
            else lowest = TileInfo::OWN;
        }
        W raw;
        int exponent = TileInfo::ZEROS;   // of the last keys or values that the wave turned
        auto load = [&](int tile) {
            raw.load(c, pages, tile % FETCH * BLOCKS, head, key0 + KEYS * tile, my_blk, my_part, part_end, value);
        };
        f32x16 s[NT];   // scores of 32 keys, and those of the next 32
        auto unseen = [&](int tile) {   // no row of the wave sees a key of the tile
            const int key = key0 + KEYS * tile;
            return key > any_hi || key + KEYS - 1 < any_lo;
        };
        // Scores of 32 keys, the t-th of a tile.  slice(y) is what the vector ALU
        // does behind the y-th product.
        auto scores = [&](int buffer, int t, f32x16& to, auto&& slice) {
            const u32x4* sk = s_k[buffer] + t * (BK + KS) * 64 + lane;
            const f32x16 zero = {};
            u32x4 next[AHEAD];
            f32x16 part;
            f32x4 f[4];
#pragma unroll
            for (int y = 0; y < AHEAD; ++y) next[y] = sk[y * 64];
#pragma unroll
            for (int y = 0; y < BK + KS; ++y) {
                const int j = y - BK;
                if (!W::SCALED && j >= 0 && j % (GS / 16) == 0) {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        f[x] = *reinterpret_cast<const f32x4*>(
                            &s_factor[buffer][KEYS * (j / (GS / 16)) + 32 * t + 8 * x + 4 * hh]);
                }
                u32x4 mine_q = y < BK ? qb[y < BK ? y : 0] : q[j >= 0 && j < KQ ? j : 0];
                if (j >= KQ) mine_q = s_q[wave][(j - KQ) * 64 + lane];
                const u32x4 operand = next[y % AHEAD];
                if (y + AHEAD < BK + KS) next[y % AHEAD] = sk[(y + AHEAD) * 64];
                if (y < BK) to = mfma32_type<DT>(operand, mine_q, y == 0 ? zero : to);
                else if (W::SCALED) to = mfma32(operand, mine_q, to);
                else part = mfma32(operand, mine_q, j % (GS / 16) == 0 ? zero : part);
                slice(y);
                keep_order();
                if (!W::SCALED && j >= 0 && j % (GS / 16) == GS / 16 - 1) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) to[e] = fmaf(f[e / 4][e % 4], part[e], to[e]);
                }
            }
        };
        // The t-th 32 keys of the tile, whose scores are in x: probabilities, among
        // the products for the next 32's scores (`more`: there are such), then sums.
        TileInfo info;   // of the tile at hand, read one barrier ahead of its use
        auto sums = [&](int tile, int buffer, int t, f32x16& x, bool more, int next_buffer, int next_t, f32x16& y) {
            const int key = key0 + KEYS * tile + 32 * t;
            const u32x4* sv = s_v[buffer] + 2 * t * DB * 64 + lane;
            const int now = __builtin_amdgcn_readfirstlane(info.value_exponent);
            auto of_tile = [&](int e) { return 32 * t + 8 * (e / 4) + 4 * hh + e % 4; };   // the lane's e-th key
            bool all = key >= full_lo && key + 31 <= full_hi, there[2] = {true, true};
            float by[W::SCALED ? 2 : 1];   // what takes a block's scores to powers of two
            const int e0 = __builtin_amdgcn_readfirstlane(info.block[2 * t]);
            const int e1 = __builtin_amdgcn_readfirstlane(info.block[2 * t + 1]);
            by[0] = W::SCALED ? ldexpf(rf, e0) : rf;
            if constexpr (W::SCALED) by[1] = ldexpf(rf, e1);
            if (__builtin_expect(min(e0, e1) < lowest || max(e0, e1) > highest, 0)) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int e = b ? e1 : e0;
                    there[b] = e != TileInfo::MISSING;
                    all = all && there[b];
                    if constexpr (W::SCALED) {
                        by[b] = e == TileInfo::OWN ? 1.0f : score_scale(a, there[b] ? shift + e : 0);
                        if (e == TileInfo::OWN) {
#pragma unroll
                            for (int z = 8 * b; z < 8 * b + 8; ++z)
                                x[z] = ldexpf(x[z] * a.scale_log2, shift + s_key_power[buffer][of_tile(z)]);
                        }
                    }
                }
            }
            if (!all) {
                const int first = key + 4 * hh - lo;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const bool see = (uint32_t)(first + 8 * (e / 4) + e % 4) <= (uint32_t)reach;
                    x[e] = see && there[e / 8] ? x[e] : -INFINITY;
                }
            }
            float mx = -INFINITY;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float z = x[8 * b];
#pragma unroll
                for (int e = 1; e < 8; ++e) z = fmaxf(z, x[8 * b + e]);
                mx = fmaxf(mx, z * by[W::SCALED ? b : 0]);
            }
            float base = top - (kUp + kSlack);   // what scores lose before they are exponents
            if (now != common || __any(mx > top)) {
                const bool fresh = top == kLeast;
                float higher = fmaxf(mx, top - kSlack);
                higher = fmaxf(higher, __shfl_xor(higher, 32, 64));
                top = higher + kSlack;
                float fade = __builtin_amdgcn_exp2f(base - (top - (kUp + kSlack)));
                base = top - (kUp + kSlack);
                l *= fade;
                if (__builtin_expect(now != common, 0)) {
                    // The sums' power rises to the largest that the row sees.
                    auto power_of = [&](int e) {
                        const int own = s_value_power[buffer][of_tile(e)];
                        return now == TileInfo::OWN ? own : now;
                    };
                    int r = TileInfo::ZEROS, most = power;
#pragma unroll
                    for (int e = 0; e < 16; ++e) r = x[e] > -INFINITY ? max(r, power_of(e)) : r;
                    r = max(r, __shfl_xor(r, 32, 64));
                    if (fresh) {
                        most = now != TileInfo::OWN && top == kLeast ? now : r;   // any: there is no sum yet
                    } else {
                        r = max(r, most);
                        fade = ldexpf(fade, max(most - r, -126));
                        most = r;
                    }
                    power = most;
                    common = __builtin_amdgcn_readfirstlane(most);
                    if (__any(most != common)) common = TileInfo::NONE;
                    if (now != common) {   // what is left of a power goes to the probability, but not to their sum
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float z = fmaf(x[e], by[W::SCALED ? e / 8 : 0], -base);
                            x[e] = z + (float)min(power_of(e) - most, 0);
                            l += __builtin_amdgcn_exp2f(z) - __builtin_amdgcn_exp2f(x[e]);
                        }
#pragma unroll
                        for (float& b : by) b = 1.0f;
                        base = 0.0f;
                    }
                }
#pragma unroll
                for (int d = 0; d < DB; ++d) o[d] *= fade;
            }
            u32x4 p[2], rest[2];   // float16 caches: what probabilities lose as float16
            auto pair = [&](int e) {   // two probabilities
                const float p0 = __builtin_amdgcn_exp2f(fmaf(x[2 * e], by[W::SCALED ? e / 4 : 0], -base));
                const float p1 = __builtin_amdgcn_exp2f(fmaf(x[2 * e + 1], by[W::SCALED ? e / 4 : 0], -base));
                l += p0 + p1;
                const f16x2 h = half2_of(p0, p1);
                p[e / 4][e % 4] = __builtin_bit_cast(uint32_t, h);
                if constexpr (DT == DT_F16)
                    rest[e / 4][e % 4] =
                        __builtin_bit_cast(uint32_t, half2_of(p0 - (float)h[0], p1 - (float)h[1]));
            };
            if (NT == 2 && more) {
                scores(next_buffer, next_t, y, [&](int z) {
#pragma unroll
                    for (int e = z * 8 / (BK + KS); e < (z + 1) * 8 / (BK + KS); ++e) pair(e);
                });
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) pair(e);
            }
            u32x4 next[AHEAD];
#pragma unroll
            for (int z = 0; z < AHEAD; ++z) next[z] = sv[z * 64];
#pragma unroll
            for (int z = 0; z < 2 * DB; ++z) {
                const u32x4 operand = next[z % AHEAD];
                if (z + AHEAD < 2 * DB) next[z % AHEAD] = sv[(z + AHEAD) * 64];
                o[z % DB] = mfma32(operand, p[z / DB], o[z % DB]);
                if constexpr (DT == DT_F16) o[z % DB] = mfma32(operand, rest[z / DB], o[z % DB]);
                keep_order();
            }
        };
        // Values that are not finite, to the rows that see them.
        auto mend = [&](int tile) {
            const int key = key0 + KEYS * tile;
            for (int t = 0; t < KEYS; ++t) {
                const int at = key + t;
                const int page = (at >> 4) < blocks ? table[at >> 4 >> c.page_shift] : -1;
                if (at >= part_end || page < 0 || page >= c.num_pages) continue;
                const size_t tok = (size_t)block_number(c, page, head, at >> 4) * 16 + (at & 15);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const uint32_t p = c.vs[tok * G + g];
                    const float x = half_lo<DT>(p), y = half_hi<DT>(p);
                    if ((x - x) + (y - y) == 0.0f) continue;
                    const float add = (uint32_t)(at - lo) <= (uint32_t)reach ? fmaf(0.0f, x, y) : 0.0f;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if ((32 * d + 8 * (e / 4)) / GS == g) o[d][e] += add;
                }
            }
        };

        if (threadIdx.x < 3) s_info[threadIdx.x].bad = 0;
        if (tiles > 0) {
            fetch(0);
            load(0);
        }
        __syncthreads();
        // Tile t + 1 to LDS, the next one's codes to registers.
        auto turn = [&](int t, int after) {
            if (t + 1 < tiles) {
                if (value) {
                    bool good;
                    const int e = raw.values(s_v[after], exponent, s_value_power[after], my_blk, my_part, good);
                    if (wave == 4) {
                        if (!good) s_info[after].bad = t + 2;
                        s_info[after].value_exponent = e;
                    }
                } else {
                    const int e = raw.keys(s_k[(t + 1) & 1], s_factor[(t + 1) & 1], exponent, s_key_power[after],
                                           my_blk, my_part);
                    if (my_part == 0) s_info[after].block[my_blk] = raw.there ? e : TileInfo::MISSING;
                }
            }
            fetch(t + 2);
            load(t + 2);
        };
        int buffer = 2;   // of tile t's values
        for (int t = tiles > 0 ? -1 : 0; t < tiles; ++t) {   // no key, no read: there may be no page at all
            const int after = buffer == 2 ? 0 : buffer + 1;
            const bool more = t + 1 < tiles, here = t >= 0 && !unseen(t);
            turn(t, after);
            if constexpr (NT == 2) {
                if (here) sums(t, buffer, 0, s[0], true, t & 1, 1, s[1]);
                __syncthreads();   // tile t + 1 is in LDS
                if (here) sums(t, buffer, 1, s[1], more, (t + 1) & 1, 0, s[0]);
            } else {
                __syncthreads();
                if (here) sums(t, buffer, 0, s[0], false, 0, 0, s[0]);
            }
            if (here && __builtin_amdgcn_readfirstlane(info.bad) == t + 1) mend(t);
            info = s_info[after];
            if (more && !unseen(t + 1) && (NT == 1 || !here)) scores((t + 1) & 1, 0, s[0], [](int) {});
            buffer = after;
        }

        l += __shfl_xor(l, 32, 64);
        if (mine && n < rows) {
            const bool seen = top > kLeast || l != l;
            const float m = top - (kUp + kSlack);
            const int most = power;
            const long long at = token * a.heads + qhead;
            const long long place = ((long long)u.place * c.heads + head) * PROMPT_ROWS + 32 * wave + n;
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;   // parts too: their sums may pass float32's range
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    f32x4 v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = ldexpf(o[d][4 * x + e] * inv, most);
                    const int dim = 32 * d + 8 * x + 4 * hh;
                    if (u.place >= 0)
                        *reinterpret_cast<f32x4*>(a.part + place * D + dim) = v;
                    else
                        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at * D + dim) =
                            u32x2{H::pack(v[0], v[1]), H::pack(v[2], v[3])};
                }
            if (hh == 0) {
                if (u.place >= 0)
                    *reinterpret_cast<f32x2*>(a.stat + 2 * place) = f32x2{seen ? m : -INFINITY, l};
                else if (a.lse)
                    a.lse[at] = l != 0.0f ? (m + __builtin_amdgcn_logf(l)) * LN2 : -INFINITY;
            }
        }
        __syncthreads();
    }
}

}  // namespace kv4
}  // namespace qmx
