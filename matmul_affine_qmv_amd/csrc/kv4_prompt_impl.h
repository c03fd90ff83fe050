// kv4_prompt_impl.h -- attention over the 4-bit cache for many rows a key head
// (prompts, and chunks of them): bound by the matrix cores and the vector
// ALU beside them, where kv4_attn_impl.h is bound by what it reads.
//
// A work-group of 8 waves takes 256 rows, a wave 32 of them, and walks the keys
// 64 at a time.  Four waves turn the keys' codes into numbers and four the
// values', once for all 256 rows, into LDS (two buffers, one barrier a tile) in
// the order in which the products read them: 16 bytes a lane, lane after lane.
// The first four do so before their own products of a tile and the others
// after, so that of the two waves on a SIMD one has the vector ALU's work when
// the other has the matrix cores'.
//
//   S^T[key, row] = K Q^T,  O^T[dim, row] += V^T P:  v_mfma_32x32x16, where the
//   probabilities that a lane computes are the operand it needs (as in
//   kv4_attn_impl.h), the values' tokens being put into that order.
//
// A code c enters both products as the bits of the float16 number c 2^-18, which
// is exact.  Keys stay codes: a group's product is multiplied by the token's
// scale in 32 bits, and the biases times the queries' sums (each in three
// pieces of the type, which hold 24 bits) are one more step of the product; so
// scores are as exact as their 32-bit sums.  Queries are float16, brought to at
// most 1 by a power of two a row (what is under 2^-14 of the largest keeps
// 2^-25 of it).  A value becomes c s + b in one multiply-add, a block of 16
// tokens brought to at most 1 by a power of two that goes into the
// probabilities' exponent, relative to the largest met so far; values and
// probabilities are rounded to float16, half a step 2^-11, as the matrix cores
// need (bfloat16 would cost eight times that).  All sums are float32.
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

__device__ __forceinline__ f16x2 half2_of(float lo, float hi) {
    const f32x2 v = {lo, hi};
    return __builtin_convertvector(v, f16x2);
}

// Codes at bits 4f of both halves, as float16 c 2^-18.
__device__ __forceinline__ uint32_t tiny_codes(uint32_t w, int f) {
    return (f < 2 ? w << (6 - 4 * f) : w >> (4 * f - 6)) & 0x03c003c0u;
}

constexpr int PROMPT_WAVES = 8, PROMPT_ROWS = 256, PROMPT_KEYS = 64;

// The codes and pairs of one block of 16 tokens, as a lane takes them to turn
// them into operands.  Keys: the lane's token n = lane % 16 with all its pairs;
// values: the tokens 4h .. 4h + 3, h = lane / 16, their pairs spread over the
// row's 16 lanes as in kv4_attn_impl.h.
template <int D, int GS, int DT>
struct Raw {
    static constexpr int NJ = D / 32, G = D / GS, KS = D / 16, DB = D / 32;
    static constexpr int BK = (3 * G + 15) / 16;          // steps of the product of biases
    static constexpr int SHARE = (4 * G + 15) / 16;       // registers of a lane's share of the values' pairs
    static constexpr int EMPTY = -120;                    // exponent of a block of zeros
    uint32_t w[NJ], sb[G > SHARE ? G : SHARE];
    bool there;
    int tokens;   // of the block, from its first on, that are there

    __device__ __forceinline__ void load(const Kv4View& c, int page, int head, int blk, int end, bool value) {
        const int lane = threadIdx.x & 63;
        tokens = end - 16 * blk;
        there = tokens > 0 && page >= 0 && page < c.num_pages;
        if (!there) return;
        const size_t at = (((size_t)page * c.heads + head) << c.page_shift) + (blk & ((1 << c.page_shift) - 1));
        load_words(w, (value ? c.vc : c.kc) + at * (64 * NJ) + lane * NJ);
        if (value) {
            const uint32_t* from = c.vs + at * (16 * G) + (lane >> 4) * (4 * G);
#pragma unroll
            for (int r = 0; r < SHARE; ++r) sb[r] = from[(16 * r + (lane & 15)) & (4 * G - 1)];
        } else {
            const uint32_t* from = c.ks + at * (16 * G) + (lane & 15) * G;
#pragma unroll
            for (int g = 0; g < G; ++g) sb[g] = from[g];
        }
    }

    // Keys to `k` [2 blocks of 32][KS + BK][2][32] of 16 bytes, the scales times
    // 2^18 to `factor` [G][64]; `blk` counts in the tile.
    __device__ __forceinline__ void keys(u32x4* k, float* factor, int blk) const {
        const int lane = threadIdx.x & 63, n = lane & 15, h = lane >> 4;
        u32x4* to = k + (blk >> 1) * (KS + BK) * 64 + (blk & 1) * 16 + n;
        const bool live = there && n < tokens;
        if (h == 0) {
#pragma unroll
            for (int g = 0; g < G; ++g) factor[64 * g + 16 * blk + n] = live ? half_lo<DT>(sb[g]) * 0x1p18f : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            u32x4 x;
#pragma unroll
            for (int f = 0; f < 4; ++f) x[f] = tiny_codes(w[j], f);
            to[(2 * j + (h >> 1)) * 64 + (h & 1) * 32] = x;
        }
#pragma unroll
        for (int y = 0; y < 2 * BK; ++y) {
            if (h == y) {   // eight slots: slot 3g + i takes group g's bias
                u32x4 x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int g0 = (8 * y + 2 * i) / 3, g1 = (8 * y + 2 * i + 1) / 3;
                    const uint32_t b0 = g0 < G && live ? sb[g0 < G ? g0 : 0] >> 16 : 0u;
                    const uint32_t b1 = g1 < G && live ? sb[g1 < G ? g1 : 0] & 0xffff0000u : 0u;
                    x[i] = b0 | b1;
                }
                to[(KS + (y >> 1)) * 64 + (y & 1) * 32] = x;
            }
        }
    }

    // Values to `v` [4 blocks of 16][DB][2][32] of 16 bytes, all of the block's
    // divided by 2^exponent.  Whether they are finite.
    __device__ __forceinline__ bool values(u32x4* v, int& exponent, int blk) const {
        const int lane = threadIdx.x & 63, n = lane & 15, h = lane >> 4;
        u32x2* to = reinterpret_cast<u32x2*>(v + (blk * DB * 2 + (h & 1)) * 32 + n) + (h >> 1);
        float s[SHARE], b[SHARE], most = 0.0f;
        bool good = true;
#pragma unroll
        for (int r = 0; r < SHARE; ++r) {
            const bool live = there && 4 * h + ((16 * r + n) & (4 * G - 1)) / G < tokens;
            const float x = half_lo<DT>(sb[r]), y = half_hi<DT>(sb[r]);
            const bool finite = (x - x) + (y - y) == 0.0f;
            good = good && (finite || !live);
            s[r] = live && finite ? x : 0.0f;
            b[r] = live && finite ? y : 0.0f;
            most = fmaxf(most, fmaxf(fabsf(b[r]), fabsf(fmaf(15.0f, s[r], b[r]))));
        }
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
        const int e = most > 0.0f ? __builtin_amdgcn_frexp_expf(fminf(most, 0x1.fffffep127f)) : EMPTY;
        exponent = e;
        uint32_t pair[SHARE];   // scale 2^18 and bias, float16
#pragma unroll
        for (int r = 0; r < SHARE; ++r)
            pair[r] = __builtin_bit_cast(uint32_t, half2_of(ldexpf(s[r], 18 - e), ldexpf(b[r], -e)));
#pragma unroll
        for (int g = 0; g < G; ++g) {
            f16x2 s2[2], b2[2];   // of two tokens
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint32_t x[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int at = (2 * p + i) * G + g;
                    x[i] = (uint32_t)__float_as_int(row_lane(__int_as_float((int)pair[at / 16]), at % 16));
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
        return good;
    }
};

template <int D, int GS, int DT>
__global__ __launch_bounds__(64 * PROMPT_WAVES, 2) void kv4_prompt_kernel(Kv4AttnArgs a) {
    using W = Raw<D, GS, DT>;
    constexpr int KS = D / 16, DB = D / 32, G = D / GS, BK = W::BK, NT = D == 256 ? 1 : 2;
    constexpr float kSlack = 8.0f;
    using H = Half<DT>;
    __shared__ u32x4 s_k[2][2 * (KS + BK) * 64], s_v[2][4 * DB * 64];
    __shared__ float s_factor[2][G * PROMPT_KEYS];
    __shared__ int s_bad[2], s_there[2][4], s_exponent[2][4];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, n = lane & 31, hh = lane >> 5;
    const Kv4View& c = a.c;
    const int head = blockIdx.x % c.heads;
    const bool value = wave >= 4;   // which codes this wave turns into numbers
    const int my_blk = wave & 3;

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
        const int lo = a.window ? u.back + i - a.window + 1 : 0, hi = min(u.back + i, part_end - 1);
        const int pos0 = u.back + row0 / a.each, pos1 = mine ? u.back + (row0 + rows - 1) / a.each : 0;
        const int full_lo = a.window ? pos1 - a.window + 1 : 0, full_hi = min(pos0, part_end - 1);
        const int any_lo = a.window ? pos0 - a.window + 1 : 0, any_hi = mine ? min(pos1, part_end - 1) : -1;

        u32x4 q[KS], qb[BK];
        float rf;
        {
            const uint16_t* from = static_cast<const uint16_t*>(a.q) + token * a.q_ts + qhead * a.q_hs + 8 * hh;
            const bool vec = (((uintptr_t)a.q & 15) | ((a.q_ts | a.q_hs) & 7)) == 0;
            float most = 0.0f;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                if (vec) {
                    q[j] = *reinterpret_cast<const u32x4*>(from + 16 * j);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        q[j][e] = (uint32_t)from[16 * j + 2 * e] | ((uint32_t)from[16 * j + 2 * e + 1] << 16);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    most = fmaxf(most, fmaxf(fabsf(half_lo<DT>(q[j][e])), fabsf(half_hi<DT>(q[j][e]))));
            }
            most = fmaxf(most, __shfl_xor(most, 32, 64));
            const int e = min(__builtin_amdgcn_frexp_expf(most), 127);
            rf = ldexpf(a.scale_log2, e);
            u32x4 sums[4] = {};   // slot 3g + i: piece i of group g's sum
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float sum = 0.0f;
#pragma unroll
                for (int j = g * (GS / 16); j < (g + 1) * (GS / 16); ++j)
#pragma unroll
                    for (int w = 0; w < 4; ++w) sum += half_lo<DT>(q[j][w]) + half_hi<DT>(q[j][w]);
                sum = ldexpf(sum + __shfl_xor(sum, 32, 64), -e);
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const int slot = 3 * g + i;
                    const uint32_t piece = H::pack(sum, 0.0f) & 0xffffu;
                    sum -= half_lo<DT>(piece);
                    sums[slot / 8][slot % 8 / 2] |= piece << (16 * (slot % 2));
                }
            }
#pragma unroll
            for (int y = 0; y < BK; ++y)
#pragma unroll
                for (int w = 0; w < 4; ++w) qb[y][w] = hh ? sums[2 * y + 1][w] : sums[2 * y][w];
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    q[j][w] = __builtin_bit_cast(uint32_t, half2_of(ldexpf(half_lo<DT>(q[j][w]), -e),
                                                                    ldexpf(half_hi<DT>(q[j][w]), -e)));
        }

        float m = 0.0f, top = -INFINITY, l = 0.0f;
        int most = 2 * W::EMPTY;   // the sums o are divided by 2^most
        f32x16 o[DB];
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;

        const int* table = a.table + u.req * a.table_stride;
        const int blocks = min((part_end + 15) >> 4, a.columns << c.page_shift);
        const int tiles = (part_end - key0 + PROMPT_KEYS - 1) / PROMPT_KEYS;
        auto page_of = [&](int tile) {
            const int blk = (key0 >> 4) + 4 * tile + my_blk;
            return blk < blocks ? table[blk >> c.page_shift] : -1;
        };
        W raw;
        auto load = [&](int page, int tile) {
            raw.load(c, page, head, (key0 >> 4) + 4 * tile + my_blk, part_end, value);
        };
        auto turn = [&](int tile) {   // this wave's block of the tile into LDS
            if (value) {
                int e;
                if (!raw.values(s_v[tile & 1], e, my_blk)) s_bad[tile & 1] = tile + 1;
                s_exponent[tile & 1][my_blk] = e;
            } else {
                raw.keys(s_k[tile & 1], s_factor[tile & 1], my_blk);
                s_there[tile & 1][my_blk] = raw.there ? 1 : 0;
            }
        };
        auto work = [&](int tile) {
            const int tile_key = key0 + PROMPT_KEYS * tile;
            if (tile_key > any_hi || tile_key + PROMPT_KEYS - 1 < any_lo) return;
            // NT blocks of 32 keys at a time (one where the sums leave no registers for two)
#pragma unroll 1
            for (int t0 = 0; t0 < 2; t0 += NT) {
                const int key = tile_key + 32 * t0;
                const u32x4* sk = s_k[tile & 1] + t0 * (KS + BK) * 64 + lane;
                const u32x4* sv = s_v[tile & 1] + 2 * t0 * DB * 64 + lane;
                f32x16 s[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[t][e] = 0.0f;
#pragma unroll
                    for (int y = 0; y < BK; ++y)
                        s[t] = mfma32_type<DT>(sk[(t * (KS + BK) + KS + y) * 64], qb[y], s[t]);
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        f32x16 part;
#pragma unroll
                        for (int e = 0; e < 16; ++e) part[e] = 0.0f;
#pragma unroll
                        for (int j = g * (GS / 16); j < (g + 1) * (GS / 16); ++j)
                            part = mfma32(sk[(t * (KS + BK) + j) * 64], q[j], part);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const f32x4 f = *reinterpret_cast<const f32x4*>(
                                &s_factor[tile & 1][64 * g + 32 * (t0 + t) + 8 * x + 4 * hh]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[t][4 * x + e] = fmaf(f[e], part[4 * x + e], s[t][4 * x + e]);
                        }
                    }
                }
                bool all = key >= full_lo && key + 32 * NT - 1 <= full_hi;
                uint32_t there = 0;   // a bit for each block of 16 keys
#pragma unroll
                for (int x = 0; x < 2 * NT; ++x)
                    there |= (uint32_t)__builtin_amdgcn_readfirstlane(s_there[tile & 1][2 * t0 + x]) << x;
                if (!all || there != (1u << (2 * NT)) - 1) {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int at = key + 32 * t + 8 * (e / 4) + 4 * hh + e % 4;
                            const bool see = at >= lo && at <= hi && ((there >> (2 * t + e / 8)) & 1u);
                            s[t][e] = see ? s[t][e] : -INFINITY;
                        }
                }
                float mx = s[0][0];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[t][e]);
                mx *= rf;
                if (__any(mx > top)) {
                    float now = fmaxf(mx, top - kSlack);
                    now = fmaxf(now, __shfl_xor(now, 32, 64));
                    const float safe = now > -INFINITY ? now : 0.0f;
                    const float fade = top > -INFINITY ? __builtin_amdgcn_exp2f(m - safe) : 0.0f;
                    top = now + kSlack;
                    m = safe;
                    l *= fade;
#pragma unroll
                    for (int d = 0; d < DB; ++d) o[d] *= fade;
                }
                int exponent[2 * NT], now = most;
#pragma unroll
                for (int x = 0; x < 2 * NT; ++x) {
                    exponent[x] = __builtin_amdgcn_readfirstlane(s_exponent[tile & 1][2 * t0 + x]);
                    now = max(now, exponent[x]);
                }
                if (now > most) {
#pragma unroll
                    for (int d = 0; d < DB; ++d) o[d] *= ldexpf(1.0f, most - now);
                    most = now;
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        // what is 2^-60 of the largest need not be told from 0
                        const int less = max(exponent[2 * t + x] - most, -60);
                        const float off = (float)less - m;
                        float sum = 0.0f;
#pragma unroll
                        for (int e = 8 * x; e < 8 * x + 8; ++e) {
                            s[t][e] = __builtin_amdgcn_exp2f(fmaf(s[t][e], rf, off));
                            sum += s[t][e];
                        }
                        l = fmaf(sum, ldexpf(1.0f, -less), l);
                        u32x4 p;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            p[e] = __builtin_bit_cast(uint32_t, half2_of(s[t][8 * x + 2 * e], s[t][8 * x + 2 * e + 1]));
#pragma unroll
                        for (int d = 0; d < DB; ++d) o[d] = mfma32(sv[((2 * t + x) * DB + d) * 64], p, o[d]);
                    }
                }
            }
            if (s_bad[tile & 1] == tile + 1) {   // values that are not finite, to the rows that see them
                for (int t = 0; t < PROMPT_KEYS; ++t) {
                    const int at = tile_key + t;
                    const int page = (at >> 4) < blocks ? table[at >> 4 >> c.page_shift] : -1;
                    if (at >= part_end || page < 0 || page >= c.num_pages) continue;
                    const size_t tok = (((size_t)page * c.heads + head) << (c.page_shift + 4)) +
                                       (at & ((16 << c.page_shift) - 1));
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        const uint32_t p = c.vs[tok * G + g];
                        const float x = half_lo<DT>(p), y = half_hi<DT>(p);
                        if ((x - x) + (y - y) == 0.0f) continue;
                        const float add = at >= lo && at <= hi ? fmaf(0.0f, x, y) : 0.0f;
#pragma unroll
                        for (int d = 0; d < DB; ++d)
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if ((32 * d + 8 * (e / 4)) / GS == g) o[d][e] += add;
                    }
                }
            }
        };

        if (threadIdx.x < 2) s_bad[threadIdx.x] = 0;
        __syncthreads();
        if (tiles > 0) {
            load(page_of(0), 0);
            int page = page_of(1);
            turn(0);
            load(page, 1);
            page = page_of(2);
            __syncthreads();
            for (int t = 0; t < tiles; ++t) {
                if (value) work(t);
                if (t + 1 < tiles) {
                    turn(t + 1);
                    load(page, t + 2);
                    page = page_of(t + 3);
                }
                if (!value) work(t);
                __syncthreads();
            }
        }

        l += __shfl_xor(l, 32, 64);
        if (mine && n < rows) {
            const bool seen = top > -INFINITY || l != l;
            const long long at = token * a.heads + qhead;
            const long long place = ((long long)u.place * c.heads + head) * PROMPT_ROWS + 32 * wave + n;
            const float inv = u.place >= 0 ? 1.0f : l != 0.0f ? 1.0f / l : 0.0f;
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
