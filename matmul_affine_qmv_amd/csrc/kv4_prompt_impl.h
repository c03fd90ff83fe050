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
// Keys and queries enter as float16 for either type of cache, each token's keys
// and each row's queries brought to at most 1 by a power of two that goes back
// in at the exponent: 11 bits of a number, or 2^-25 of the largest.  A key's
// code c, as the bits of the float16 number c 2^-18, takes one multiply-add to
// become c s + b.  Values and probabilities have the cache's type (half a step
// of it each), as the matrix cores need; all sums are float32.
//
// 0 * NaN is NaN in a product, so values that are not finite are entered as 0
// and added afterwards to the rows that see them (a tile that holds one is rare
// and says so).
#pragma once

#include "kv4_attn_impl.h"

namespace qmx {
namespace kv4 {

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int DT>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    if constexpr (DT == DT_F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
}

__device__ __forceinline__ f16x2 half2_of(float lo, float hi) {
    const f32x2 v = {lo, hi};
    return __builtin_convertvector(v, f16x2);
}

constexpr int PROMPT_WAVES = 8, PROMPT_ROWS = 256, PROMPT_KEYS = 64;

// The codes and pairs of one block of 16 tokens, as a lane takes them to turn
// them into numbers.  Keys: the lane's token n = lane % 16 with all its pairs;
// values: the tokens 4h .. 4h + 3, h = lane / 16.
template <int D, int GS, int DT>
struct Raw {
    static constexpr int NJ = D / 32, G = D / GS, KS = D / 16, DB = D / 32;
    uint32_t w[NJ], sb[4 * G];
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
            load_words(sb, c.vs + at * (16 * G) + (lane >> 4) * (4 * G));
        } else {
            const uint32_t* from = c.ks + at * (16 * G) + (lane & 15) * G;
#pragma unroll
            for (int g = 0; g < G; ++g) sb[g] = from[g];
        }
    }

    // Keys to `k` [2 blocks of 32][KS][2][32] of 16 bytes, the power of two
    // that was taken out to `factor`; `blk` counts in the tile.
    __device__ __forceinline__ void keys(u32x4* k, float* factor, int blk) const {
        const int lane = threadIdx.x & 63, n = lane & 15, h = lane >> 4;
        u32x4* to = k + (((blk >> 1) * KS + (h >> 1)) * 2 + (h & 1)) * 32 + (blk & 1) * 16 + n;
        const bool live = there && n < tokens;
        float most = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float s = half_lo<DT>(sb[g]), b = half_hi<DT>(sb[g]);
            most = fmaxf(most, fmaxf(fabsf(b), fabsf(fmaf(15.0f, s, b))));
        }
        const int e = live ? min(__builtin_amdgcn_frexp_expf(most), 127) : 0;
        if (h == 0) factor[16 * blk + n] = ldexpf(1.0f, e);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint32_t p = sb[j * 32 / GS];
            const float s = live ? ldexpf(half_lo<DT>(p), 18 - e) : 0.0f, b = live ? ldexpf(half_hi<DT>(p), -e) : 0.0f;
            const f16x2 s2 = half2_of(s, s), b2 = half2_of(b, b);
            const uint32_t c[4] = {w[j] << 6, w[j] << 2, w[j] >> 2, w[j] >> 6};
            u32x4 x;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(
                                                        __builtin_bit_cast(f16x2, c[i] & 0x03c003c0u), s2, b2));
            to[j * 128] = x;   // two k-steps on
        }
    }

    // Values to `v` [4 blocks of 16][DB][2][32] of 16 bytes.  Whether all are
    // finite.
    __device__ __forceinline__ bool values(u32x4* v, int blk) const {
        const int lane = threadIdx.x & 63, n = lane & 15, h = lane >> 4;
        u32x2* to = reinterpret_cast<u32x2*>(v + (blk * DB * 2 + (h & 1)) * 32 + n) + (h >> 1);
        float s[4][G], b[4][G];
        bool good = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const bool live = there && 4 * h + i < tokens;
                float x = half_lo<DT>(sb[i * G + g]), y = half_hi<DT>(sb[i * G + g]);
                const bool finite = (x - x) + (y - y) == 0.0f;
                good = good && (finite || !live);
                x = live && finite ? x : 0.0f;
                y = live && finite ? y : 0.0f;
                if constexpr (DT == DT_F16) {   // a rounded scale may take the last code past the type's range
                    x = y + 15.0f * x > 65504.0f ? (65504.0f - y) * (1.0f / 15.0f) : x;
                    x = y + 15.0f * x < -65504.0f ? (-65504.0f - y) * (1.0f / 15.0f) : x;
                }
                s[i][g] = x;
                b[i][g] = y;
            }
        }
#pragma unroll
        for (int a = 0; a < D / 64; ++a) {
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int g = (64 * a + 16 * f) / GS;
                u32x2 x;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint32_t m = (w[2 * a + p] >> (4 * (f & 1))) & 0x0f0f0f0fu;
                    const float lo = (float)((m >> (8 * (f >> 1))) & 0xffu);
                    const float hi = (float)((m >> (16 + 8 * (f >> 1))) & 0xffu);
                    x[p] = Half<DT>::pack(fmaf(lo, s[2 * p][g], b[2 * p][g]),
                                          fmaf(hi, s[2 * p + 1][g], b[2 * p + 1][g]));
                }
                to[2 * ((2 * a + (f >> 1)) * 64 + (f & 1) * 16)] = x;
            }
        }
        return good;
    }
};

template <int D, int GS, int DT>
__global__ __launch_bounds__(64 * PROMPT_WAVES, 2) void kv4_prompt_kernel(Kv4AttnArgs a) {
    constexpr int KS = D / 16, DB = D / 32, G = D / GS, NT = D == 256 ? 1 : 2;
    constexpr float kSlack = 8.0f;
    using H = Half<DT>;
    __shared__ u32x4 s_k[2][2 * KS * 64], s_v[2][4 * DB * 64];
    __shared__ float s_factor[2][PROMPT_KEYS];
    __shared__ int s_bad[2], s_there[2][4];
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

        u32x4 q[KS];
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
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    q[j][w] = __builtin_bit_cast(uint32_t, half2_of(ldexpf(half_lo<DT>(q[j][w]), -e),
                                                                    ldexpf(half_hi<DT>(q[j][w]), -e)));
        }

        float m = 0.0f, top = -INFINITY, l = 0.0f;
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
        Raw<D, GS, DT> raw;
        auto load = [&](int page, int tile) {
            raw.load(c, page, head, (key0 >> 4) + 4 * tile + my_blk, part_end, value);
        };
        auto turn = [&](int tile) {   // this wave's block of the tile into LDS
            if (value) {
                if (!raw.values(s_v[tile & 1], my_blk)) s_bad[tile & 1] = tile + 1;
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
                const u32x4* sk = s_k[tile & 1] + t0 * KS * 64 + lane;
                const u32x4* sv = s_v[tile & 1] + 2 * t0 * DB * 64 + lane;
                f32x16 s[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[t][e] = 0.0f;
#pragma unroll
                    for (int j = 0; j < KS; ++j) s[t] = mfma32<DT_F16>(sk[(t * KS + j) * 64], q[j], s[t]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const f32x4 f =
                            *reinterpret_cast<const f32x4*>(&s_factor[tile & 1][32 * (t0 + t) + 8 * x + 4 * hh]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[t][4 * x + e] *= f[e];
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
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        s[t][e] = __builtin_amdgcn_exp2f(fmaf(s[t][e], rf, -m));
                        l += s[t][e];
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        u32x4 p;
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[e] = H::pack(s[t][8 * x + 2 * e], s[t][8 * x + 2 * e + 1]);
#pragma unroll
                        for (int d = 0; d < DB; ++d) o[d] = mfma32<DT>(sv[((2 * t + x) * DB + d) * 64], p, o[d]);
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
                    const f32x4 v = f32x4{o[d][4 * x], o[d][4 * x + 1], o[d][4 * x + 2], o[d][4 * x + 3]} * inv;
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
