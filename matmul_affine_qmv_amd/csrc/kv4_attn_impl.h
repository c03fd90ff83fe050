// kv4_attn_impl.h -- attention over the paged 4-bit key/value cache.
//
// A row is one (query, head); the heads that share a key head are neighbouring
// rows.  A wave takes 16 of them and walks its keys 32 at a time:
//
//   S^T[token, row] = K Q^T   v_mfma_16x16x32: K's codes are the A operand as
//                             they come from memory, 16 bytes a lane at a head
//                             size of 128 (the cache's layout is this operand);
//   softmax                   in registers: a lane holds four tokens of one row;
//   O^T[dim, row] += V^T P    the lane's eight probabilities of 32 tokens are the
//                             B operand as they stand, V's codes the A operand.
//
// So neither codes nor probabilities pass through LDS.  With c the codes, s and
// b the scales and biases, g the groups of the head dimension:
//
//   S = sum_g s_tg (sum_{d in g} q_d c_td) + b_tg (sum_{d in g} q_d)
//   O = sum_t (p_t s_tg) c_td + sum_t p_t b_tg
//
// K's codes enter the product as the bits of the float16 numbers c 2^-18, queries
// as float16 brought under 2^15 by a power of two a row (exact, but for what is
// under 2^-29 of the row's largest and keeps 2^-40 of it), so S is as exact as its
// 32-bit sums.  With K's codes as OFF + c the offset, up to 128 times the codes'
// share, cost the row sums 3 to 5 bits (error of the logarithm of the sum 4e-8
// now) and the same time.  V's codes enter as the bfloat16 numbers OFF + c, an
// exponent set above the four bits, and the offset is taken off in 32 bits through
// the sum of the p_t s_tg as they enter, in the same step as sum_t p_t b_tg; the
// bias is moved to the middle of the codes (b + 8 s), so the two sums do not
// cancel.  p_t s_tg enters in two bfloat16 pieces, to 2^-16 of itself and at any
// size: as float16, what lay under 2^-25 was lost, and with it the tail behind a
// key of a large score (13 % of the output over 1200 keys 9 under it, scales of
// 2^-13); as one bfloat16 piece it was off by 2^-8.  The second piece's products and 24 vector
// instructions a group cost 2 to 8 % (1 to 48 requests of a token or few over 641
// to 131000 keys, heads of 64 to 256; most where a group is 32).
//
// A work-group of WK waves takes a unit (kv4.h); the waves take every WK-th step
// and are joined in LDS.  The running maximum is raised only when a score passes
// it by more than kSlack (in powers of two); until then no lane needs another's
// scores.  A step's loads go out into the registers that the step before has just
// used, so a wave has a step under way in 60 registers fewer than with two sets.
//
// Measured: two tokens of 64 heads over up to 131000 cached ones (8 key heads of
// 128, groups of 128, float16) 38 us and 5 us for joining the parts, 143 MB at 3.3
// TB/s (a large copy: 4.9); bound by what is in flight, two waves a SIMD with 4.6 KB
// each.  48 tokens over up to 8000 (40 heads, bfloat16) 28 + 5.5 us for 64 MB: half
// of it is the wait for lengths, block table, queries and first codes, one after the
// other.  Cut by splits of one length for all requests, as the host alone could do
// it, they took 55 + 14 and 40 + 4 us.  Pairs read by every lane that needs them
// instead of shared by a row cost 72 registers and 20 % of the time.  Heads of 256
// spill 49 registers in groups of 64 and 240 in groups of 32, whose 48 tokens over up
// to 8000 take 72 and 239 us (groups of 128, none spilled: 43).
#pragma once

#include <type_traits>

#include "kv4.h"
#include "kv4_units.h"
#include "qmx_device.h"

namespace qmx {
namespace kv4 {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// What depends on the 16-bit type.
template <int DT>
struct Half;

template <>
struct Half<DT_BF16> {
    static constexpr float OFF = 128.0f;
    static constexpr uint32_t ONES = 0x3f803f80u;
    // Codes at bits 4f of both halves, as the numbers OFF + code.
    static __device__ __forceinline__ uint32_t codes(uint32_t w, int f) {
        return ((w >> (4 * f)) & 0x000f000fu) | 0x43004300u;
    }
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const f32x2 v = {lo, hi};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    }
    static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c,
                                               false);
    }
};

template <>
struct Half<DT_F16> {
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const f32x2 v = {lo, hi};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
    }
};

__device__ __forceinline__ f16x2 half2_of(float lo, float hi) {
    const f32x2 v = {lo, hi};
    return __builtin_convertvector(v, f16x2);
}

// Codes at bits 4f of both halves, as float16 c 2^-18.
__device__ __forceinline__ uint32_t tiny_codes(uint32_t w, int f) {
    return (f < 2 ? w << (6 - 4 * f) : w >> (4 * f - 6)) & 0x03c003c0u;
}

// Sum over the four lanes that hold one row.
__device__ __forceinline__ float row_sum(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}

// Lane k's value of each row of 16 lanes, for all of the row; k is a constant
// once loops are unrolled.  The move folds into the product that takes it.
__device__ __forceinline__ float row_lane(float v, int k) {
    const int x = __float_as_int(v);
#define QMX_ROW_LANE(K) \
    case K: return __int_as_float(__builtin_amdgcn_mov_dpp(x, 0x150 + K, 0xf, 0xf, true));
    switch (k) {
        QMX_ROW_LANE(0) QMX_ROW_LANE(1) QMX_ROW_LANE(2) QMX_ROW_LANE(3) QMX_ROW_LANE(4) QMX_ROW_LANE(5)
        QMX_ROW_LANE(6) QMX_ROW_LANE(7) QMX_ROW_LANE(8) QMX_ROW_LANE(9) QMX_ROW_LANE(10) QMX_ROW_LANE(11)
        QMX_ROW_LANE(12) QMX_ROW_LANE(13) QMX_ROW_LANE(14) QMX_ROW_LANE(15)
    }
#undef QMX_ROW_LANE
    return v;
}

// The softmax scale times 2^e, held to what is neither 0 nor infinite: a hidden
// score's -inf times 0 would be NaN.
__device__ __forceinline__ float score_scale(const Kv4AttnArgs& a, int e) {
    return fminf(fmaxf(ldexpf(a.scale_log2, e), 0x1p-126f), 0x1.fffffep127f);
}

// The (scale, bias) pairs of a block's tokens.  The 16 lanes of a row all need
// the 4 * G pairs of the row's four tokens, keys' and values': each lane holds
// its share, as numbers, and row_lane passes them round.  They are set right for
// the codes: keys' 8 s, values' b + 8 s.
template <int DT, int G>
struct Pairs {
    static constexpr int PAIRS = (8 * G + 15) / 16;
    float s[PAIRS], b[PAIRS];
    __device__ __forceinline__ void set(const uint32_t (&w)[PAIRS]) {
#pragma unroll
        for (int r = 0; r < PAIRS; ++r) {
            const bool value = (16 * r + (int)(threadIdx.x & 15)) & (4 * G);
            const float x = half_lo<DT>(w[r]);
            s[r] = value ? x : x * 8.0f;
            b[r] = fmaf(value ? 8.0f : 0.0f, x, half_hi<DT>(w[r]));
        }
    }
    __device__ __forceinline__ float scale(bool value, int i, int g) const {
        const int at = (value ? 4 * G : 0) + i * G + g;
        return row_lane(s[at / 16], at % 16);
    }
    __device__ __forceinline__ float bias(bool value, int i, int g) const {
        const int at = (value ? 4 * G : 0) + i * G + g;
        return row_lane(b[at / 16], at % 16);
    }
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&to)[N], const uint32_t* from) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const u32x4 w = reinterpret_cast<const u32x4*>(from)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) to[4 * i + j] = w[j];
        }
    } else {
        const u32x2 w = *reinterpret_cast<const u32x2*>(from);
        to[0] = w[0];
        to[1] = w[1];
    }
}

// One wave's 16 rows, its state, and the 32 tokens at hand.
template <int D, int GS, int DT>
struct Rows {
    static constexpr int NJ = D / 32, G = D / GS, NB = D / 16;
    using H = Half<DT>;
    static constexpr float kSlack = 8.0f;
    u32x4 q[NJ];       // float16, over the row's power of two, times 2^15
    float qsum[G];     // over the row's power of two
    float m, top, l;   // the maximum taken off (0 at first), what a score may reach, the sum
    float fix[G];      // sum p b + the offsets of V's codes, this lane's tokens
    f32x4 o[NB];
    int lo, hi;        // keys the row sees
    uint32_t k[2][NJ], v[2][NJ], sb[2][Pairs<DT, G>::PAIRS];
    float s[8];        // scores, then probabilities

    __device__ __forceinline__ void clear() {
        m = 0.0f;
        top = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) fix[g] = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b) o[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // `at`: the numbers of the two blocks.
    __device__ __forceinline__ void load_pairs(const Kv4View& c, const uint32_t (&at)[2]) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < Pairs<DT, G>::PAIRS; ++r) {
                const int w = 16 * r + (lane & 15);   // of the row's 8 * G pairs (fewer than 16: the rest repeat)
                const uint32_t* from = (w & (4 * G)) ? c.vs : c.ks;
                sb[i][r] = from[(uint64_t)at[i] * (16 * G) + (lane >> 4) * (4 * G) + (w & (4 * G - 1))];
            }
    }
    __device__ __forceinline__ void load_codes(uint32_t (&to)[2][NJ], const uint32_t* codes, const uint32_t (&at)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) load_words(to[i], codes + (uint64_t)at[i] * (64 * NJ) + (threadIdx.x & 63) * NJ);
    }

    __device__ __forceinline__ void scores(const Pairs<DT, G> (&pair)[2]) {
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = g * (GS / 32); j < (g + 1) * (GS / 32); ++j) {
                    const uint32_t w = k[blk][j];
                    const u32x4 a = {tiny_codes(w, 0), tiny_codes(w, 1), tiny_codes(w, 2), tiny_codes(w, 3)};
                    part = Half<DT_F16>::mfma(a, q[j], part);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float& to = s[4 * blk + i];
                    const float b = pair[blk].bias(false, i, g);
                    to = g == 0 ? b * qsum[g] : fmaf(b, qsum[g], to);
                    to = fmaf(pair[blk].scale(false, i, g), part[i], to);
                }
            }
        }
    }

    // The tokens from `key` on that the row sees, a bit each.
    __device__ __forceinline__ uint32_t hide(int key, bool there0, bool there1) {
        const int h = (threadIdx.x & 63) >> 4;
        uint32_t seen = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int t = key + 16 * (e / 4) + 4 * h + e % 4;
            const bool see = t >= lo && t <= hi && (e < 4 ? there0 : there1);
            seen |= (see ? 1u : 0u) << e;
            s[e] = see ? s[e] : -INFINITY;
        }
        return seen;
    }

    __device__ __forceinline__ void probabilities(float scale) {
        float mx = s[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) mx = fmaxf(mx, s[e]);
        mx *= scale;
        if (__any(mx > top)) {
            const float now = row_max(fmaxf(mx, top - kSlack));
            const float safe = now > -INFINITY ? now : 0.0f;
            const float fade = top > -INFINITY ? __builtin_amdgcn_exp2f(m - safe) : 0.0f;
            top = now + kSlack;
            m = safe;
            l *= fade;
#pragma unroll
            for (int g = 0; g < G; ++g) fix[g] *= fade;
#pragma unroll
            for (int b = 0; b < NB; ++b) o[b] *= fade;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], scale, -m));
            l += s[e];
        }
    }

    // all: every row sees every token; else `seen` says.  What is not seen has a
    // probability of 0, but its scale and bias may be infinite.
    __device__ __forceinline__ void values(const Pairs<DT, G> (&pair)[2], bool all, uint32_t seen) {
        using B = Half<DT_BF16>;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float w[8], y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                w[e] = s[e] * pair[e / 4].scale(true, e % 4, g);
                y[e] = pair[e / 4].bias(true, e % 4, g);
            }
            if (!all) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    w[e] = (seen >> e) & 1u ? w[e] : 0.0f;
                    y[e] = (seen >> e) & 1u ? y[e] : 0.0f;
                }
            }
            u32x4 ps[2];   // p s in two pieces
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) fix[g] = fmaf(s[e], y[e], fix[g]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t first = B::pack(w[2 * e], w[2 * e + 1]);
                ps[0][e] = first;
                ps[1][e] = B::pack(w[2 * e] - half_lo<DT_BF16>(first), w[2 * e + 1] - half_hi<DT_BF16>(first));
                sum = B::dot2(ps[0][e], B::ONES, sum);
                sum = B::dot2(ps[1][e], B::ONES, sum);
            }
            fix[g] = fmaf(-(B::OFF + 8.0f), sum, fix[g]);
            constexpr int MOST = GS < 64 ? 2 : 4;   // blocks of 16 elements at a time
#pragma unroll
            for (int n0 = g * (GS / 16); n0 < (g + 1) * (GS / 16); n0 += MOST) {
                u32x4 x[MOST];
#pragma unroll
                for (int i = 0; i < MOST; ++i) {
                    const int a = (n0 + i) / 4, f = (n0 + i) % 4;
                    x[i] = u32x4{B::codes(v[0][2 * a], f), B::codes(v[0][2 * a + 1], f), B::codes(v[1][2 * a], f),
                                 B::codes(v[1][2 * a + 1], f)};
                    o[n0 + i] = B::mfma(x[i], ps[0], o[n0 + i]);
                }
#pragma unroll
                for (int i = 0; i < MOST; ++i) o[n0 + i] = B::mfma(x[i], ps[1], o[n0 + i]);
            }
        }
    }

    // Adds the lanes' parts: after this o is the row's sum of p v, l of p.
    __device__ __forceinline__ void join() {
        l = row_sum(l);
#pragma unroll
        for (int g = 0; g < G; ++g) fix[g] = row_sum(fix[g]);
#pragma unroll
        for (int b = 0; b < NB; ++b) o[b] += fix[b * 16 / GS];
    }
};

// A request's row of the block table, read a step (two blocks) at a time.
struct Pages {
    const int* table;
    int blocks;   // those from here on are not there
    int page[2];
    __device__ __forceinline__ void read(const Kv4View& c, int step) {
#pragma unroll
        for (int i = 0; i < 2; ++i) page[i] = 2 * step + i < blocks ? table[(2 * step + i) >> c.page_shift] : -1;
    }
    __device__ __forceinline__ bool there(const Kv4View& c, int i) const {
        return page[i] >= 0 && page[i] < c.num_pages;
    }
    // The two blocks' numbers in the cache (page 0's where there is none: its
    // tokens are hidden).
    __device__ __forceinline__ void place(const Kv4View& c, int head, int step, uint32_t (&at)[2]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            at[i] = block_number(c, there(c, i) ? page[i] : 0, head, 2 * step + i);
    }
};

// WK waves on units of 16 rows.
template <int D, int GS, int DT, int WK>
__global__ __launch_bounds__(64 * WK, 2) void kv4_attn_kernel(Kv4AttnArgs a) {
    using R = Rows<D, GS, DT>;
    constexpr int NJ = R::NJ, G = R::G, NB = R::NB, PITCH = D + 4;
    __shared__ float s_o[WK][16 * PITCH];
    __shared__ float s_m[WK][16], s_l[WK][16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, n = lane & 15, h = lane >> 4;
    const Kv4View& c = a.c;
    const int head = blockIdx.x % c.heads;

    Units<64 * WK> units(a, blockIdx.x / c.heads, head);
    for (Unit u; units.next(a, u);) {
        const int last = u.rows - 1;
        const int row = min(n, last);
        const int i = (u.row0 + row) / a.each;
        const long long token = (long long)u.start + i;
        const int qhead = head * a.each + u.row0 + row - i * a.each;
        R x;
        x.clear();
        x.lo = a.window ? u.back + i - a.window + 1 : 0;
        x.hi = min(u.back + i, u.end - 1);
        const uint16_t* q = static_cast<const uint16_t*>(a.q) + token * a.q_ts + qhead * a.q_hs + 8 * h;
        const bool vec = (((uintptr_t)a.q & 15) | ((a.q_ts | a.q_hs) & 7)) == 0;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            if (vec) {
                x.q[j] = *reinterpret_cast<const u32x4*>(q + 32 * j);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x.q[j][e] = (uint32_t)q[32 * j + 2 * e] | ((uint32_t)q[32 * j + 2 * e + 1] << 16);
            }
        }
        float most = 0.0f;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                most = fmaxf(most, fmaxf(fabsf(half_lo<DT>(x.q[j][e])), fabsf(half_hi<DT>(x.q[j][e]))));
        // bfloat16 has no digits under 2^-133, which 2^(15 + 94) takes to float16's last
        const int exponent = max(min(__builtin_amdgcn_frexp_expf(row_max(most)), 127), -94);
        const float scale = score_scale(a, exponent);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float sum = 0.0f;
#pragma unroll
            for (int j = g * (GS / 32); j < (g + 1) * (GS / 32); ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w = x.q[j][e];
                    const float lo = ldexpf(half_lo<DT>(w), -exponent), hi = ldexpf(half_hi<DT>(w), -exponent);
                    sum += lo + hi;
                    x.q[j][e] = __builtin_bit_cast(uint32_t, half2_of(lo * 0x1p15f, hi * 0x1p15f));
                }
            }
            x.qsum[g] = row_sum(sum);
        }
        Pages pages{a.table + u.req * a.table_stride, min((u.end + 15) >> 4, a.columns << c.page_shift), {-1, -1}};
        const int steps = u.step + u.steps;
        int step = u.step + wave;
        if (step < steps) {
            // A step's loads go out as soon as the step before has used the same
            // registers, its block table entries another step ahead.
            uint32_t at[2];
            pages.read(c, step);
            pages.place(c, head, step, at);
            bool there0 = pages.there(c, 0), there1 = pages.there(c, 1);
            x.load_pairs(c, at);
            x.load_codes(x.k, c.kc, at);
            x.load_codes(x.v, c.vc, at);
            pages.read(c, step + WK);
            for (;;) {
                const int key = step * 32;
                const bool all = key >= u.full_lo && key + 31 <= u.full_hi && there0 && there1;
                step += WK;
                const bool more = step < steps;
                Pairs<DT, G> pair[2];
                pair[0].set(x.sb[0]);
                pair[1].set(x.sb[1]);
                const bool was0 = there0, was1 = there1;
                if (more) {
                    there0 = pages.there(c, 0);
                    there1 = pages.there(c, 1);
                    pages.place(c, head, step, at);
                    pages.read(c, step + WK);
                    x.load_pairs(c, at);
                }
                x.scores(pair);
                if (more) x.load_codes(x.k, c.kc, at);
                const uint32_t seen = all ? 0xffu : x.hide(key, was0, was1);
                x.probabilities(scale);
                x.values(pair, all, seen);
                if (!more) break;
                x.load_codes(x.v, c.vc, at);
            }
        }
        x.join();

        const bool seen = x.top > -INFINITY || x.l != x.l;
        if (h == 0) {
            s_m[wave][n] = seen ? x.m : -INFINITY;
            s_l[wave][n] = x.l;
        }
        __syncthreads();
        float m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int w = 0; w < WK; ++w) m = fmaxf(m, s_m[w][n]);
        const float safe = m > -INFINITY ? m : 0.0f;
#pragma unroll
        for (int w = 0; w < WK; ++w) l += s_l[w][n] * __builtin_amdgcn_exp2f(s_m[w][n] - safe);
        const float f = seen ? __builtin_amdgcn_exp2f(x.m - safe) : 0.0f;
        if (n <= last) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
                *reinterpret_cast<f32x4*>(&s_o[wave][n * PITCH + 16 * b + 4 * h]) = x.o[b] * f;
        }
        __syncthreads();
        if (n <= last) {
            const long long at = token * a.heads + qhead;
            const long long place = ((long long)u.place * c.heads + head) * 16 + n;
            const float inv = u.place >= 0 ? 1.0f : l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
            for (int b0 = 0; b0 < NB; b0 += WK) {
                const int b = b0 + wave;
                if (NB % WK != 0 && b >= NB) break;
                f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < WK; ++w) v += *reinterpret_cast<const f32x4*>(&s_o[w][n * PITCH + 16 * b + 4 * h]);
                v *= inv;
                if (u.place >= 0)
                    *reinterpret_cast<f32x4*>(a.part + place * D + 16 * b + 4 * h) = v;
                else
                    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at * D + 16 * b + 4 * h) =
                        u32x2{R::H::pack(v[0], v[1]), R::H::pack(v[2], v[3])};
            }
            if (lane == n && wave == 0) {
                if (u.place >= 0)
                    *reinterpret_cast<f32x2*>(a.stat + 2 * place) = f32x2{m, l};
                else if (a.lse)
                    a.lse[at] = l != 0.0f ? (safe + __builtin_amdgcn_logf(l)) * LN2 : -INFINITY;
            }
        }
        __syncthreads();
    }
}

}  // namespace kv4
}  // namespace qmx
