// kv4_attn_impl.h -- attention over the paged 4-bit key/value cache.
//
// A row is one (query, head); the heads that share a key head are neighbouring
// rows.  One wave takes RT tiles of 16 rows and walks its keys 32 at a time:
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
// Codes enter the products as OFF + c, an exponent set above the four bits, and
// the offsets are taken off in 32 bits: K's through b, V's through the sum of
// the rounded p_t s_tg, in the same step as sum_t p_t b_tg.  V's bias is moved to
// the middle of the codes (b + 8 s), so the two sums do not cancel.  K's codes
// are exact and S is as exact as its 32-bit sums; the one rounding to 16 bits is
// that of p_t s_tg (half a step: 2^-8 of it in bfloat16, 2^-11 in float16), which
// the matrix cores need.
//
// The running maximum is raised only when a score passes it by more than
// kSlack (in powers of two); until then no lane needs another's scores.
#pragma once

#include <type_traits>

#include "kv4.h"
#include "qmx_device.h"

namespace qmx {
namespace kv4 {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// What depends on the 16-bit type.
template <int DT>
struct Half;

template <>
struct Half<DT_BF16> {
    static constexpr float OFF = 128.0f;
    static constexpr float kSlack = 8.0f;
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
    static constexpr float OFF = 64.0f;
    // p s stays finite: scales are at most (2 * 65504) / 15, p at most 4.
    static constexpr float kSlack = 2.0f;
    static constexpr uint32_t ONES = 0x3c003c00u;
    static __device__ __forceinline__ uint32_t codes(uint32_t w, int f) {
        const uint32_t x = f == 0 ? w << 4 : w >> (4 * (f - 1));
        return (x & 0x00f000f0u) | 0x54005400u;
    }
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const f32x2 v = {lo, hi};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
    }
    static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), __builtin_bit_cast(f16x2, b), c, false);
    }
};

// Sum over the four lanes that hold one row.
__device__ __forceinline__ float row_sum(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}

// The codes and pairs of 32 tokens, as one lane holds them.
template <int NJ, int G>
struct Tokens {
    uint32_t k[2][NJ], v[2][NJ], ks[2][4 * G], vs[2][4 * G];
    bool there[2];   // the block's page is in the cache
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

// One wave's rows and its state.
template <int D, int GS, int DT, int RT>
struct Rows {
    static constexpr int NJ = D / 32, G = D / GS, NB = D / 16;
    using H = Half<DT>;
    u32x4 q[RT][NJ];
    float qsum[RT][G];
    float m[RT], top[RT], l[RT];   // the maximum taken off (0 at first), what a score may reach, the sum
    float fix[RT][G];              // sum p b + the offsets of V's codes, this lane's tokens
    f32x4 o[RT][NB];
    int lo[RT], hi[RT];            // keys the row sees

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            m[r] = 0.0f;
            top[r] = -INFINITY;
            l[r] = 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g) fix[r][g] = 0.0f;
#pragma unroll
            for (int b = 0; b < NB; ++b) o[r][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }

    // 32 tokens from `key` on.  MASK: some row does not see all of them.
    template <bool MASK>
    __device__ __forceinline__ void step(const Tokens<NJ, G>& x, int key, float scale) {
        const int h = (threadIdx.x & 63) >> 4;
        float s[RT][8];
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                f32x4 part[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) part[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = g * (GS / 32); j < (g + 1) * (GS / 32); ++j) {
                    const uint32_t w = x.k[blk][j];
                    const u32x4 a = {H::codes(w, 0), H::codes(w, 1), H::codes(w, 2), H::codes(w, 3)};
#pragma unroll
                    for (int r = 0; r < RT; ++r) part[r] = H::mfma(a, q[r][j], part[r]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t sb = x.ks[blk][i * G + g];
                    const float sc = half_lo<DT>(sb), b = fmaf(-H::OFF, sc, half_hi<DT>(sb));
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        float& to = s[r][4 * blk + i];
                        to = g == 0 ? b * qsum[r][g] : fmaf(b, qsum[r][g], to);
                        to = fmaf(sc, part[r][i], to);
                    }
                }
            }
        }
        uint32_t seen[RT];   // a bit for each of the lane's tokens
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            seen[r] = 0xffu;
            if constexpr (MASK) {
                seen[r] = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int t = key + 16 * (e / 4) + 4 * h + e % 4;
                    const bool see = t >= lo[r] && t <= hi[r] && x.there[e / 4];
                    seen[r] |= (see ? 1u : 0u) << e;
                    s[r][e] = see ? s[r][e] : -INFINITY;
                }
            }
            float mx = s[r][0];
#pragma unroll
            for (int e = 1; e < 8; ++e) mx = fmaxf(mx, s[r][e]);
            mx *= scale;
            if (__any(mx > top[r])) {
                const float now = row_max(fmaxf(mx, top[r] - H::kSlack));
                const float safe = now > -INFINITY ? now : 0.0f;
                const float fade = top[r] > -INFINITY ? __builtin_amdgcn_exp2f(m[r] - safe) : 0.0f;
                top[r] = now + H::kSlack;
                m[r] = safe;
                l[r] *= fade;
#pragma unroll
                for (int g = 0; g < G; ++g) fix[r][g] *= fade;
#pragma unroll
                for (int b = 0; b < NB; ++b) o[r][b] *= fade;
            }
        }
        // p, and p s as the matrix cores take it
        u32x4 ps[RT][G];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[r][e] = __builtin_amdgcn_exp2f(fmaf(s[r][e], scale, -m[r]));
                if constexpr (MASK) s[r][e] = (seen[r] >> e) & 1u ? s[r][e] : 0.0f;
                l[r] += s[r][e];
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float sc[8], b[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t sb = x.vs[e / 4][(e % 4) * G + g];
                sc[e] = half_lo<DT>(sb);
                b[e] = fmaf(8.0f, sc[e], half_hi<DT>(sb));
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const bool see = !MASK || ((seen[r] >> e) & 1u);   // what is not seen may hold infinities
                    w[e] = see ? s[r][e] * sc[e] : 0.0f;
                    fix[r][g] = see ? fmaf(s[r][e], b[e], fix[r][g]) : fix[r][g];
                }
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    ps[r][g][e] = H::pack(w[2 * e], w[2 * e + 1]);
                    sum = H::dot2(ps[r][g][e], H::ONES, sum);
                }
                fix[r][g] = fmaf(-(H::OFF + 8.0f), sum, fix[r][g]);
            }
        }
#pragma unroll
        for (int a = 0; a < D / 64; ++a) {
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const u32x4 v = {H::codes(x.v[0][2 * a], f), H::codes(x.v[0][2 * a + 1], f),
                                 H::codes(x.v[1][2 * a], f), H::codes(x.v[1][2 * a + 1], f)};
                const int nb = 4 * a + f;
#pragma unroll
                for (int r = 0; r < RT; ++r) o[r][nb] = H::mfma(v, ps[r][nb * 16 / GS], o[r][nb]);
            }
        }
    }

    // Adds the lanes' parts: after this o is the row's sum of p v, l of p.
    __device__ __forceinline__ void join() {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            l[r] = row_sum(l[r]);
#pragma unroll
            for (int g = 0; g < G; ++g) fix[r][g] = row_sum(fix[r][g]);
#pragma unroll
            for (int b = 0; b < NB; ++b) o[r][b] += fix[r][b * 16 / GS];
        }
    }
};

// 32 tokens from step * 32 on into registers.  `table` is the request's row of
// the block table; blocks from `blocks` on are not read.
template <int NJ, int G>
__device__ __forceinline__ void load_tokens(Tokens<NJ, G>& x, const Kv4View& c, const int* table, int blocks,
                                            int head, int step) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int blk = 2 * step + i;
        int page = blk < blocks ? table[blk >> c.page_shift] : -1;
        x.there[i] = page >= 0 && page < c.num_pages;
        if (!x.there[i]) page = 0;
        const size_t at = (((size_t)page * c.heads + head) << c.page_shift) + (blk & ((1 << c.page_shift) - 1));
        load_words(x.k[i], c.kc + at * (64 * NJ) + lane * NJ);
        load_words(x.v[i], c.vc + at * (64 * NJ) + lane * NJ);
        load_words(x.ks[i], c.ks + at * (16 * G) + (lane >> 4) * (4 * G));
        load_words(x.vs[i], c.vs + at * (16 * G) + (lane >> 4) * (4 * G));
    }
}

// Keys that a request's splits divide: from the first that its first query
// sees (a multiple of 32) to the end.
__device__ __forceinline__ void key_span(const Kv4AttnArgs& a, int kv, int count, int& begin, int& end) {
    const int first = kv - count;
    begin = a.window ? max(0, first - a.window + 1) & ~31 : 0;
    end = min(kv, a.max_kv);
}

// WM waves along the rows, each with its own RT tiles; WK waves along the keys,
// which take every WK-th step of 32 tokens and are joined in LDS.
template <int D, int GS, int DT, int RT, int WM, int WK>
__global__ __launch_bounds__(64 * WM * WK) void kv4_attn_kernel(Kv4AttnArgs a) {
    static_assert(WM == 1 || WK == 1, "waves are along one axis");
    using R = Rows<D, GS, DT, RT>;
    constexpr int NJ = R::NJ, G = R::G, NB = R::NB, PITCH = D + 4;
    __shared__ float s_o[WK > 1 ? WK : 1][WK > 1 ? 16 * PITCH : 1];
    __shared__ float s_m[WK][16], s_l[WK][16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, n = lane & 15, h = lane >> 4;
    const Kv4View& c = a.c;

    int id = blockIdx.x;
    const int head = id % c.heads;
    id /= c.heads;
    const int tile = a.tiles - 1 - id % a.tiles;   // the tiles that see most keys first
    id /= a.tiles;
    const int req = id % (a.requests + 1);
    const int split = id / (a.requests + 1);

    if (req == a.requests) {   // the tokens of no request
        if (split || a.splits > 1) return;
        const int begin = max(a.offsets[a.requests], 0);
        const long long per = (long long)a.each * D / 8;
        const long long all = max(0, a.tokens - begin) * per;
        for (long long i = (long long)tile * blockDim.x + threadIdx.x; i < all; i += (long long)a.tiles * blockDim.x) {
            const long long at = (begin + i / per) * a.heads + (long long)head * a.each;
            reinterpret_cast<u32x4*>(a.out)[at * (D / 8) + i % per] = u32x4{0, 0, 0, 0};
            if (a.lse && i % per < a.each) a.lse[at + i % per] = -INFINITY;
        }
        return;
    }

    const int start = max(a.offsets[req], 0), kv = a.kv_lens[req];
    const int count = min(min(a.offsets[req + 1], a.tokens) - start, a.max_query);
    const int rows = count * a.each;
    const int row0 = (tile * WM + (WM > 1 ? wave : 0)) * 16 * RT;
    const bool mine = row0 < rows;
    if (WK > 1 && !mine) return;   // the whole work-group

    int begin, end;
    key_span(a, kv, a.offsets[req + 1] - start, begin, end);
    if (a.splits > 1) {
        begin += split * a.chunk;
        if (begin >= end) return;
        end = min(end, begin + a.chunk);
    }

    R x;
    x.clear();
    const int back = kv - (a.offsets[req + 1] - start);   // the first query's position
    const int last_row = min(row0 + 16 * RT, rows) - 1;
    const int pos0 = back + row0 / a.each, pos1 = back + last_row / a.each;
    const float scale = a.scale_log2;
    long long token[RT];
    int qhead[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int row = min(row0 + 16 * r + n, last_row);
        const int i = mine ? row / a.each : 0;
        token[r] = (long long)start + i;
        qhead[r] = head * a.each + (mine ? row - i * a.each : 0);
        const int pos = back + i;
        x.lo[r] = a.window ? pos - a.window + 1 : 0;
        x.hi[r] = min(pos, end - 1);
    }
    if (mine) {
        const uint16_t* q = static_cast<const uint16_t*>(a.q);
        const bool vec = (((uintptr_t)a.q & 15) | ((a.q_ts | a.q_hs) & 7)) == 0;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const uint16_t* from = q + token[r] * a.q_ts + qhead[r] * a.q_hs + 8 * h;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                if (vec) {
                    x.q[r][j] = *reinterpret_cast<const u32x4*>(from + 32 * j);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x.q[r][j][e] = (uint32_t)from[32 * j + 2 * e] | ((uint32_t)from[32 * j + 2 * e + 1] << 16);
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float sum = 0.0f;
#pragma unroll
                for (int j = g * (GS / 32); j < (g + 1) * (GS / 32); ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum += half_lo<DT>(x.q[r][j][e]) + half_hi<DT>(x.q[r][j][e]);
                x.qsum[r][g] = row_sum(sum);
            }
        }
        const int first = max(begin, a.window ? pos0 - a.window + 1 : 0);
        const int stop = min(end, pos1 + 1);
        const int full_lo = a.window ? pos1 - a.window + 1 : 0, full_hi = min(pos0, end - 1);
        const int* table = a.table + req * a.table_stride;
        const int blocks = min(((stop + 15) >> 4), a.columns << c.page_shift);
        int step = first >> 5;
        if (WK > 1) step += wave;
        const int steps = (stop + 31) >> 5;
        Tokens<NJ, G> t[2];
        auto work = [&](const Tokens<NJ, G>& y, int at) {
            const int key = at * 32;
            if (key >= full_lo && key + 31 <= full_hi && y.there[0] && y.there[1])
                x.template step<false>(y, key, scale);
            else
                x.template step<true>(y, key, scale);
        };
        if (step < steps) load_tokens(t[0], c, table, blocks, head, step);
        while (step < steps) {
            if (step + WK < steps) load_tokens(t[1], c, table, blocks, head, step + WK);
            work(t[0], step);
            step += WK;
            if (step >= steps) break;
            if (step + WK < steps) load_tokens(t[0], c, table, blocks, head, step + WK);
            work(t[1], step);
            step += WK;
        }
        x.join();
    }

#pragma unroll
    for (int r = 0; r < RT; ++r) {
        float m = x.m[r], l = x.l[r];
        bool seen = x.top[r] > -INFINITY || l != l;
        const bool row_there = mine && row0 + 16 * r + n <= last_row;
        if constexpr (WK > 1) {
            if (r) __syncthreads();
            if (h == 0) {
                s_m[wave][n] = seen ? m : -INFINITY;
                s_l[wave][n] = l;
            }
            __syncthreads();
            float all = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < WK; ++w) all = fmaxf(all, s_m[w][n]);
            const float safe = all > -INFINITY ? all : 0.0f;
#pragma unroll
            for (int w = 0; w < WK; ++w) sum += s_l[w][n] * __builtin_amdgcn_exp2f(s_m[w][n] - safe);
            const float f = seen ? __builtin_amdgcn_exp2f(m - safe) : 0.0f;
#pragma unroll
            for (int b = 0; b < NB; ++b)
                *reinterpret_cast<f32x4*>(&s_o[wave][n * PITCH + 16 * b + 4 * h]) = x.o[r][b] * f;
            __syncthreads();
            m = safe;
            l = sum;
            seen = all > -INFINITY || l != l;
        }
        const long long at = token[r] * a.heads + qhead[r];
        const float inv = a.splits > 1 ? 1.0f : l != 0.0f ? 1.0f / l : 0.0f;
        auto store = [&](int b, f32x4 v) {
            v *= inv;
            if (a.splits > 1)
                *reinterpret_cast<f32x4*>(a.part + ((long long)split * a.tokens * a.heads + at) * D + 16 * b + 4 * h) = v;
            else
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at * D + 16 * b + 4 * h) =
                    u32x2{R::H::pack(v[0], v[1]), R::H::pack(v[2], v[3])};
        };
        if (!row_there) continue;
        if constexpr (WK > 1) {
#pragma unroll
            for (int b0 = 0; b0 < NB; b0 += WK) {
                const int b = b0 + wave;
                if (NB % WK != 0 && b >= NB) break;
                f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < WK; ++w) v += *reinterpret_cast<const f32x4*>(&s_o[w][n * PITCH + 16 * b + 4 * h]);
                store(b, v);
            }
        } else {
#pragma unroll
            for (int b = 0; b < NB; ++b) store(b, x.o[r][b]);
        }
        if (h == 0 && (WM > 1 || wave == 0)) {
            if (a.splits > 1) {
                float* stat = a.part + (long long)a.splits * a.tokens * a.heads * D;
                f32x2* to = reinterpret_cast<f32x2*>(stat) + (long long)split * a.tokens * a.heads + at;
                *to = f32x2{seen ? m : -INFINITY, l};
            } else if (a.lse) {
                a.lse[at] = seen ? (m + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f : -INFINITY;
            }
        }
    }
}

// Joins the splits: a wave takes one (query, head).
template <int D, int DT>
__global__ __launch_bounds__(256) void kv4_join_kernel(Kv4AttnArgs a) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63;
    long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int head = (int)(id % a.heads);
    id /= a.heads;
    const int i = (int)(id % a.max_query), req = (int)(id / a.max_query);
    if (req > a.requests) return;
    uint16_t* out = static_cast<uint16_t*>(a.out);
    const int start = max(a.offsets[req], 0);
    if (req == a.requests) {
        for (long long t = (long long)start + i; t < a.tokens; t += a.max_query) {
#pragma unroll
            for (int e = 0; e < E; ++e) out[(t * a.heads + head) * D + e * 64 + lane] = 0;
            if (a.lse && lane == 0) a.lse[t * a.heads + head] = -INFINITY;
        }
        return;
    }
    const int count = a.offsets[req + 1] - start;
    if (i >= count || start + i >= a.tokens) return;
    int begin, end;
    key_span(a, a.kv_lens[req], count, begin, end);
    const int splits = end > begin ? (end - begin + a.chunk - 1) / a.chunk : 0;
    const long long at = ((long long)start + i) * a.heads + head, all = (long long)a.tokens * a.heads;
    const f32x2* stat = reinterpret_cast<const f32x2*>(a.part + (long long)a.splits * all * D);
    float m = -INFINITY;
    for (int s = lane; s < splits; s += 64) m = fmaxf(m, stat[s * all + at][0]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    const float safe = m > -INFINITY ? m : 0.0f;
    float l = 0.0f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        const f32x2 st = stat[s * all + at];
        const float f = __builtin_amdgcn_exp2f(st[0] - safe);
        l += st[1] * f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += f * a.part[(s * all + at) * D + e * 64 + lane];
    }
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) store_elem<DT>(out, at * D + e * 64 + lane, o[e] * inv);
    if (a.lse && lane == 0)
        a.lse[at] = l != 0.0f ? (m + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f : -INFINITY;
}

template <int D, int GS, int DT>
hipError_t launch_format(const Kv4AttnArgs& a, const Kv4AttnPlan& p, hipStream_t st) {
    const dim3 grid((unsigned)((long long)p.splits * (a.requests + 1) * p.tiles * a.c.heads));
    if (p.wk == 8) kv4_attn_kernel<D, GS, DT, 1, 1, 8><<<grid, dim3(512), 0, st>>>(a);
    else if (p.wk == 4) kv4_attn_kernel<D, GS, DT, 1, 1, 4><<<grid, dim3(256), 0, st>>>(a);
    else kv4_attn_kernel<D, GS, DT, 2, 4, 1><<<grid, dim3(256), 0, st>>>(a);
    hipError_t err = hipGetLastError();
    if (err == hipSuccess && p.splits > 1) {
        const long long rows = (long long)(a.requests + 1) * a.max_query * a.heads;
        kv4_join_kernel<D, DT><<<dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st>>>(a);
        err = hipGetLastError();
    }
    return err;
}

// One source for each head size and type.
template <int D, int DT>
hipError_t launch_dim(const Kv4AttnArgs& a, const Kv4AttnPlan& p, hipStream_t st) {
    if (a.c.group == 32) return launch_format<D, 32, DT>(a, p, st);
    if constexpr (D >= 128)
        if (a.c.group == 128) return launch_format<D, 128, DT>(a, p, st);
    return launch_format<D, 64, DT>(a, p, st);
}

extern template hipError_t launch_dim<64, DT_F16>(const Kv4AttnArgs&, const Kv4AttnPlan&, hipStream_t);
extern template hipError_t launch_dim<128, DT_F16>(const Kv4AttnArgs&, const Kv4AttnPlan&, hipStream_t);
extern template hipError_t launch_dim<256, DT_F16>(const Kv4AttnArgs&, const Kv4AttnPlan&, hipStream_t);
extern template hipError_t launch_dim<64, DT_BF16>(const Kv4AttnArgs&, const Kv4AttnPlan&, hipStream_t);
extern template hipError_t launch_dim<128, DT_BF16>(const Kv4AttnArgs&, const Kv4AttnPlan&, hipStream_t);
extern template hipError_t launch_dim<256, DT_BF16>(const Kv4AttnArgs&, const Kv4AttnPlan&, hipStream_t);

}  // namespace kv4
}  // namespace qmx
