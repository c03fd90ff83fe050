// rope.hip -- rotary positions of queries and keys: the pair (a, b) of a head's
// elements turns by t = position * frequency,
//   (a, b) -> scale * (a cos t - b sin t, b cos t + a sin t).
//
// Bound by memory: each head is read and written once.  A token's cosines and
// sines are formed once for all of its heads, in LDS: the angle in turns in 64
// bits, of which a whole number is taken off exactly, the rest in 32.  An item is
// eight pairs, two loads of 16 bytes: of both halves of the rotated part, or of
// 16 neighbours; the part that is not rotated is copied in items of 16 elements.
// 8192 tokens of 40 + 8 heads of 128 in bfloat16: 41 us, 4.9 TB/s, a large copy's rate.
#include <algorithm>

#include "f8.h"
#include "f8_device.h"

namespace qmx {
namespace {

constexpr int THREADS = 256;
constexpr int MOST_TOKENS = 1 << 23;   // of a launch, whose grid has below 2^32 threads

struct Ends {   // what an item holds of its two runs of 8 elements
    u32x4 lo, hi;
};

// TOK tokens a work-group; a token's heads may be spread over gridDim.y groups.
template <int DT, bool INTER, int TOK>
__global__ __launch_bounds__(THREADS) void rope_kernel(RopeArgs a) {
    extern __shared__ float2 turn[];   // [TOK][pairs]
    const int tid = threadIdx.x, n = a.pairs;
    const long long t0 = (long long)blockIdx.x * TOK;
    for (int i = tid; i < TOK * n; i += THREADS) {
        const int k = i / n, pair = i - k * n;
        const long long t = t0 + k;
        float2 cs = {1.0f, 0.0f};
        if (t < a.tokens) {
            const int at = a.positions[t];
            if (at >= 0) {
                const double turns = (double)at * (a.frequencies[pair] * 0.15915494309189533577);
                const float rest = (float)(turns - rint(turns));
                float s, c;
                sincospif(2.0f * rest, &s, &c);
                cs = {c * a.scale, s * a.scale};
            }
        }
        turn[i] = cs;
    }
    __syncthreads();
    const int rotated = (n + 7) / 8, rest = (a.dim - 2 * n + 15) / 16, items = rotated + rest;
    const int heads = a.heads[0] + a.heads[1];
    const int total = TOK * heads * items;
    for (int i = blockIdx.y * THREADS + tid; i < total; i += gridDim.y * THREADS) {
        const int k = i / (heads * items), left = i - k * (heads * items);
        const int both = left / items, item = left - both * items;
        const long long t = t0 + k;
        if (t >= a.tokens) continue;
        const int which = both >= a.heads[0] ? 1 : 0, head = both - (which ? a.heads[0] : 0);
        const uint16_t* in = static_cast<const uint16_t*>(a.in[which]) + t * a.in_ts[which] + head * a.in_hs[which];
        uint16_t* out = static_cast<uint16_t*>(a.out[which]) + t * a.out_ts[which] + head * a.out_hs[which];
        int p0, p1, n0, n1;   // where the two runs begin, and how long they are
        if (item >= rotated) {
            p0 = 2 * n + 16 * (item - rotated);
            p1 = p0 + 8;
            n0 = a.dim - p0;
            n1 = a.dim - p1;
        } else if (INTER) {
            p0 = 16 * item;
            p1 = p0 + 8;
            n0 = 2 * n - p0;
            n1 = 2 * n - p1;
        } else {
            p0 = 8 * item;
            p1 = n + p0;
            n0 = n1 = n - p0;
        }
        const bool turned = item < rotated && a.positions[t] >= 0;
        if (!turned && a.in_place[which]) continue;
        Ends e = {load_part(in + p0, n0), load_part(in + p1, n1)};
        if (turned) {
            const float2* cs = turn + k * n + 8 * item;
            const int pairs = min(8, n - 8 * item);
            Ends o = e;
            if (INTER) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 c = cs[min(j, pairs - 1)];
                    const uint32_t w = j < 4 ? e.lo[j & 3] : e.hi[j & 3];
                    const float x = half_lo<DT>(w), y = half_hi<DT>(w);
                    const uint32_t r = pack2<DT>(fmaf(x, c.x, -y * c.y), fmaf(y, c.x, x * c.y));
                    if (j < 4) o.lo[j & 3] = r;
                    else o.hi[j & 3] = r;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 c = cs[min(2 * j, pairs - 1)], d = cs[min(2 * j + 1, pairs - 1)];
                    const float x0 = half_lo<DT>(e.lo[j]), y0 = half_lo<DT>(e.hi[j]);
                    const float x1 = half_hi<DT>(e.lo[j]), y1 = half_hi<DT>(e.hi[j]);
                    o.lo[j] = pack2<DT>(fmaf(x0, c.x, -y0 * c.y), fmaf(x1, d.x, -y1 * d.y));
                    o.hi[j] = pack2<DT>(fmaf(y0, c.x, x0 * c.y), fmaf(y1, d.x, x1 * d.y));
                }
            }
            e = o;
        }
        store_part<false>(out + p0, e.lo, n0);
        store_part<false>(out + p1, e.hi, n1);
    }
}

template <int DT, bool INTER, int TOK>
void go(const RopeArgs& a, int per_token, hipStream_t st) {
    const unsigned groups = (unsigned)((a.tokens + TOK - 1) / TOK);
    const int each = groups <= 1024 ? THREADS : 2 * THREADS;
    hipLaunchKernelGGL((rope_kernel<DT, INTER, TOK>), dim3(groups, (unsigned)((TOK * per_token + each - 1) / each)),
                       dim3(THREADS), TOK * a.pairs * sizeof(float2), st, a);
}

// Tokens with less than three quarters of a work-group's items share one by fours (8192
// of 8 + 1 heads of 128: 12.1 us, 16.1 each by itself; of 20 + 4 24.4 either way; of 40 + 8
// 44.7, 40.7).  A token is spread over as many work-groups as give each thread one item
// where they are few (512 of 40 + 8 heads: 5.5 us, 6.3 as one), and two otherwise (8192
// of 40 + 8: 40.7, 43.7 with one; 4096 of 129 heads of 576: 252, 273 unspread).
template <int DT, bool INTER>
void pick(const RopeArgs& a, hipStream_t st) {
    const int per_token = ((a.pairs + 7) / 8 + (a.dim - 2 * a.pairs + 15) / 16) * (a.heads[0] + a.heads[1]);
    if (per_token < 192) go<DT, INTER, 4>(a, per_token, st);   // so at most 1528 pairs, 48 KB of LDS
    else go<DT, INTER, 1>(a, per_token, st);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& all, int dt, hipStream_t st) {
    RopeArgs a = all;
    a.tokens = std::min(all.tokens, MOST_TOKENS);
    if (dt == DT_F16) a.interleaved ? pick<DT_F16, true>(a, st) : pick<DT_F16, false>(a, st);
    else a.interleaved ? pick<DT_BF16, true>(a, st) : pick<DT_BF16, false>(a, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.tokens == all.tokens) return e;
    for (int i = 0; i < 2; ++i) {
        a.in[i] = static_cast<const uint16_t*>(a.in[i]) + a.in_ts[i] * a.tokens;
        a.out[i] = static_cast<uint16_t*>(a.out[i]) + a.out_ts[i] * a.tokens;
    }
    a.positions += a.tokens;
    a.tokens = all.tokens - a.tokens;
    return launch_rope(a, dt, st);
}

}  // namespace qmx
