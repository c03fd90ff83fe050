// kv4_cache.hip -- tokens into the paged 4-bit cache, and back.
#include "kv4.h"
#include "qmx_device.h"

namespace qmx {
namespace {

constexpr int THREADS = 256;

// Two 16-bit floats as integers that order as they do (a NaN beyond both
// infinities, by its sign), and back: the map is its own inverse.
__device__ __forceinline__ uint32_t sortable(uint32_t w) {
    const uint32_t sign = (w >> 15) & 0x00010001u;
    return w ^ ((sign << 15) - sign);
}

typedef short s16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(s16x2, a),
                                                                  __builtin_bit_cast(s16x2, b)));
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(s16x2, a),
                                                                  __builtin_bit_cast(s16x2, b)));
}

template <int DT>
__device__ __forceinline__ float as_float(uint32_t h) {
    return DT == DT_F16 ? f16_bits_to_f32(h) : bf16_bits_to_f32(h);
}

// (hi - lo) / 15 to the type.  Two roundings, to 32 bits and to the type, give
// what one gives: the binary digits of a quotient by 15 repeat every four
// places, so it is never next to a middle between two 16-bit values.
template <int DT>
__device__ __forceinline__ uint32_t group_scale(float lo, float hi) {
    const float f = (hi - lo) / 15.0f;
    return DT == DT_F16 ? f32_to_f16_bits(f) : f32_to_bf16_bits(f);
}

// Eight codes.  rint of a product with the reciprocal, set right against the
// middles between codes by an exact remainder; where x - b itself was rounded
// the group's eight are done in 64 bits.
__device__ __forceinline__ void codes_of(const float (&x)[8], float b, float s, uint32_t (&c)[8]) {
    if (!(s > 0.0f) || !(s < INFINITY)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = 0;
        return;
    }
    const float inv = __builtin_amdgcn_rcpf(s), half = 0.5f * s;
    bool rounded = !(inv < INFINITY);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float t = x[e] - b;
        rounded |= (t + b != x[e]) | (x[e] - t != b);
        float c0 = fminf(rintf(t * inv), 15.0f);
        const float r = fmaf(-c0, s, t);
        const bool odd = ((int)c0 & 1) != 0;
        c0 += (odd ? r >= half : r > half) ? 1.0f : 0.0f;
        c0 -= (odd ? r <= -half : r < -half) ? 1.0f : 0.0f;
        c[e] = (uint32_t)(int)fminf(fmaxf(c0, 0.0f), 15.0f);
    }
    if (rounded) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            c[e] = (uint32_t)(int)fmin(fmax(rint(((double)x[e] - (double)b) / (double)s), 0.0), 15.0);
    }
}

template <bool VEC>
__device__ __forceinline__ u32x4 load8(const uint16_t* p) {
    if constexpr (VEC) return *reinterpret_cast<const u32x4*>(p);
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
    return w;
}

// Codes of the lane's eight elements, and the (scale, bias) pair of its group,
// whose elements lie in GS / 8 neighbouring lanes.
template <int DT, int GS>
__device__ __forceinline__ uint32_t quantise8(u32x4 w, uint32_t (&c)[8]) {
    uint32_t lo = sortable(w[0]), hi = lo;
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        const uint32_t k = sortable(w[i]);
        lo = min2(lo, k);
        hi = max2(hi, k);
    }
#pragma unroll
    for (int off = 1; off < GS / 8; off <<= 1) {
        lo = min2(lo, __shfl_xor(lo, off, 64));
        hi = max2(hi, __shfl_xor(hi, off, 64));
    }
    lo = min2(lo, (lo >> 16) | (lo << 16));
    hi = max2(hi, (hi >> 16) | (hi << 16));
    const uint32_t lob = sortable(lo) & 0xffffu, hib = sortable(hi) & 0xffffu;
    const float b = as_float<DT>(lob);
    const uint32_t sb = group_scale<DT>(b, as_float<DT>(hib));
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = half_lo<DT>(w[i]);
        x[2 * i + 1] = half_hi<DT>(w[i]);
    }
    codes_of(x, b, as_float<DT>(sb), c);
    return sb | (lob << 16);
}

// D / 8 lanes take one row (token, head): a lane its eight neighbouring
// elements.  Keys: the lane's codes are one word.  Values: a half holds the
// codes of elements 16 apart, which lie in four lanes; two exchanges leave
// each of the four with two whole halves.
template <int D, int GS, int DT, bool VEC>
__global__ __launch_bounds__(THREADS) void kv4_write_kernel(Kv4View c, const uint16_t* k, const uint16_t* v,
                                                            long long k_ts, long long k_hs, long long v_ts,
                                                            long long v_hs, const int* slots, int tokens) {
    constexpr int LANES = D / 8;
    const long long unit = ((long long)blockIdx.x * THREADS + threadIdx.x) / LANES;
    const int u = threadIdx.x % LANES;
    const long long token = unit / c.heads;
    const int head = (int)(unit % c.heads);
    const int slot = token < tokens ? slots[token] : -1;
    const int page_tokens = 16 << c.page_shift;
    const int page = slot >= 0 ? slot / page_tokens : -1;
    if (page < 0 || page >= c.num_pages) return;   // whole rows leave together
    const int at = slot % page_tokens;
    const long long row = (long long)page * c.heads + head;
    const long long block = (row << c.page_shift) + (at >> 4);
    const long long pair = (row * page_tokens + at) * (D / GS) + u / (GS / 8);
    const int t = at & 15;
    uint32_t x[8];

    const u32x4 kw = load8<VEC>(k + token * k_ts + head * k_hs + 8 * u);
    const u32x4 vw = load8<VEC>(v + token * v_ts + head * v_hs + 8 * u);
    uint32_t sb = quantise8<DT, GS>(kw, x);
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) word |= x[e] << (4 * (e / 2) + 16 * (e % 2));
    c.kc[block * (2 * D) + ((u & 3) * 16 + t) * (D / 32) + u / 4] = word;
    if (u % (GS / 8) == 0) c.ks[pair] = sb;

    sb = quantise8<DT, GS>(vw, x);
    const int f = (u >> 1) & 3;
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = (x[2 * i] | (x[2 * i + 1] << 16)) << (4 * f);
    const bool up = f & 2;
    uint32_t a0 = up ? p[2] : p[0], a1 = up ? p[3] : p[1];
    a0 |= __shfl_xor(up ? p[0] : p[2], 4, 64);
    a1 |= __shfl_xor(up ? p[1] : p[3], 4, 64);
    const bool odd = f & 1;
    uint32_t h = odd ? a1 : a0;
    h |= __shfl_xor(odd ? a0 : a1, 2, 64);
    const int n = 8 * (u & 1) + 2 * f;
    uint16_t* to = reinterpret_cast<uint16_t*>(c.vc) + block * (4 * D) +
                   ((((t >> 2) * 16 + n) * (D / 64) + u / 8) * 4 + (t & 3));
    to[0] = (uint16_t)h;
    to[D / 16] = (uint16_t)(h >> 16);
    if (u % (GS / 8) == 0) c.vs[pair] = sb;
}

// The same cut of the work: a lane gives eight neighbouring elements.
template <int D, int GS, int DT>
__global__ __launch_bounds__(THREADS) void kv4_read_kernel(Kv4View c, uint16_t* k, uint16_t* v, const int* slots,
                                                           int tokens) {
    constexpr int LANES = D / 8;
    const long long unit = ((long long)blockIdx.x * THREADS + threadIdx.x) / LANES;
    const int u = threadIdx.x % LANES;
    const long long token = unit / c.heads;
    const int head = (int)(unit % c.heads);
    if (token >= tokens) return;
    const int slot = slots[token];
    const int page_tokens = 16 << c.page_shift;
    const int page = slot >= 0 ? slot / page_tokens : -1;
    u32x4 ko = {0, 0, 0, 0}, vo = {0, 0, 0, 0};
    if (page >= 0 && page < c.num_pages) {
        const int at = slot % page_tokens;
        const long long row = (long long)page * c.heads + head;
        const long long block = (row << c.page_shift) + (at >> 4);
        const long long pair = (row * page_tokens + at) * (D / GS) + u / (GS / 8);
        const int t = at & 15, f = (u >> 1) & 3;
        const uint32_t word = c.kc[block * (2 * D) + ((u & 3) * 16 + t) * (D / 32) + u / 4];
        const uint32_t ksb = c.ks[pair], vsb = c.vs[pair];
        const uint16_t* from = reinterpret_cast<const uint16_t*>(c.vc) + block * (4 * D) +
                               ((((t >> 2) * 16 + 8 * (u & 1)) * (D / 64) + u / 8) * 4 + (t & 3));
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = from[i * (D / 16)];
        const float s = half_lo<DT>(ksb), b = half_hi<DT>(ksb);
        const float s2 = half_lo<DT>(vsb), b2 = half_hi<DT>(vsb);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[2], w2[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float x = fmaf((float)((word >> (4 * i + 16 * j)) & 15u), s, b);
                const float y = fmaf((float)((h[2 * i + j] >> (4 * f)) & 15u), s2, b2);
                w[j] = DT == DT_F16 ? f32_to_f16_bits(x) : f32_to_bf16_bits(x);
                w2[j] = DT == DT_F16 ? f32_to_f16_bits(y) : f32_to_bf16_bits(y);
            }
            ko[i] = w[0] | (w[1] << 16);
            vo[i] = w2[0] | (w2[1] << 16);
        }
    }
    *reinterpret_cast<u32x4*>(k + unit * D + 8 * u) = ko;
    *reinterpret_cast<u32x4*>(v + unit * D + 8 * u) = vo;
}

// Calls f with the cache's head size, group size and type as constants.
template <class F>
hipError_t with_format(const Kv4View& c, F&& f) {
    auto by_type = [&](auto d, auto g) {
        return c.dt == DT_F16 ? f(d, g, std::integral_constant<int, DT_F16>())
                              : f(d, g, std::integral_constant<int, DT_BF16>());
    };
    auto by_group = [&](auto d) {
        if (c.group == 32) return by_type(d, std::integral_constant<int, 32>());
        if constexpr (decltype(d)::value >= 128)
            if (c.group == 128) return by_type(d, std::integral_constant<int, 128>());
        return by_type(d, std::integral_constant<int, 64>());
    };
    if (c.dim == 64) return by_group(std::integral_constant<int, 64>());
    if (c.dim == 128) return by_group(std::integral_constant<int, 128>());
    return by_group(std::integral_constant<int, 256>());
}

unsigned blocks_for(const Kv4View& c, int tokens) {
    return (unsigned)(((long long)tokens * c.heads * (c.dim / 8) + THREADS - 1) / THREADS);
}

}  // namespace

hipError_t launch_kv4_write(const Kv4View& c, const void* k, const void* v, long long k_ts, long long k_hs,
                            long long v_ts, long long v_hs, const int* slots, int tokens, hipStream_t st) {
    const bool vec = (((uintptr_t)k | (uintptr_t)v) & 15) == 0 && ((k_ts | k_hs | v_ts | v_hs) & 7) == 0;
    return with_format(c, [&](auto d, auto g, auto t) {
        constexpr int D = decltype(d)::value, GS = decltype(g)::value, DT = decltype(t)::value;
        const auto kernel = vec ? kv4_write_kernel<D, GS, DT, true> : kv4_write_kernel<D, GS, DT, false>;
        kernel<<<dim3(blocks_for(c, tokens)), dim3(THREADS), 0, st>>>(
            c, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_ts, k_hs, v_ts, v_hs, slots,
            tokens);
        return hipGetLastError();
    });
}

hipError_t launch_kv4_read(const Kv4View& c, void* k, void* v, const int* slots, int tokens, hipStream_t st) {
    return with_format(c, [&](auto d, auto g, auto t) {
        constexpr int D = decltype(d)::value, GS = decltype(g)::value, DT = decltype(t)::value;
        kv4_read_kernel<D, GS, DT><<<dim3(blocks_for(c, tokens)), dim3(THREADS), 0, st>>>(
            c, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), slots, tokens);
        return hipGetLastError();
    });
}

}  // namespace qmx
