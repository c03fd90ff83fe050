// kv4_cache.hip -- tokens into the paged 4-bit cache, and back.
//
// Bound by memory, but for the vector ALU's work of finding codes.  Measured:
// writing 23000 tokens (8 heads of 128, groups of 32, float16) 43 us for 188 MB, 4.3
// TB/s (60 us with 64-bit quotients at middles between codes and exchanges
// through LDS); reading 160000 tokens (8 heads of 64) 66 us for 413 MB, 6.3 TB/s
// with half of them cached (142 us a token at a time over all heads, which used
// a quarter of each line of codes; 105 us without streaming stores).
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

// Eight codes.  With 1.5 * 2^23 added, the nearest whole number to (x - b) / s
// stands in a float's low bits; the reciprocal may put it off by one next to a
// middle, so the remainder, which is exact, is held against s / 2 (just under it
// where the number is odd: middles go to even).  x - b is exact in 32 bits unless
// x, or b, has digits more than 24 places below the group's span: then the
// lane's eight are done with remainders in 64 bits.  UP: a power of two that
// everything is multiplied by.
template <int DT, class Up>
__device__ __forceinline__ void codes_times(u32x4 w, float b, float s, bool deep, Up, uint32_t (&c)[8]) {
    constexpr int MAGIC = 0x4b400000;
    constexpr float UP = Up::value ? 0x1p100f : 1.0f;
    b *= UP;
    s *= UP;
    const float inv = __builtin_amdgcn_rcpf(s), half = 0.5f * s;
    const float magic = __int_as_float(MAGIC);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = UP * (e % 2 ? half_hi<DT>(w[e / 2]) : half_lo<DT>(w[e / 2]));
        const float t = x - b, y = fmaf(t, inv, magic);
        const int k = __float_as_int(y);
        const float r = fmaf(magic - y, s, t), most = __int_as_float(__float_as_int(half) - (k & 1));
        c[e] = (uint32_t)min(max(k + (r > most ? 1 : 0) - (r < -most ? 1 : 0), MAGIC), MAGIC + 15) & 15u;
        if (deep) {
            const double rd = fma((double)(magic - y), (double)s, (double)x - (double)b), md = (double)most;
            c[e] = (uint32_t)min(max(k + (rd > md ? 1 : 0) - (rd < -md ? 1 : 0), MAGIC), MAGIC + 15) & 15u;
        }
    }
}

template <int DT>
__device__ __forceinline__ void codes_of(u32x4 w, float b, float hi, float s, uint32_t (&c)[8]) {
    if (!(s > 0.0f) || !(s < INFINITY)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = 0;
        return;
    }
    // the least magnitude but 0, less one step (so that 0 wraps to the top)
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u16x2 least = {0xffff, 0xffff};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t magnitudes = w[i] & 0x7fff7fffu;
        least = __builtin_elementwise_min(least, (u16x2)(__builtin_bit_cast(u16x2, magnitudes) - u16x2{1, 1}));
    }
    const uint32_t small = min((uint32_t)least[0], (uint32_t)least[1]);
    const float span = (hi - b) * (DT == DT_F16 ? 0x1p-13f : 0x1p-16f);
    const bool deep = (small < 0x8000u && as_float<DT>(small + 1) <= span) || (b != 0.0f && fabsf(b) <= span);
    // The reciprocal takes a subnormal for 0.  A group of so small a scale holds
    // nothing above 2^-98, bfloat16 having 8 digits, so its numbers stay finite.
    if (DT == DT_BF16 && s < 0x1p-110f) codes_times<DT>(w, b, s, deep, std::true_type(), c);
    else codes_times<DT>(w, b, s, deep, std::false_type(), c);
}

template <bool VEC>
__device__ __forceinline__ u32x4 load8(const uint16_t* p) {
    if constexpr (VEC) return *reinterpret_cast<const u32x4*>(p);
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
    return w;
}

// The value of the lane whose number differs in the bits of MASK (1, 2, 4 or 8),
// without a trip through LDS.
template <int MASK>
__device__ __forceinline__ uint32_t across(uint32_t v) {
    const int x = (int)v;
    if constexpr (MASK == 1) return (uint32_t)__builtin_amdgcn_mov_dpp(x, 0xb1, 0xf, 0xf, true);    // quad 1 0 3 2
    if constexpr (MASK == 2) return (uint32_t)__builtin_amdgcn_mov_dpp(x, 0x4e, 0xf, 0xf, true);    // quad 2 3 0 1
    if constexpr (MASK == 8) return (uint32_t)__builtin_amdgcn_mov_dpp(x, 0x128, 0xf, 0xf, true);   // row turned by 8
    const int y = __builtin_amdgcn_mov_dpp(x, 0x141, 0xf, 0xf, true);                               // halves mirrored
    return (uint32_t)__builtin_amdgcn_mov_dpp(y, 0x1b, 0xf, 0xf, true);                             // quad 3 2 1 0
}

// A row (token, head) is cut among D / 8 lanes: lane u has the eight elements
// from elements_of(u) on.  The four lanes of a quad have those 16 apart, which
// share the 16-bit halves of the value codes; a group of GS elements lies in the
// lanes that differ in bits 0 and 2 (GS = 32), 0..2 (64) or 0..3 (128).
__device__ __forceinline__ int elements_of(int u) { return 64 * (u >> 3) + 16 * (u & 3) + 8 * ((u >> 2) & 1); }

// Codes of the lane's eight elements, and the (scale, bias) pair of its group.
template <int DT, int GS>
__device__ __forceinline__ uint32_t quantise8(u32x4 w, uint32_t (&c)[8]) {
    uint32_t lo = sortable(w[0]), hi = lo;
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        const uint32_t k = sortable(w[i]);
        lo = min2(lo, k);
        hi = max2(hi, k);
    }
    auto join = [&](auto mask) {
        lo = min2(lo, across<decltype(mask)::value>(lo));
        hi = max2(hi, across<decltype(mask)::value>(hi));
    };
    join(std::integral_constant<int, 1>());
    join(std::integral_constant<int, 4>());
    if constexpr (GS >= 64) join(std::integral_constant<int, 2>());
    if constexpr (GS >= 128) join(std::integral_constant<int, 8>());
    lo = min2(lo, (lo >> 16) | (lo << 16));
    hi = max2(hi, (hi >> 16) | (hi << 16));
    const uint32_t lob = sortable(lo) & 0xffffu, hib = sortable(hi) & 0xffffu;
    const float b = as_float<DT>(lob);
    const uint32_t sb = group_scale<DT>(b, as_float<DT>(hib));
    codes_of<DT>(w, b, as_float<DT>(hib), as_float<DT>(sb), c);
    return sb | (lob << 16);
}

// Rows in the order in which the cache keeps them: 16 tokens of a head, then
// the next head, so that a work-group's rows share the cache's lines.
struct Row {
    long long token;
    int head, u;
};
template <int D>
__device__ __forceinline__ Row row_of(int heads, int tokens) {
    constexpr uint32_t LANES = D / 8;
    const uint32_t unit = blockIdx.x * (THREADS / LANES) + threadIdx.x / LANES;   // at most tokens * heads and a group
    const uint32_t block = unit / (16u * heads), in = unit - block * (16u * heads);
    const int u = (int)(threadIdx.x % LANES);
    const long long first = 16ll * block;
    if (first + 16 <= tokens) return {first + (in & 15), (int)(in >> 4), u};
    const uint32_t left = first < tokens ? (uint32_t)(tokens - first) : 1;   // the last block is short
    return {first + in % left, (int)(in / left), u};
}

// Where a token's codes and pairs are.
struct Place {
    bool there;
    long long block, pair;   // pair: of the row's first group
    int t;
};
template <int D, int GS>
__device__ __forceinline__ Place place_of(const Kv4View& c, int slot, int head) {
    Place p;
    const int page_tokens = 16 << c.page_shift;
    const int page = slot >= 0 ? slot / page_tokens : -1;
    p.there = page >= 0 && page < c.num_pages;
    const int at = slot % page_tokens;
    const long long row = (long long)page * c.heads + head;
    p.block = (row << c.page_shift) + (at >> 4);
    p.pair = (row * page_tokens + at) * (D / GS);
    p.t = at & 15;
    return p;
}

// Keys: the lane's codes are one word.  Values: a quad's codes are eight halves,
// two of which each lane is left with after two exchanges.
template <int D, int GS, int DT, bool VEC>
__global__ __launch_bounds__(THREADS) void kv4_write_kernel(Kv4View c, const uint16_t* k, const uint16_t* v,
                                                            long long k_ts, long long k_hs, long long v_ts,
                                                            long long v_hs, const int* slots, int tokens) {
    const Row row = row_of<D>(c.heads, tokens);
    if (row.token >= tokens || row.head >= c.heads) return;   // whole rows leave together
    const Place at = place_of<D, GS>(c, slots[row.token], row.head);
    if (!at.there) return;
    const int e0 = elements_of(row.u), g = e0 / GS;
    const bool tells = (e0 & (GS - 1)) == 0;   // the group's first lane
    uint32_t x[8];

    const u32x4 kw = load8<VEC>(k + row.token * k_ts + row.head * k_hs + e0);
    const u32x4 vw = load8<VEC>(v + row.token * v_ts + row.head * v_hs + e0);
    uint32_t sb = quantise8<DT, GS>(kw, x);
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) word |= x[e] << (4 * (e / 2) + 16 * (e % 2));
    c.kc[at.block * (2 * D) + ((e0 / 8 & 3) * 16 + at.t) * (D / 32) + e0 / 32] = word;
    if (tells) c.ks[at.pair + g] = sb;

    sb = quantise8<DT, GS>(vw, x);
    const int f = row.u & 3;
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = (x[2 * i] | (x[2 * i + 1] << 16)) << (4 * f);
    const bool up = f & 2, odd = f & 1;
    const uint32_t a0 = (up ? p[2] : p[0]) | across<2>(up ? p[0] : p[2]);
    const uint32_t a1 = (up ? p[3] : p[1]) | across<2>(up ? p[1] : p[3]);
    const uint32_t h = (odd ? a1 : a0) | across<1>(odd ? a0 : a1);
    const int n = (e0 & 8) + 2 * f;
    uint16_t* to = reinterpret_cast<uint16_t*>(c.vc) + at.block * (4 * D) +
                   ((((at.t >> 2) * 16 + n) * (D / 64) + e0 / 64) * 4 + (at.t & 3));
    to[0] = (uint16_t)h;
    to[D / 16] = (uint16_t)(h >> 16);
    if (tells) c.vs[at.pair + g] = sb;
}

// The same cut of the work; a lane reads two halves of the value codes and has
// the quad's other six from its neighbours.
template <int D, int GS, int DT>
__global__ __launch_bounds__(THREADS) void kv4_read_kernel(Kv4View c, uint16_t* k, uint16_t* v, const int* slots,
                                                           int tokens) {
    const Row row = row_of<D>(c.heads, tokens);
    if (row.token >= tokens || row.head >= c.heads) return;
    const Place at = place_of<D, GS>(c, slots[row.token], row.head);
    const int e0 = elements_of(row.u), f = row.u & 3;
    u32x4 ko = {0, 0, 0, 0}, vo = {0, 0, 0, 0};
    if (at.there) {
        const uint32_t word = c.kc[at.block * (2 * D) + ((e0 / 8 & 3) * 16 + at.t) * (D / 32) + e0 / 32];
        const uint32_t ksb = c.ks[at.pair + e0 / GS], vsb = c.vs[at.pair + e0 / GS];
        const uint16_t* from = reinterpret_cast<const uint16_t*>(c.vc) + at.block * (4 * D) +
                               ((((at.t >> 2) * 16 + (e0 & 8) + 2 * f) * (D / 64) + e0 / 64) * 4 + (at.t & 3));
        const int own = (int)((uint32_t)from[0] | ((uint32_t)from[D / 16] << 16));
        const uint32_t h[4] = {(uint32_t)__builtin_amdgcn_mov_dpp(own, 0x00, 0xf, 0xf, true),    // quad's lane 0
                               (uint32_t)__builtin_amdgcn_mov_dpp(own, 0x55, 0xf, 0xf, true),
                               (uint32_t)__builtin_amdgcn_mov_dpp(own, 0xaa, 0xf, 0xf, true),
                               (uint32_t)__builtin_amdgcn_mov_dpp(own, 0xff, 0xf, 0xf, true)};
        const float s = half_lo<DT>(ksb), b = half_hi<DT>(ksb);
        const float s2 = half_lo<DT>(vsb), b2 = half_hi<DT>(vsb);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[2], w2[2];
            const uint32_t codes = h[i] >> (4 * f);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float x = fmaf((float)((word >> (4 * i + 16 * j)) & 15u), s, b);
                const float y = fmaf((float)((codes >> (16 * j)) & 15u), s2, b2);
                w[j] = DT == DT_F16 ? f32_to_f16_bits(x) : f32_to_bf16_bits(x);
                w2[j] = DT == DT_F16 ? f32_to_f16_bits(y) : f32_to_bf16_bits(y);
            }
            ko[i] = w[0] | (w[1] << 16);
            vo[i] = w2[0] | (w2[1] << 16);
        }
    }
    const long long to = (row.token * c.heads + row.head) * D + e0;
    __builtin_nontemporal_store(ko, reinterpret_cast<u32x4*>(k + to));
    __builtin_nontemporal_store(vo, reinterpret_cast<u32x4*>(v + to));
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
