// f8_device.h -- device-side helpers of the 8-bit float kernels: e4m3 codes with
// a power of two for each group, held as its exponent plus 127.
#pragma once

#include "qmx_device.h"

namespace qmx {

// Eight 16-bit elements from any address of whole elements (the hardware takes
// 16-byte loads at any alignment).
struct __attribute__((packed, aligned(2))) Any16 { u32x4 v; };
__device__ __forceinline__ u32x4 load_any(const uint16_t* p) { return reinterpret_cast<const Any16*>(p)->v; }
// PASS: past the caches, where a call writes more than they are worth.
template <bool PASS>
__device__ __forceinline__ void store_any(uint16_t* p, u32x4 v) {
    if constexpr (PASS) __builtin_nontemporal_store(v, &reinterpret_cast<Any16*>(p)->v);
    else reinterpret_cast<Any16*>(p)->v = v;
}
// Eight elements or, from the end of a row on, the `n` that are there (zeros behind).
__device__ __forceinline__ u32x4 load_part(const uint16_t* p, int n) {
    if (n >= 8) return load_any(p);
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) v[i / 2] |= (uint32_t)p[i] << (16 * (i % 2));
    return v;
}
template <bool PASS>
__device__ __forceinline__ void store_part(uint16_t* p, u32x4 v, int n) {
    if (n >= 8) {
        store_any<PASS>(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (uint16_t)(v[i / 2] >> (16 * (i % 2)));
}

template <int DT>
__device__ __forceinline__ float elem(const u32x4& w, int i) {
    return i % 2 ? half_hi<DT>(w[i / 2]) : half_lo<DT>(w[i / 2]);
}

// Two floats to nearest even: gfx950 has the pair of bfloat16 in one instruction.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (DT == DT_F16) {
        return f32_to_f16_bits(a) | (f32_to_f16_bits(b) << 16);
    } else {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
    }
}

template <int DT>
__device__ __forceinline__ uint32_t to_half(float v) {
    return pack2<DT>(v, 0.0f) & 0xffffu;
}

// The largest of the 16 lanes of a row, as whole numbers, in every one of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true));    // quad 1 0 3 2
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true));    // quad 2 3 0 1
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, true));   // halves mirrored
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xf, 0xf, true));   // row mirrored
    return v;
}

// The scale of a group whose largest magnitude has the float bits `most`: e + 127,
// e the least whole number from -127 on with most <= 448 * 2^e = 1.75 * 2^(e + 8).
// A mantissa above 0.75 carries into the exponent.  255 for an infinity or a NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t most) {
    if (most >= 0x7f800000u) return 255u;
    return (uint32_t)max((int)((most + 0x1fffffu) >> 23) - 8, 0);
}

// 2^-e of a scale of at most 247 (all that scale_byte gives for numbers).
__device__ __forceinline__ float unscale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^e of any scale: 0 is 2^-127, 255 a NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
    const uint32_t u = byte == 0 ? 0x00400000u : byte << 23;
    return __uint_as_float(byte == 255 ? 0x7fc00000u : u);
}

// Eight codes of v[i] * 2^-e, each of at most 448: to nearest even.  What falls
// under float32's range by the power of two is 0 in e4m3 too.
__device__ __forceinline__ u32x2 codes8(const float (&v)[8], uint32_t byte) {
    if (byte == 255) return u32x2{0x7f7f7f7fu, 0x7f7f7f7fu};
    const float up = unscale(byte);
    u32x2 c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * up, v[4 * i + 1] * up, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * up, v[4 * i + 3] * up, w, true);
        c[i] = (uint32_t)w;
    }
    return c;
}

}  // namespace qmx
