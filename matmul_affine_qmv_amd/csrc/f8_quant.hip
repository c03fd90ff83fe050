// f8_quant.hip -- 16-bit floats into e4m3 codes with a power of two for each
// group, and back.  A lane holds 8 elements and 16 lanes a group of 128; weights
// share a scale among 128 rows.  Every step is exact but the one rounding of
// x * 2^-e, so codes are the definition's.  Bound by memory: 17408 x 5120 in blocks
// 57 us, 4.7 TB/s, and back 54 (42 while the codes are in the Infinity Cache); 40 x
// 14336 3.7 and 3.4 us.
#include "f8.h"
#include "f8_device.h"

namespace qmx {
namespace {

constexpr int THREADS = 256;
constexpr int TEAMS = THREADS / 16;   // groups a work-group holds at a time

// The largest magnitude of eight 16-bit elements, as the bits of a float.
template <int DT>
__device__ __forceinline__ uint32_t most8(u32x4 w) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    return __float_as_uint(DT == DT_F16 ? f16_bits_to_f32(m) : bf16_bits_to_f32(m));
}

template <int DT>
__device__ __forceinline__ u32x2 codes_of(u32x4 w, uint32_t byte) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = elem<DT>(w, i);
    return codes8(v, byte);
}

// UNROLL groups a team, TEAMS groups apart; groups are counted over all rows.
template <int DT, int UNROLL>
__global__ __launch_bounds__(THREADS) void quantize_kernel(const uint16_t* __restrict__ x, long long stride,
                                                           uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                           unsigned per_row, long long groups) {
    const int u = threadIdx.x % 16;
    const long long first = (long long)blockIdx.x * TEAMS * UNROLL + threadIdx.x / 16;
    u32x4 w[UNROLL];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
        const long long g = min(first + j * TEAMS, groups - 1);
        const long long row = g / per_row;
        w[j] = load_any(x + row * stride + (g - row * per_row) * 128 + 8 * u);
    }
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
        const long long g = first + j * TEAMS;
        const uint32_t byte = scale_byte(max16(most8<DT>(w[j])));
        if (g < groups) {
            *reinterpret_cast<u32x2*>(codes + g * 128 + 8 * u) = codes_of<DT>(w[j], byte);
            if (u == 0) scales[g] = (uint8_t)byte;
        }
    }
}

// A work-group takes a block of 128 rows by 128; a thread 8 rows of it, 16 apart.
template <int DT>
__global__ __launch_bounds__(THREADS) void quantize_block_kernel(const uint16_t* __restrict__ x, long long stride,
                                                                 uint8_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales, int rows, int width) {
    __shared__ uint32_t part[TEAMS];
    const int u = threadIdx.x % 16, team = threadIdx.x / 16;
    const int per_row = width / 128, at = (int)(blockIdx.x % per_row) * 128 + 8 * u;
    const long long top = (long long)(blockIdx.x / per_row) * 128;
    u32x4 w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = load_any(x + min(top + team + 16 * j, (long long)rows - 1) * stride + at);
    uint32_t most = 0;   // rows past the last repeat it
#pragma unroll
    for (int j = 0; j < 8; ++j) most = max(most, most8<DT>(w[j]));
    most = max16(most);
    if (u == 0) part[team] = most;
    __syncthreads();
    most = max16(part[u]);
    const uint32_t byte = scale_byte(most);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const long long row = top + team + 16 * j;
        if (row < rows) *reinterpret_cast<u32x2*>(codes + row * width + at) = codes_of<DT>(w[j], byte);
    }
    if (threadIdx.x == 0) scales[blockIdx.x] = (uint8_t)byte;
}

// c * s in float32, kept apart from what rounds it: the two as one instruction
// would round once where the definition does twice, and add a 0, which a -0 does
// not survive.
__device__ __forceinline__ float value_of(float c, float s) {
    float v = c * s;
    asm volatile("" : "+v"(v));
    return v;
}

// 8 lanes a group, 16 elements a lane.
template <int DT, bool F32, int UNROLL>
__global__ __launch_bounds__(THREADS) void dequantize_kernel(const uint8_t* __restrict__ codes,
                                                             const void* __restrict__ scales, uint16_t* __restrict__ out,
                                                             unsigned per_row, int block, long long groups) {
    const int u = threadIdx.x % 8;
    const long long first = (long long)blockIdx.x * (THREADS / 8) * UNROLL + threadIdx.x / 8;
    u32x4 w[UNROLL];
    float s[UNROLL];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
        const long long g = min(first + j * (THREADS / 8), groups - 1);
        w[j] = *reinterpret_cast<const u32x4*>(codes + g * 128 + 16 * u);
        long long at = g;
        if (block != 1) {
            const long long row = g / per_row;
            at = row / 128 * per_row + (g - row * per_row);
        }
        s[j] = F32 ? static_cast<const float*>(scales)[at] : scale_value(static_cast<const uint8_t*>(scales)[at]);
    }
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
        const long long g = first + j * (THREADS / 8);
        if (g >= groups) continue;
        u32x4 o[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j][i], false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j][i], true);
            o[i / 2][i % 2 * 2] = pack2<DT>(value_of(lo[0], s[j]), value_of(lo[1], s[j]));
            o[i / 2][i % 2 * 2 + 1] = pack2<DT>(value_of(hi[0], s[j]), value_of(hi[1], s[j]));
        }
        u32x4* to = reinterpret_cast<u32x4*>(out + g * 128 + 16 * u);
        to[0] = o[0];
        to[1] = o[1];
    }
}

template <int DT>
void quantize(const uint16_t* x, long long stride, uint8_t* codes, uint8_t* scales, int rows, int width, int block,
              hipStream_t st) {
    const unsigned per_row = (unsigned)width / 128;
    if (block == 1) {
        constexpr int U = 4;
        const long long groups = (long long)rows * per_row;
        hipLaunchKernelGGL((quantize_kernel<DT, U>), dim3((unsigned)((groups + TEAMS * U - 1) / (TEAMS * U))),
                           dim3(THREADS), 0, st, x, stride, codes, scales, per_row, groups);
    } else {
        hipLaunchKernelGGL((quantize_block_kernel<DT>), dim3((unsigned)(((long long)rows + 127) / 128 * per_row)),
                           dim3(THREADS), 0, st, x, stride, codes, scales, rows, width);
    }
}

template <int DT>
void dequantize(const uint8_t* codes, const void* scales, bool f32, uint16_t* out, int rows, int width, int block,
                hipStream_t st) {
    constexpr int U = 4;
    const unsigned per_row = (unsigned)width / 128;
    const long long groups = (long long)rows * per_row;
    const dim3 grid((unsigned)((groups + THREADS / 8 * U - 1) / (THREADS / 8 * U)));
    if (f32)
        hipLaunchKernelGGL((dequantize_kernel<DT, true, U>), grid, dim3(THREADS), 0, st, codes, scales, out, per_row,
                           block, groups);
    else
        hipLaunchKernelGGL((dequantize_kernel<DT, false, U>), grid, dim3(THREADS), 0, st, codes, scales, out, per_row,
                           block, groups);
}

}  // namespace

hipError_t launch_f8_quantize(const void* x, long long stride, uint8_t* codes, uint8_t* scales, int rows, int width,
                              int block, int dt, hipStream_t st) {
    const uint16_t* p = static_cast<const uint16_t*>(x);
    if (dt == DT_F16) quantize<DT_F16>(p, stride, codes, scales, rows, width, block, st);
    else quantize<DT_BF16>(p, stride, codes, scales, rows, width, block, st);
    return hipGetLastError();
}

hipError_t launch_f8_dequantize(const uint8_t* codes, const void* scales, bool f32, void* out, int rows, int width,
                                int block, int dt, hipStream_t st) {
    uint16_t* o = static_cast<uint16_t*>(out);
    if (dt == DT_F16) dequantize<DT_F16>(codes, scales, f32, o, rows, width, block, st);
    else dequantize<DT_BF16>(codes, scales, f32, o, rows, width, block, st);
    return hipGetLastError();
}

}  // namespace qmx
