// norm.hip -- root mean square norm of rows, after the residual's addition, into
// the rows' type or into 8-bit floats with a scale for each 128:
//   h = round(x + residual),  y = h * w / sqrt(sum h^2 / width + eps).
//
// Bound by memory: x, residual and w are read once and h and y written once, the
// row staying in registers between its sum and its use.  The sum of squares is
// formed in 64 bits, so neither large nor tiny rows leave the range on the way.  y
// is two products in 32 bits, and its codes are those of 64 bits all the same: a
// lane whose eight y's are not all clear of the middles between two codes forms
// them again in 64 bits (one wave in 100 does on random numbers).
//
// 8192 rows of 5120 in bfloat16 with a residual into 8 bits: 59 us, 4.9 TB/s, a large
// copy's rate; 2500 of 4097 in float16 11 us, 3.7 TB/s, all rows being read before the
// first is written; one row of 5120 3.7 us, a launch and two ways to memory.
#include <algorithm>

#include "f8.h"
#include "f8_device.h"

namespace qmx {
namespace {

// A float that every rounding to fewer than 23 bits takes where it would take y:
// y cut to 24 bits, the last of them set if anything was cut off.
__device__ __forceinline__ float to_odd(double y) {
    const float f = (float)y;
    const uint32_t u = __float_as_uint(f);
    const double back = (double)f;
    const bool cut = back != y && !(u & 1u) && (u & 0x7fffffffu) < 0x7f800000u;
    return __uint_as_float(cut ? (fabs(back) < fabs(y) ? u + 1u : u - 1u) : u);
}

// What a row is multiplied by, in 64 and in 32 bits.
struct Rstd {
    double whole;
    float rounded;
    bool ordinary;   // rounded is far from the ends of its range
};

__device__ __forceinline__ Rstd rstd_of(double sum, int width, double eps) {
    Rstd r;
    r.whole = 1.0 / sqrt(sum / width + eps);
    r.rounded = (float)r.whole;
    r.ordinary = r.rounded >= 0x1p-100f && r.rounded <= 0x1p100f;
    return r;
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

template <int DT>
__device__ __forceinline__ u32x4 add8(u32x4 x, u32x4 r) {
    // two roundings, to 32 bits and to the type, give what one gives: 24 >= 2 * 11 + 2
    u32x4 h;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = pack2<DT>(half_lo<DT>(x[i]) + half_lo<DT>(r[i]), half_hi<DT>(x[i]) + half_hi<DT>(r[i]));
    return h;
}

template <int DT>
__device__ __forceinline__ double squares8(u32x4 h, double sum) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const double v = (double)elem<DT>(h, i);
        sum = fma(v, v, sum);
    }
    return sum;
}

// Whether y, off by at most three of its last digits (three roundings of half a
// digit, of a number up to twice its power of two), rounds to a code as what it
// stands for does, for all eight: magnitudes of 2^-60 to 2^100 (`most` the largest),
// none within three of a number of five digits, as middles between codes are (w below
// 2^60 then leaves h * rstd a normal number); or all 0 because h is, as in padding.
template <int DT>
__device__ __forceinline__ bool clear_of_middles(const float (&y)[8], u32x4 h, u32x4 w, uint32_t most) {
    uint32_t least = 0xffffffffu, near = 0xffffffffu, heavy = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(y[i]);
        least = min(least, u & 0x7fffffffu);
        near = min(near, (u + 3u) & 0x7ffffu);
    }
    if constexpr (DT == DT_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) heavy = max(heavy, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    }
    const bool clear = least >= (127u - 60u) << 23 && most <= (127u + 100u) << 23 && near > 6u;
    const bool none = ((h[0] | h[1] | h[2] | h[3]) & 0x7fff7fffu) == 0 && most == 0;
    return (clear && heavy < (127u + 60u) << 7) || none;
}

__device__ __forceinline__ uint32_t most_of(const float (&y)[8]) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(y[i]) & 0x7fffffffu);
    return most;
}

// Eight elements of a row of which `n` are left.  Into 8 bits rows are whole groups.
template <bool F8>
__device__ __forceinline__ u32x4 load8(const uint16_t* p, int n) {
    if constexpr (F8) return n > 0 ? load_any(p) : u32x4{0, 0, 0, 0};
    else return load_part(p, n);
}
template <bool F8, bool PASS>
__device__ __forceinline__ void store8(uint16_t* p, u32x4 v, int n) {
    if constexpr (F8) {
        if (n > 0) store_any<PASS>(p, v);
    } else {
        store_part<PASS>(p, v, n);
    }
}

// y of eight elements from element `at` on, and where they go.
template <int DT, bool F8>
__device__ __forceinline__ void finish8(const NormArgs& a, size_t row, int at, int n, u32x4 h, const Rstd& r) {
    const uint32_t one = DT == DT_F16 ? 0x3c003c00u : 0x3f803f80u;
    u32x4 w = {one, one, one, one};
    if (a.weight) w = load8<F8>(static_cast<const uint16_t*>(a.weight) + at, n);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = elem<DT>(h, i) * r.rounded * elem<DT>(w, i);
    uint32_t most = F8 ? most_of(y) : 0;
    if (!r.ordinary || (F8 && n > 0 && !clear_of_middles<DT>(y, h, w, most))) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = to_odd((double)elem<DT>(h, i) * r.whole * (double)elem<DT>(w, i));
        if (F8) most = most_of(y);
    }
    const size_t to = row * a.width + at;
    if constexpr (F8) {   // 16 lanes hold a group
        const uint32_t byte = scale_byte(max16(most));
        if (n > 0) {
            *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.out) + to) = codes8(y, byte);
            if (at % 128 == 0) a.scales[to / 128] = (uint8_t)byte;
        }
    } else {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack2<DT>(y[2 * i], y[2 * i + 1]);
        store_part<false>(static_cast<uint16_t*>(a.out) + to, o, n);
    }
}

// A row for each work-group, whose lanes hold up to VPT * 8 of its elements each.
template <int DT, bool F8, bool PASS, int VPT>
__global__ __launch_bounds__(VPT == 1 ? 1024 : 512) void norm_kernel(NormArgs a) {
    __shared__ double part[16];
    const int lanes = blockDim.x, lane = threadIdx.x;
    const size_t row = blockIdx.x;
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * a.x_stride;
    u32x4 h[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int at = (j * lanes + lane) * 8;
        h[j] = load8<F8>(x + at, a.width - at);
    }
    if (a.residual) {
        const uint16_t* r = static_cast<const uint16_t*>(a.residual) + row * a.r_stride;
        uint16_t* s = static_cast<uint16_t*>(a.sum) + row * a.s_stride;
        u32x4 v[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int at = (j * lanes + lane) * 8;
            v[j] = load8<F8>(r + at, a.width - at);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int at = (j * lanes + lane) * 8;
            h[j] = add8<DT>(h[j], v[j]);
            store8<F8, PASS>(s + at, h[j], a.width - at);
        }
    }
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) sum = squares8<DT>(h[j], sum);
    sum = wave_sum64(sum);
    if (lanes > 64) {
        if (lane % 64 == 0) part[lane / 64] = sum;
        __syncthreads();
        sum = 0.0;
        for (int i = 0; i < lanes / 64; ++i) sum += part[i];
    }
    const Rstd r = rstd_of(sum, a.width, a.eps);
    // What the elements are as floats and doubles is formed anew: kept from the sum it
    // would take three to six times the registers.
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(h[j][i]));
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int at = (j * lanes + lane) * 8;
        if (F8 || at < a.width) finish8<DT, F8>(a, row, at, a.width - at, h[j], r);
    }
}

// Rows of any length, read a second time: from the sum, if there is one.  Each
// thread reads again only what it has itself read or written.
template <int DT, bool F8>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormArgs a) {
    __shared__ double part[16];
    const size_t row = blockIdx.x;
    const int lane = threadIdx.x;
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * a.x_stride;
    const uint16_t* r = static_cast<const uint16_t*>(a.residual) + row * a.r_stride;
    uint16_t* s = static_cast<uint16_t*>(a.sum) + row * a.s_stride;
    double sum = 0.0;
    for (long long at = lane * 8; at < a.width; at += 1024 * 8) {
        const int n = (int)min(8ll, a.width - at);
        u32x4 h = load8<F8>(x + at, n);
        if (a.residual) {
            h = add8<DT>(h, load8<F8>(r + at, n));
            store8<F8, false>(s + at, h, n);
        }
        sum = squares8<DT>(h, sum);
    }
    sum = wave_sum64(sum);
    if (lane % 64 == 0) part[lane / 64] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += part[i];
    const Rstd scale = rstd_of(sum, a.width, a.eps);
    const uint16_t* from = a.residual ? s : x;
    const long long end = F8 ? ((long long)a.width + 8191) / 8192 * 8192 : (long long)a.width;
    for (long long at = lane * 8; at < end; at += 1024 * 8) {
        const int n = (int)max(0ll, min(8ll, a.width - at));
        finish8<DT, F8>(a, row, (int)min(at, (long long)a.width), n, load8<F8>(from + at, n), scale);
    }
}

constexpr int MOST_ROWS = 1 << 21;   // of a launch, whose grid has below 2^32 threads

template <int DT, bool F8, bool PASS, int VPT>
void go(const NormArgs& a, int waves, hipStream_t st) {
    hipLaunchKernelGGL((norm_kernel<DT, F8, PASS, VPT>), dim3((unsigned)a.rows), dim3((unsigned)waves * 64), 0, st, a);
}

// A lane takes as many eights of a row as leave the device full of waves: one while all
// the rows' waves are at most half of what it holds (1024 rows of 2048 into 8 bits: 5.1
// us, two 5.2, four 5.8), two while they are at most all (1024 rows of 5120: 8.3, one
// 9.7, four 8.7), then up to four, so that few waves meet for a row's sum and each has
// more on its way (8192 rows of 5120: 33.7 us, 37.6 with two and 55.7 with one; of 8192
// 44.8, 50.4 and 69.9), and no more than fill its waves (2500 rows of 4104 into 16 bits
// 12.1 with three, 12.4 with four).
template <int DT, bool F8, bool PASS>
void pick(const NormArgs& a, hipStream_t st) {
    const int eights = (int)(((long long)a.width + 7) / 8);
    if (eights > 2048) {
        hipLaunchKernelGGL((norm_long_kernel<DT, F8>), dim3((unsigned)a.rows), dim3(1024), 0, st, a);
        return;
    }
    const int one = (eights + 63) / 64, two = (eights + 127) / 128;
    const int waves = one <= 16 && (long long)a.rows * one <= 4096 ? one
                      : (long long)a.rows * two <= 8192            ? std::min(two, 8)
                                                                   : (eights + 255) / 256;
    switch ((eights + 64 * waves - 1) / (64 * waves)) {
        case 1: go<DT, F8, PASS, 1>(a, waves, st); break;
        case 2: go<DT, F8, PASS, 2>(a, waves, st); break;
        case 3: go<DT, F8, PASS, 3>(a, waves, st); break;
        default: go<DT, F8, PASS, 4>(a, waves, st); break;
    }
}

}  // namespace

// The sum is read again only a layer's products later: large ones go past the caches,
// which keep the result for what comes next.
hipError_t launch_rms_norm(const NormArgs& all, int dt, hipStream_t st) {
    const bool f8 = all.scales != nullptr, pass = all.sum && (long long)all.rows * all.width >= (4ll << 20);
    NormArgs a = all;
    a.rows = std::min(all.rows, MOST_ROWS);
    if (dt == DT_F16) {
        if (pass) f8 ? pick<DT_F16, true, true>(a, st) : pick<DT_F16, false, true>(a, st);
        else f8 ? pick<DT_F16, true, false>(a, st) : pick<DT_F16, false, false>(a, st);
    } else {
        if (pass) f8 ? pick<DT_BF16, true, true>(a, st) : pick<DT_BF16, false, true>(a, st);
        else f8 ? pick<DT_BF16, true, false>(a, st) : pick<DT_BF16, false, false>(a, st);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.rows == all.rows) return e;
    const auto behind = [](const void* p, long long bytes) {
        return p ? const_cast<char*>(static_cast<const char*>(p)) + bytes : nullptr;
    };
    const long long n = a.rows;
    return launch_rms_norm({behind(a.x, 2 * n * a.x_stride), behind(a.residual, 2 * n * a.r_stride), a.weight,
                            behind(a.sum, 2 * n * a.s_stride), behind(a.out, n * a.width * (f8 ? 1 : 2)),
                            f8 ? a.scales + n * (a.width / 128) : nullptr, a.x_stride, a.r_stride, a.s_stride,
                            all.rows - a.rows, a.width, a.eps},
                           dt, st);
}

}  // namespace qmx
