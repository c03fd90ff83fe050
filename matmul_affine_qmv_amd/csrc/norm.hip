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
// stands for does, for all eight: magnitudes of 2^-60 to 2^100, none within three
// of a number of five digits, as middles between codes are.  (w below 2^60 then
// leaves h * rstd a normal number.)
template <int DT>
__device__ __forceinline__ bool clear_of_middles(const float (&y)[8], u32x4 w) {
    uint32_t least = 0xffffffffu, most = 0, near = 0xffffffffu, heavy = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(y[i]) & 0x7fffffffu;
        least = min(least, u);
        most = max(most, u);
        near = min(near, (u + 3u) & 0x7ffffu);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) heavy = max(heavy, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    return least >= (127u - 60u) << 23 && most <= (127u + 100u) << 23 && near > 6u &&
           (DT == DT_F16 || heavy < (127u + 60u) << 7);
}

// y of eight elements from element `at` on, and where they go.
template <int DT, bool F8>
__device__ __forceinline__ void finish8(const NormArgs& a, size_t row, int at, int n, u32x4 h, const Rstd& r) {
    const uint32_t one = DT == DT_F16 ? 0x3c003c00u : 0x3f803f80u;
    u32x4 w = {one, one, one, one};
    if (a.weight) w = load_part(static_cast<const uint16_t*>(a.weight) + at, n);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = elem<DT>(h, i) * r.rounded * elem<DT>(w, i);
    const bool again = !r.ordinary || (F8 && n > 0 && !clear_of_middles<DT>(y, w));
    if (again) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = to_odd((double)elem<DT>(h, i) * r.whole * (double)elem<DT>(w, i));
    }
    const size_t to = row * a.width + at;
    if constexpr (F8) {   // 16 lanes hold a group
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(y[i]) & 0x7fffffffu);
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

// One row for each wave (WAVE) or for the whole work-group, whose lanes hold up to
// VPT * 8 of its elements each.
template <int DT, bool F8, bool PASS, bool WAVE, int VPT>
__global__ __launch_bounds__(WAVE ? 256 : VPT == 1 ? 1024 : 512) void norm_kernel(NormArgs a) {
    __shared__ double part[16];
    const int lanes = WAVE ? 64 : blockDim.x, lane = WAVE ? threadIdx.x % 64 : threadIdx.x;
    const size_t row = WAVE ? (size_t)blockIdx.x * 4 + threadIdx.x / 64 : blockIdx.x;
    if (WAVE && row >= (size_t)a.rows) return;
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * a.x_stride;
    u32x4 h[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int at = (j * lanes + lane) * 8;
        h[j] = load_part(x + at, a.width - at);
    }
    if (a.residual) {
        const uint16_t* r = static_cast<const uint16_t*>(a.residual) + row * a.r_stride;
        uint16_t* s = static_cast<uint16_t*>(a.sum) + row * a.s_stride;
        u32x4 v[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int at = (j * lanes + lane) * 8;
            v[j] = load_part(r + at, a.width - at);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int at = (j * lanes + lane) * 8;
            h[j] = add8<DT>(h[j], v[j]);
            store_part<PASS>(s + at, h[j], a.width - at);
        }
    }
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) sum = squares8<DT>(h[j], sum);
    sum = wave_sum64(sum);
    if (!WAVE) {
        if (lane % 64 == 0) part[lane / 64] = sum;
        __syncthreads();
        sum = 0.0;
        for (int i = 0; i < lanes / 64; ++i) sum += part[i];
    }
    const Rstd r = rstd_of(sum, a.width, a.eps);
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
        u32x4 h = load_part(x + at, n);
        if (a.residual) {
            h = add8<DT>(h, load_part(r + at, n));
            store_part<false>(s + at, h, n);
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
        finish8<DT, F8>(a, row, (int)min(at, (long long)a.width), n, load_part(from + at, n), scale);
    }
}

template <int DT, bool F8, bool PASS, bool WAVE, int VPT>
void go(const NormArgs& a, int lanes, hipStream_t st) {
    hipLaunchKernelGGL((norm_kernel<DT, F8, PASS, WAVE, VPT>), dim3(WAVE ? ((unsigned)a.rows + 3) / 4 : (unsigned)a.rows),
                       dim3((unsigned)lanes), 0, st, a);
}

constexpr int MOST_ROWS = 1 << 21;   // of a launch, whose grid has below 2^32 threads

// Lanes and elements of a row (for rows of 5120 into 8 bits, 7812 of them: 66.5 us with
// 256 lanes of 24, 71.5 with 320 of 16, 70.7 with 640 of 8; 8192 wide 66.6 with 512 of
// 16, 74.1 with 256 of 32; 1024 wide 61.7 with a wave a row, 88 with four).  Few rows
// take as many lanes as they have eights (1 of 5120: 3.7 us, 5.9 with 256 lanes).
template <int DT, bool F8, bool PASS>
void pick(const NormArgs& a, hipStream_t st) {
    const int eights = (int)(((long long)a.width + 7) / 8);
    if (eights <= 64) go<DT, F8, PASS, true, 1>(a, 256, st);
    else if (a.rows < 256 && eights <= 1024) go<DT, F8, PASS, false, 1>(a, (eights + 63) / 64 * 64, st);
    else if (eights <= 128) go<DT, F8, PASS, true, 2>(a, 256, st);
    else if (eights <= 256) go<DT, F8, PASS, false, 2>(a, 128, st);
    else if (eights <= 512) go<DT, F8, PASS, false, 2>(a, 256, st);
    else if (eights <= 768) go<DT, F8, PASS, false, 3>(a, 256, st);
    else if (eights <= 1024) go<DT, F8, PASS, false, 2>(a, 512, st);
    else if (eights <= 1536) go<DT, F8, PASS, false, 3>(a, 512, st);
    else if (eights <= 2048) go<DT, F8, PASS, false, 4>(a, 512, st);
    else hipLaunchKernelGGL((norm_long_kernel<DT, F8>), dim3((unsigned)a.rows), dim3(1024), 0, st, a);
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
