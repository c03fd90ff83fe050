// kv_scan.h -- sums over a work-group, and a search in their result.
#pragma once

#include <hip/hip_runtime.h>

namespace qmx {

// a + b of numbers from 0 on, held to 2^31 - 1 (which keeps it associative).
__device__ __forceinline__ int add_held(int a, int b) {
    return (int)min((uint32_t)a + (uint32_t)b, 0x7fffffffu);
}

// Inclusive sums over a wave, held: in rows of 16 lanes, then from row to row.
__device__ __forceinline__ int scan_wave(int v) {
#define QMX_SCAN_STEP(CTRL, ROWS) v = add_held(v, __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false))
    QMX_SCAN_STEP(0x111, 0xf);   // from 1, 2, 4 and 8 lanes below in the row
    QMX_SCAN_STEP(0x112, 0xf);
    QMX_SCAN_STEP(0x114, 0xf);
    QMX_SCAN_STEP(0x118, 0xf);
    QMX_SCAN_STEP(0x142, 0xa);   // row 0's last lane to row 1, row 2's to row 3
    QMX_SCAN_STEP(0x143, 0xc);   // lane 31 to rows 2 and 3
#undef QMX_SCAN_STEP
    return v;
}

// Sums over the work-group's threads before this one, held, of N numbers at a
// time (a difference of held sums would not do); `total` is the sum of all.
// `waves`: N rows of WAVES in LDS.
template <int WAVES, int N>
__device__ __forceinline__ void scan_group(int (&v)[N], int (*waves)[WAVES], int (&total)[N]) {
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = scan_wave(v[i]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
        if ((threadIdx.x & 63) == 63) waves[i][wave] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        int before = 0;
        total[i] = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const int x = waves[i][w];
            before = w < wave ? add_held(before, x) : before;
            total[i] = add_held(total[i], x);
        }
        const int up = __shfl_up(v[i], 1, 64);
        v[i] = (threadIdx.x & 63) ? add_held(before, up) : before;
    }
}

// First index whose end is greater than x, of `count` ends in order.
__device__ __forceinline__ int first_after(const int* ends, int count, int x) {
    int lo = 0, hi = count;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] <= x) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

}  // namespace qmx
