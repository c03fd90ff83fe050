// kv_scan.h -- sums over a work-group, and a search in their result.
#pragma once

#include <hip/hip_runtime.h>

namespace qmx {

template <class T>
__device__ __forceinline__ T scan_wave(T v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const T up = __shfl_up(v, off, 64);
        if (lane >= off) v += up;
    }
    return v;
}

// Inclusive sum over the work-group's threads; `total` is the sum of all.
template <int WAVES, class T>
__device__ __forceinline__ T scan_group(T v, T* waves, T& total) {
    v = scan_wave(v);
    const int wave = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 63) waves[wave] = v;
    __syncthreads();
    T before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const T x = waves[w];
        before += w < wave ? x : 0;
        total += x;
    }
    return v + before;
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
