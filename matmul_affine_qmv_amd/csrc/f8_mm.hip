// f8_mm.hip -- launches of the 8-bit products, and the rule that picks a kernel.
#include "f8_mm_impl.h"

#include <algorithm>

#include "qmx_internal.h"

namespace qmx {
namespace {

template <int DT, bool F32, int MT, int NT, int WAVES>
void rows(const F8MmArgs& a, hipStream_t st) {
    hipLaunchKernelGGL((f8::rows_kernel<DT, F32, MT, NT, WAVES>), dim3((unsigned)((a.N + 16 * NT - 1) / (16 * NT))),
                       dim3(WAVES * 64), 0, st, a);
}

template <int DT, bool F32, int BM, int BN, int WM, int WN, int STAGES>
void tiles(const F8MmArgs& a, int splits, hipStream_t st) {
    const long long n = (long long)((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN) * splits;
    const unsigned grid = f8::tile_groups(n, f8::tile_fit<BM, BN, STAGES>() * device_cu_count());
    if (splits > 1)
        hipLaunchKernelGGL((f8::tile_kernel<DT, F32, BM, BN, WM, WN, STAGES, true>), dim3(grid), dim3(WM * WN * 64), 0, st, a, splits);
    else
        hipLaunchKernelGGL((f8::tile_kernel<DT, F32, BM, BN, WM, WN, STAGES, false>), dim3(grid), dim3(WM * WN * 64), 0, st, a, 1);
}

// K = 0: a sum over nothing.
__global__ void zero_kernel(uint16_t* out, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) out[i] = 0;
}

template <int DT, bool F32>
void pick(const F8MmArgs& a, F8Plan p, hipStream_t st) {
    switch (p.tile) {
        case 0:
            if (a.M <= 16) rows<DT, F32, 1, 1, 8>(a, st);
            else if (a.M <= 32) rows<DT, F32, 2, 2, 8>(a, st);
            else if (a.M <= 48) rows<DT, F32, 3, 2, 8>(a, st);
            else rows<DT, F32, 4, 2, 8>(a, st);
            break;
        case 1: tiles<DT, F32, 128, 128, 2, 2, 4>(a, p.splits, st); break;
        default: tiles<DT, F32, 256, 256, 2, 4, 2>(a, p.splits, st); break;
    }
}

}  // namespace

F8Plan f8_plan(int M, int N, int K, int cus) {
    if (M <= 64) return {0, 1};
    const long long big = (long long)((M + 255) / 256) * ((N + 255) / 256);
    if (big >= cus) return {2, 1};
    const long long small = (long long)((M + 127) / 128) * ((N + 127) / 128);
    const int splits = (int)std::max(1ll, std::min<long long>({cus / std::max(1ll, small), K / 512, 8}));
    return {1, splits};
}

hipError_t launch_qmm_f8(const F8MmArgs& a, F8Plan p, int dt, hipStream_t st) {
    if (a.K == 0) {
        const size_t n = (size_t)a.M * a.N;
        hipLaunchKernelGGL(zero_kernel, dim3((unsigned)std::min<size_t>((n + 255) / 256, 4096)), dim3(256), 0, st,
                           static_cast<uint16_t*>(a.out), n);
        return hipGetLastError();
    }
    if (dt == DT_F16) a.w_f32 ? pick<DT_F16, true>(a, p, st) : pick<DT_F16, false>(a, p, st);
    else a.w_f32 ? pick<DT_BF16, true>(a, p, st) : pick<DT_BF16, false>(a, p, st);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.splits > 1)
        e = launch_splitk_accum(a.partials, a.out, p.splits, (size_t)a.M * a.N, dt, st);
    return e;
}

}  // namespace qmx
