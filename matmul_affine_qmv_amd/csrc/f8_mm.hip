// f8_mm.hip -- which kernel an 8-bit product takes, and how K is cut.
#include <algorithm>

#include "f8.h"
#include "qmx.h"
#include "qmx_internal.h"

namespace qmx {
namespace {

// K = 0: a sum over nothing.
__global__ void zero_kernel(uint16_t* out, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) out[i] = 0;
}

struct Kind {
    F8Tile tile;
    int rows, cols;
    double start, step;   // microseconds: of a launch, and of 128 of K
    double most;          // tiles that a launch can take (kernels that go on by themselves: any)
};
constexpr Kind KINDS[] = {{F8_32x64, 32, 64, 4.9, 0.168, 0x1p22},
                          {F8_64x64, 64, 64, 5.4, 0.216, 0x1p22},
                          {F8_64x128, 64, 128, 4.9, 0.329, 0x1p22},
                          {F8_128x128, 128, 128, 5.2, 0.452, 0x1p31},
                          {F8_256x256, 256, 256, 9.2, 1.12, 0x1p31}};

}  // namespace

// The least of estimates, in microseconds, fitted to 322 sizes (M 1 to 4096, N 512 to
// 28672, K 1024 to 27648; weights from memory): the pick is 0.6 % over the fastest of all
// kinds and cuts on the geometric mean, 25 % at worst (512 x 5120 over 14336).  Tiles go
// by rounds of the device, a step slower by up to a third the fuller it is; cutting K
// adds a launch, and float32 sums written and read.  Measured on both sides: 96 rows by
// 4096 over 4096, 9.4 us by 32 x 64 and 11.1 by 64 x 64; 192 rows 11.4 by 64 x 64 and
// 13.7 by 64 x 128; 384 rows 14.2 by 64 x 128 and 17.6 by 128 x 128; 2048 by 14336 over
// 5120, 168 by 128 x 128 and 130 by 256 x 256; 33 rows by 5120 over 14336, 28 whole and
// 21 in three parts; 16 by 2048 over 2048, 5.0 by rows of w and 6.9 by 32 x 64, by 14336
// over 5120, 23 and 19.
F8Plan f8_plan(int M, int N, int K, int cus) {
    const int groups = K / 128;
    const double bytes = (double)N * K;
    F8Plan best = {F8_256x256, 1};
    double least = 1e300;
    if (M <= 32) {   // x is read again for each 16 rows of w, from L2
        least = 3.7 + 2.3 * ((groups + 31) / 32) + bytes / 16e6 + M * (N / 16.0) * K / 9.7e6;
        best = {F8_ROWS, 1};
    }
    for (const Kind& k : KINDS) {
        const double tiles = (double)((M + k.rows - 1) / k.rows) * ((N + k.cols - 1) / k.cols);
        if (tiles > k.most) continue;
        for (int splits = 1; splits <= 8 && splits <= std::max(1, groups / 4); ++splits) {
            const double full = tiles * splits / cus;
            if (splits > 1 && full > 2) break;
            const double rounds = (double)(long long)(full + 0.999999);
            double t = k.start + std::max(rounds * ((groups + splits - 1) / splits) * k.step * (0.86 + 0.38 * std::min(1.0, full)),
                                          bytes / 7.8e6);
            if (splits > 1) t += 2.6 + (double)M * N * (8 * splits + 2) / 3.6e6;
            if (t < least) {
                least = t;
                best = {k.tile, splits};
            }
        }
    }
    return best;
}

hipError_t launch_qmm_f8(const F8MmArgs& a, F8Plan p, int cus, int dt, hipStream_t st) {
    if (a.K == 0) {
        const size_t n = (size_t)a.M * a.N;
        hipLaunchKernelGGL(zero_kernel, dim3((unsigned)std::min<size_t>((n + 255) / 256, 4096)), dim3(256), 0, st,
                           static_cast<uint16_t*>(a.out), n);
        return hipGetLastError();
    }
    if (dt == QMX_F16) a.w_f32 ? f8::launch_f16_f32(a, p, cus, st) : f8::launch_f16_e8m0(a, p, cus, st);
    else a.w_f32 ? f8::launch_bf16_f32(a, p, cus, st) : f8::launch_bf16_e8m0(a, p, cus, st);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.splits > 1)
        e = launch_splitk_accum(a.partials, a.out, p.splits, (size_t)a.M * a.N, dt, st);
    return e;
}

}  // namespace qmx
