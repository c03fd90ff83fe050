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
    double start, one, two;   // microseconds: of a launch, and of 128 of K with one and two work-groups a compute unit
    double most;              // tiles that a launch can take (kernels that go on by themselves: any)
};
constexpr Kind KINDS[] = {{F8_32x64, 32, 64, 4.4, 0.172, 0.327, 0x1p23},
                          {F8_64x64, 64, 64, 4.6, 0.189, 0.455, 0x1p23},
                          {F8_64x128, 64, 128, 5.0, 0.352, 0.576, 0x1p23},
                          {F8_128x128, 128, 128, 5.8, 0.493, 0.767, 0x1p31},
                          {F8_256x256, 256, 256, 10.0, 1.00, 2.00, 0x1p31}};   // one at a time

}  // namespace

// The least of estimates, in microseconds, fitted to 322 sizes (M 1 to 4096, N 512 to
// 28672, K 1024 to 27648; weights from memory): the pick is 0.4 % over the fastest of all
// kinds and cuts on the geometric mean, 13 % at worst (32 x 512 over 4096).  Tiles go by
// rounds of two a compute unit, or one; cutting K adds a launch, and float32 sums written
// and read.  Measured on both sides: 96 rows by 4096 over 4096, 9.3 us by 32 x 64 and
// 10.3 by 64 x 64; 192 rows 10.5 by 64 x 64 and 12.5 by 32 x 64; 384 rows 14.5 by 64 x 128
// and 15.6 by 64 x 64; 640 rows 18.1 by 128 x 128 and 22.1 by 64 x 128; 2048 by 14336 over
// 5120, 167 by 128 x 128 and 130 by 256 x 256; 33 rows by 5120 over 14336, 24 in two parts
// and 21 in three; 16 by 2048 over 2048, 5.0 by rows of w and 6.6 by 32 x 64, by 14336
// over 5120, 23 and 18.
F8Plan f8_plan(int M, int N, int K, int cus) {
    const int groups = K / 128;
    const double bytes = (double)N * K;
    F8Plan best = {F8_256x256, 1};
    double least = 1e300;
    if (M <= 32) {   // x is read again for each 16 rows of w, from L2
        least = 3.4 + 2.5 * ((groups + 31) / 32) + bytes / 26e6 + M * (N / 16.0) * K / 5.0e6;
        best = {F8_ROWS, 1};
    }
    for (const Kind& k : KINDS) {
        const double tiles = (double)((M + k.rows - 1) / k.rows) * ((N + k.cols - 1) / k.cols);
        if (tiles > k.most) continue;
        for (int splits = 1; splits <= 8 && splits <= std::max(1, groups / 4); ++splits) {
            const long long each = (long long)((tiles * splits + cus - 1) / cus);   // of the fullest compute unit
            if (splits > 1 && each > 2) break;
            const int part = (groups + splits - 1) / splits;
            double t = k.start + std::max(part * (each / 2 * k.two + each % 2 * k.one), bytes / 8.1e6);
            if (splits > 1) t += 3.2 + (double)M * N * (8 * splits + 2) / 7.1e6;
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
