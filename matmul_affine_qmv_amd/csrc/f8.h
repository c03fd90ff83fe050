// f8.h -- host-side launchers of the 8-bit float operators and of the rotary
// positions, shared between their kernels and the C ABI in f8_api.cpp.
// Arguments are validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qmx {

// Rows `stride` elements apart.
struct NormArgs {
    const void* x;
    const void* residual;   // NULL: none (then sum is NULL too)
    const void* weight;     // NULL: ones
    void* sum;
    void* out;
    uint8_t* scales;        // NULL: out in the inputs' type; else e4m3 codes and these
    long long x_stride, r_stride, s_stride;
    int rows, width;
    double eps;
};
hipError_t launch_rms_norm(const NormArgs& a, int dt, hipStream_t st);

// x [rows, width] in 16 bits to codes and scales, a scale for each 128 of `block` rows (1 or 128).
hipError_t launch_f8_quantize(const void* x, long long stride, uint8_t* codes, uint8_t* scales, int rows, int width,
                              int block, int dt, hipStream_t st);
// Codes back to values; scales as bytes or float32.
hipError_t launch_f8_dequantize(const uint8_t* codes, const void* scales, bool f32, void* out, int rows, int width,
                                int block, int dt, hipStream_t st);

struct RopeArgs {
    const void* in[2];      // queries, keys
    void* out[2];
    long long in_ts[2], in_hs[2], out_ts[2], out_hs[2];   // token and head strides in elements
    int heads[2];
    const int32_t* positions;
    const double* frequencies;
    int tokens, dim, pairs;
    float scale;
    bool interleaved;
    bool in_place[2];
};
hipError_t launch_rope(const RopeArgs& a, int dt, hipStream_t st);

// out [M, N] of codes w [N, K] and x [M, K]: by rows of w straight from memory (M up
// to 32), or by tiles of so many rows of x by so many of w.
enum F8Tile { F8_ROWS, F8_32x64, F8_64x64, F8_64x128, F8_128x128, F8_256x256 };
struct F8Plan {
    F8Tile tile;
    int splits;   // partitions of K, each to its own float32 partials (1: none)
};
struct F8MmArgs {
    const uint8_t* w;
    const void* w_scales;
    bool w_f32;
    const uint8_t* x;
    const uint8_t* x_scales;
    void* out;
    float* partials;
    int M, N, K;
};
F8Plan f8_plan(int M, int N, int K, int cus);
hipError_t launch_qmm_f8(const F8MmArgs& a, F8Plan p, int cus, int dt, hipStream_t st);
namespace f8 {
// One for each type of out and of w's scales, in files of their own.
void launch_bf16_e8m0(const F8MmArgs& a, F8Plan p, int cus, hipStream_t st);
void launch_bf16_f32(const F8MmArgs& a, F8Plan p, int cus, hipStream_t st);
void launch_f16_e8m0(const F8MmArgs& a, F8Plan p, int cus, hipStream_t st);
void launch_f16_f32(const F8MmArgs& a, F8Plan p, int cus, hipStream_t st);
}  // namespace f8

}  // namespace qmx
