// f8_api.cpp -- the C ABI of the 8-bit float operators, the norm before them and
// the rotary positions: host-side validation and the launches.  Every check runs
// before any launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <utility>

#include "f8.h"
#include "qmx.h"
#include "qmx_internal.h"

namespace {

bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int launch_status(hipError_t e) { return e == hipSuccess ? QMX_OK : QMX_ERR_LAUNCH; }

bool is_half(int dtype) { return dtype == QMX_F16 || dtype == QMX_BF16; }

// Rows of codes in groups of 128: what quantize and dequantize share.
int check_codes(int rows, int width, int block_rows, int dtype) {
    if (!is_half(dtype)) return QMX_ERR_DTYPE;
    if (rows < 0 || width < 0) return QMX_ERR_SHAPE;
    if (width % 128 || (block_rows != 1 && block_rows != 128)) return QMX_ERR_GROUP;
    if ((long long)rows * (width / 128) > (1 << 29)) return QMX_ERR_SHAPE;   // below 2^32 threads
    return QMX_OK;
}

// Whether rows of `n` neighbours, `count` of them `stride` apart, `sets` times
// `set_stride` apart, share no element.
bool apart(long long n, long long count, long long stride, long long sets, long long set_stride) {
    stride = std::llabs(stride);
    set_stride = std::llabs(set_stride);
    if (count <= 1) stride = 0;
    if (sets <= 1) set_stride = 0;
    if (stride > set_stride) {
        std::swap(stride, set_stride);
        std::swap(count, sets);
    }
    const __int128 span = (__int128)std::max(0ll, count - 1) * stride + n;
    return (count <= 1 || stride >= n) && (sets <= 1 || set_stride >= span);
}

typedef __int128 wide;   // of addresses and strides: rows may be any distance apart

// Where an argument's bytes are: `rows` runs of n elements, `sets` times.
struct Area {
    const void* p;
    int size;   // of an element
    long long n, rows, stride, sets, set_stride;
    long long lo, hi;   // its first byte and the one behind its last,
    bool beyond;        // unless 64 bits do not hold that
};
Area area(const void* p, int size, long long n, long long rows = 1, long long stride = 0, long long sets = 1,
          long long set_stride = 0) {
    Area a = {p, size, n, rows, stride, sets, set_stride};
    long long row, set, bytes;
    a.beyond = __builtin_mul_overflow((rows - 1) * size, stride, &row) |
               __builtin_mul_overflow((sets - 1) * size, set_stride, &set) |
               __builtin_mul_overflow(n, (long long)size, &bytes);
    a.lo = a.hi = (long long)reinterpret_cast<uintptr_t>(p);
    a.beyond |= row < 0 ? __builtin_add_overflow(a.lo, row, &a.lo) : __builtin_add_overflow(a.hi, row, &a.hi);
    a.beyond |= set < 0 ? __builtin_add_overflow(a.lo, set, &a.lo) : __builtin_add_overflow(a.hi, set, &a.hi);
    a.beyond |= __builtin_add_overflow(a.hi, bytes, &a.hi);
    return a;
}

// The same as runs of n bytes, counted and apart by an outer and an inner step.
struct Runs {
    wide at, n, count[2], step[2];   // steps not below 0

    explicit Runs(const Area& a)
        : at((wide)reinterpret_cast<uintptr_t>(a.p)), n((wide)a.n * a.size), count{a.sets, a.rows},
          step{(wide)a.set_stride * a.size, (wide)a.stride * a.size} {
        for (int i = 0; i < 2; ++i) {
            if (count[i] == 1) step[i] = 0;
            if (step[i] < 0) {
                at += (count[i] - 1) * step[i];
                step[i] = -step[i];
            }
            if (step[i] == 0) count[i] = 1;   // the same run again
        }
        if (step[0] < step[1]) {
            std::swap(step[0], step[1]);
            std::swap(count[0], count[1]);
        }
    }
    wide span(int level) const { return level == 2 ? n : span(level + 1) + (count[level] - 1) * step[level]; }
};

wide floor_div(wide a, wide b) { return a / b - (a % b < 0 ? 1 : 0); }   // b above 0

// Whether x, from level i of its steps on, and y, from level j on, share a byte.
// Looks at up to `left` pairs of runs: two areas that are laid into one another with
// different steps more often than that without a byte in common count as apart.
bool share(Runs x, int i, const Runs& y, int j, int& left) {
    if (--left < 0 || x.at + x.span(i) <= y.at || y.at + y.span(j) <= x.at) return false;
    while (i < 2 && x.count[i] == 1) ++i;
    while (j < 2 && y.count[j] == 1) ++j;
    if (i == 2 && j == 2) return true;
    if (i == 2 || (j < 2 && y.step[j] > x.step[i])) return share(y, j, x, i, left);
    // x's outer step is the larger.  Where y's is the same, how many steps they are
    // apart is all that matters.
    const bool both = j < 2 && x.step[i] == y.step[j];
    const wide step = x.step[i], x_span = x.span(i + 1), y_span = y.span(both ? j + 1 : j);
    const wide first = std::max(both ? 1 - y.count[j] : (wide)0, floor_div(y.at - x.at - x_span, step) + 1);
    const wide last = std::min(x.count[i] - 1, floor_div(y.at + y_span - x.at - 1, step));
    const wide from = x.at;
    for (wide k = first; k <= last && left > 0; ++k) {
        x.at = from + k * step;
        if (share(x, i + 1, y, both ? j + 1 : j, left)) return true;
    }
    return false;
}
bool share(const Area& x, const Area& y) {
    if (!x.beyond && !y.beyond && (x.hi <= y.lo || y.hi <= x.lo)) return false;
    int left = 4096;
    return share(Runs(x), 0, Runs(y), 0, left);
}

int units() {
    const int cus = qmx::device_cu_count();
    return cus > 0 ? cus : 256;
}

int check_product(int M, int N, int K) {
    // 256 rows of K bytes, and 16 rows of N floats, in 32 bits; every kernel's grid
    if (M < 0 || N < 0 || K < 0 || K >= (1 << 24) || N > (1 << 25) || M > (1 << 30)) return QMX_ERR_SHAPE;
    if ((M + 15ll) / 16 * ((N + 15ll) / 16) > INT_MAX / 8) return QMX_ERR_SHAPE;
    if (K % 128) return QMX_ERR_GROUP;
    return QMX_OK;
}

}  // namespace

extern "C" {

int qmx_rms_norm(const void* x, long long x_row_stride, const void* residual, long long residual_row_stride,
                 const void* weight, void* sum, long long sum_row_stride, void* out, uint8_t* out_scales, int rows,
                 int width, double eps, int dtype, void* stream) {
    if (!is_half(dtype)) return QMX_ERR_DTYPE;
    if (rows < 0 || width < 0) return QMX_ERR_SHAPE;
    if (!std::isfinite(eps) || eps <= 0.0) return QMX_ERR_SHAPE;
    if (out_scales && width % 128) return QMX_ERR_GROUP;
    if (rows == 0 || width == 0) return QMX_OK;
    if (!x || !out || (residual != nullptr) != (sum != nullptr)) return QMX_ERR_NULL;
    if (!is_aligned(x, 2) || !is_aligned(residual, 2) || !is_aligned(weight, 2) || !is_aligned(sum, 2) ||
        !is_aligned(out, out_scales ? 8 : 2))
        return QMX_ERR_ALIGN;
    if (sum && !apart(width, rows, sum_row_stride, 1, 0)) return QMX_ERR_OVERLAP;
    const Area in[3] = {area(x, 2, width, rows, x_row_stride), area(residual, 2, width, rows, residual_row_stride),
                        area(weight, 2, width)};
    const long long in_strides[2] = {x_row_stride, residual_row_stride};
    const Area to[3] = {area(sum, 2, width, rows, sum_row_stride),
                        area(out, out_scales ? 1 : 2, (long long)rows * width),
                        area(out_scales, 1, (long long)rows * (width / 128))};
    const long long to_strides[2] = {sum_row_stride, width};
    const void *from[3] = {x, residual, weight}, *into[3] = {sum, out, out_scales};
    for (int i = 0; i < 3; ++i) {
        if (!into[i]) continue;
        for (int j = 0; j < 3; ++j) {
            // rows over their own: each work-group reads a row before it writes it
            const bool own = j < 2 && (i == 0 || (i == 1 && !out_scales)) && into[i] == from[j] &&
                             (rows == 1 || to_strides[i] == in_strides[j]);
            if (from[j] && !own && share(to[i], in[j])) return QMX_ERR_OVERLAP;
            if (j < i && into[j] && share(to[i], to[j])) return QMX_ERR_OVERLAP;
        }
    }
    const qmx::NormArgs a = {x, residual, weight, sum, out, out_scales, x_row_stride, residual_row_stride,
                             sum_row_stride, rows, width, eps};
    return launch_status(qmx::launch_rms_norm(a, dtype, static_cast<hipStream_t>(stream)));
}

int qmx_f8_quantize(const void* x, long long x_row_stride, uint8_t* codes, uint8_t* scales, int rows, int width,
                    int block_rows, int dtype, void* stream) {
    const int rc = check_codes(rows, width, block_rows, dtype);
    if (rc) return rc;
    if (rows == 0 || width == 0) return QMX_OK;
    if (!x || !codes || !scales) return QMX_ERR_NULL;
    if (!is_aligned(x, 2) || !is_aligned(codes, 16)) return QMX_ERR_ALIGN;
    return launch_status(qmx::launch_f8_quantize(x, x_row_stride, codes, scales, rows, width, block_rows, dtype,
                                                 static_cast<hipStream_t>(stream)));
}

int qmx_f8_dequantize(const uint8_t* codes, const void* scales, int scale_type, void* out, int rows, int width,
                      int block_rows, int dtype, void* stream) {
    const int rc = check_codes(rows, width, block_rows, dtype);
    if (rc) return rc;
    if (scale_type != QMX_SCALE_E8M0 && scale_type != QMX_SCALE_F32) return QMX_ERR_DTYPE;
    if (rows == 0 || width == 0) return QMX_OK;
    if (!codes || !scales || !out) return QMX_ERR_NULL;
    if (!is_aligned(codes, 16) || !is_aligned(out, 16) || (scale_type == QMX_SCALE_F32 && !is_aligned(scales, 4)))
        return QMX_ERR_ALIGN;
    return launch_status(qmx::launch_f8_dequantize(codes, scales, scale_type == QMX_SCALE_F32, out, rows, width,
                                                   block_rows, dtype, static_cast<hipStream_t>(stream)));
}

int qmx_plan_f8(int M, int N, int K, int num_cus, int* tile_rows, int* tile_cols, int* splits) {
    const int rc = check_product(M, N, K);
    if (rc) return rc;
    if (!tile_rows || !tile_cols || !splits) return QMX_ERR_NULL;
    *tile_rows = *tile_cols = 0;
    *splits = 1;
    if (M == 0 || N == 0 || K == 0) return QMX_OK;
    const qmx::F8Plan p = qmx::f8_plan(M, N, K, num_cus > 0 ? num_cus : 256);
    *splits = p.splits;
    switch (p.tile) {
        case qmx::F8_ROWS: *tile_rows = M <= 16 ? 16 : 32; *tile_cols = 16; break;
        case qmx::F8_32x64: *tile_rows = 32; *tile_cols = 64; break;
        case qmx::F8_64x64: *tile_rows = 64; *tile_cols = 64; break;
        case qmx::F8_64x128: *tile_rows = 64; *tile_cols = 128; break;
        case qmx::F8_128x128: *tile_rows = *tile_cols = 128; break;
        default: *tile_rows = *tile_cols = 256; break;
    }
    return QMX_OK;
}

size_t qmx_qmm_f8_workspace_bytes(int M, int N, int K) {
    if (check_product(M, N, K) || M == 0 || N == 0 || K == 0) return 0;
    const int splits = qmx::f8_plan(M, N, K, units()).splits;
    return splits > 1 ? (size_t)splits * M * N * sizeof(float) : 0;
}

int qmx_qmm_f8(const uint8_t* w, const void* w_scales, int w_scale_type, const uint8_t* x, const uint8_t* x_scales,
               void* out, int M, int N, int K, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (!is_half(dtype) || (w_scale_type != QMX_SCALE_E8M0 && w_scale_type != QMX_SCALE_F32)) return QMX_ERR_DTYPE;
    const int rc = check_product(M, N, K);
    if (rc) return rc;
    if (M == 0 || N == 0) return QMX_OK;
    if (!out || (K > 0 && (!w || !w_scales || !x || !x_scales))) return QMX_ERR_NULL;
    if (!is_aligned(out, 2) || !is_aligned(w, 16) || !is_aligned(x, 16) ||
        (w_scale_type == QMX_SCALE_F32 && !is_aligned(w_scales, 4)))
        return QMX_ERR_ALIGN;
    const int cus = units();
    const qmx::F8Plan p = qmx::f8_plan(M, N, K, cus);
    const size_t need = K > 0 && p.splits > 1 ? (size_t)p.splits * M * N * sizeof(float) : 0;
    if (need && (!workspace || !is_aligned(workspace, 16) || workspace_bytes < need)) return QMX_ERR_WORKSPACE;
    const qmx::F8MmArgs a = {w, w_scales, w_scale_type == QMX_SCALE_F32, x, x_scales, out,
                             static_cast<float*>(workspace), M, N, K};
    return launch_status(qmx::launch_qmm_f8(a, p, cus, dtype, static_cast<hipStream_t>(stream)));
}

int qmx_rope(const void* q, long long q_token_stride, long long q_head_stride, void* q_out,
             long long q_out_token_stride, long long q_out_head_stride, int heads, const void* k,
             long long k_token_stride, long long k_head_stride, void* k_out, long long k_out_token_stride,
             long long k_out_head_stride, int kv_heads, const int32_t* positions, const double* frequencies,
             int tokens, int head_dim, int pairs, int interleaved, float scale, int dtype, void* stream) {
    if (!is_half(dtype)) return QMX_ERR_DTYPE;
    if (tokens < 0 || heads < 0 || kv_heads < 0 || heads > 8192 || kv_heads > 8192) return QMX_ERR_SHAPE;
    if (head_dim < 1 || head_dim > 4096 || pairs < 1 || 2 * pairs > head_dim) return QMX_ERR_SHAPE;
    if (!std::isfinite(scale)) return QMX_ERR_SHAPE;
    if (tokens == 0 || heads + kv_heads == 0) return QMX_OK;
    if (!positions || !frequencies || (heads > 0 && (!q || !q_out)) || (kv_heads > 0 && (!k || !k_out)))
        return QMX_ERR_NULL;
    if (!is_aligned(q, 2) || !is_aligned(q_out, 2) || !is_aligned(k, 2) || !is_aligned(k_out, 2) ||
        !is_aligned(positions, 4) || !is_aligned(frequencies, 8))
        return QMX_ERR_ALIGN;
    qmx::RopeArgs a = {};
    a.in[0] = q;
    a.in[1] = k;
    a.out[0] = q_out;
    a.out[1] = k_out;
    a.in_ts[0] = q_token_stride;
    a.in_ts[1] = k_token_stride;
    a.in_hs[0] = q_head_stride;
    a.in_hs[1] = k_head_stride;
    a.out_ts[0] = q_out_token_stride;
    a.out_ts[1] = k_out_token_stride;
    a.out_hs[0] = q_out_head_stride;
    a.out_hs[1] = k_out_head_stride;
    a.heads[0] = heads;
    a.heads[1] = kv_heads;
    a.positions = positions;
    a.frequencies = frequencies;
    a.tokens = tokens;
    a.dim = head_dim;
    a.pairs = pairs;
    a.scale = scale;
    a.interleaved = interleaved != 0;
    Area from[2], to[2];
    for (int i = 0; i < 2; ++i) {
        a.in_place[i] = a.in[i] == a.out[i] && (a.in_ts[i] == a.out_ts[i] || tokens == 1) &&
                        (a.in_hs[i] == a.out_hs[i] || a.heads[i] == 1);
        if (a.heads[i] == 0) continue;
        from[i] = area(a.in[i], 2, head_dim, a.heads[i], a.in_hs[i], tokens, a.in_ts[i]);
        to[i] = area(a.out[i], 2, head_dim, a.heads[i], a.out_hs[i], tokens, a.out_ts[i]);
        if (!apart(head_dim, a.heads[i], a.out_hs[i], tokens, a.out_ts[i]) ||
            share(to[i], area(positions, 4, tokens)) || share(to[i], area(frequencies, 8, pairs)))
            return QMX_ERR_OVERLAP;
    }
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j) {
            if (a.heads[i] == 0 || a.heads[j] == 0) continue;
            if (!(i == j && a.in_place[i]) && share(to[i], from[j])) return QMX_ERR_OVERLAP;
            if (j < i && share(to[i], to[j])) return QMX_ERR_OVERLAP;
        }
    return launch_status(qmx::launch_rope(a, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
