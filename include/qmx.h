/*
 * qmx.h -- C ABI of libqmx: group-wise affine quantized matrix-vector and
 * small-M matrix multiply, and the Q8_0 / Q4_K block matvecs, for AMD MI355X
 * (gfx950).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every pointer argument except those named "host" is a DEVICE pointer
 *   owned by the caller.  The library never allocates, frees or copies
 *   caller memory and never synchronises: work is enqueued on `stream`
 *   (a hipStream_t; NULL means the default stream) and the call returns as
 *   soon as it is enqueued.  Outputs are valid once the stream reaches them.
 * - Arrays are dense and row-major.  `out` must not overlap any input.
 * - All arguments are validated on the host before anything is enqueued; a
 *   negative qmx_status is returned and nothing is launched when a check
 *   fails.  QMX_ERR_LAUNCH reports a launch error returned by the HIP
 *   runtime.  Empty problems (M == 0 or N == 0) return QMX_OK and launch
 *   nothing; K == 0 writes zeros.
 * - Results are bit-reproducible run to run for the same build, device,
 *   arguments and split count: no atomics, fixed reduction orders.
 * - Accumulation is float32 throughout; the output is rounded once, to
 *   nearest even.
 * - The library keeps no state between calls apart from a per-device cache
 *   of the compute-unit count; calls may come from several host threads.
 *
 * The affine format (page "metaltile-std src/mlx/quantized.rs", qmv kernel
 * header, layouts comment of the int8 kernel; page "mlx PR 4682", transposed
 * quantized_matmul):
 *   w_packed : uint32 [N, K*bits/32]; row n is a little-endian bit stream,
 *              code q[n,k] is the unsigned field at stream bits
 *              [k*bits, (k+1)*bits) (4-bit: 8 codes per word, low nibble
 *              first; 8-bit: byte j of a word is code 4*word+j; 3-, 5- and
 *              6-bit fields may straddle two words).
 *   scales, biases : [N, K/group_size] in `dtype`.
 *   x        : [M, K] in `dtype`.     out : [M, N] in `dtype`.
 *   out[m,n] = sum_g ( scales[n,g] * sum_{k in g} q[n,k] * x[m,k]
 *                    + biases[n,g] * sum_{k in g} x[m,k] )
 *            = sum_k x[m,k] * (scales[n,k/gs] * q[n,k] + biases[n,k/gs]).
 * Supported: bits in {1, 2, 3, 4, 5, 6, 8} (the widths of the staged loader
 * of page "mlx PR 4682"); group_size in {32, 64, 128}; K % group_size == 0.
 */
#ifndef QMX_H
#define QMX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QMX_API_VERSION 1

typedef enum qmx_dtype {
    QMX_F32 = 0,   /* IEEE binary32 */
    QMX_F16 = 1,   /* IEEE binary16 */
    QMX_BF16 = 2   /* bfloat16 (upper half of a binary32) */
} qmx_dtype;

typedef enum qmx_status {
    QMX_OK = 0,
    QMX_ERR_NULL = -1,       /* a required pointer is NULL                        */
    QMX_ERR_SHAPE = -2,      /* negative size, or a size the route cannot take     */
    QMX_ERR_BITS = -3,       /* bits not in {1, 2, 3, 4, 5, 6, 8}                  */
    QMX_ERR_GROUP = -4,      /* group_size not in {32, 64, 128} or K % gs != 0     */
    QMX_ERR_DTYPE = -5,      /* unknown dtype, or a dtype the route does not take  */
    QMX_ERR_ALIGN = -6,      /* a pointer lacks the alignment the route needs      */
    QMX_ERR_WORKSPACE = -7,  /* split-K workspace NULL or too small                */
    QMX_ERR_SPLITS = -8,     /* split count out of range for this K                */
    QMX_ERR_LAUNCH = -9,     /* the HIP runtime rejected a launch                  */
    QMX_ERR_DEVICE = -10,    /* no usable HIP device                               */
    QMX_ERR_SCRATCH = -11,   /* partials larger than qmx_qmm_t_splitk_noalloc holds */
    QMX_ERR_OVERLAP = -12    /* an output overlaps an input or another output      */
} qmx_status;

typedef enum qmx_route {
    QMX_ROUTE_QMV = 0,          /* qmx_qmv                      */
    QMX_ROUTE_QMM_T = 1,        /* qmx_qmm_t (unsplit)          */
    QMX_ROUTE_QMM_T_SPLITK = 2  /* qmx_qmm_t_splitk + accumulate */
} qmx_route;

/* Largest split count qmx_qmm_t_splitk accepts. */
#define QMX_MAX_SPLITS 16

/* qmx_qmv -- affine quantized matvec for small M (built for M = 1..7).
 * Computes the affine definition above with float32 accumulation on the
 * vector ALUs: weight codes are streamed once in chunks of 16 bytes (2-, 4-
 * and 8-bit) or of `bits` words = 32 codes (1, 3, 5, 6 bits), the sum
 * of x is formed once per group (bias hoist), lanes are reduced with a
 * fixed-order cross-lane tree (page "metaltile-std src/mlx/quantized.rs",
 * qmv kernel: bias hoist, x reuse across rows, simd_sum and lane-0 store).
 * dtype: QMX_F32, QMX_F16 or QMX_BF16 for x, scales, biases and out.
 * Any M >= 0 is accepted (rows of x are processed in tiles of up to 4).
 * Extra requirements: rows of w_packed are whole chunks ((K*bits) % 128 == 0
 * for 2, 4 and 8 bits; K % 32 == 0, always true, for the others), w_packed
 * 16-byte aligned, x aligned to its element size.
 */
int qmx_qmv(const uint32_t* w_packed, const void* scales, const void* biases,
            const void* x, void* out, int M, int N, int K, int bits, int group_size,
            int dtype, void* stream);

/* qmx_qmm_t -- affine quantized x * W^T on the matrix cores (any M; built
 * for M >= 8, and what qmx_plan picks at M = 2..7 for large weights)
 * (page "mlx PR 4682": staged transposed qmm that fetches the next K step
 * while the current one is consumed from threadgroup memory, with one
 * barrier per K step).  Here the packed codes and x of the next K blocks are
 * copied from HBM straight into a ring of LDS stages (global-to-LDS loads,
 * no register staging) while the matrix cores consume the current stage;
 * scales and biases are staged once per work-group in 16-byte chunks when
 * aligned, else with each stage.  Codes are expanded to exact 16-bit values
 * right before bf16/f16 MFMA, and scale and bias are applied per group in
 * float32, so the only rounding besides float32 accumulation is the final
 * one.
 * dtype: QMX_F16 or QMX_BF16 only (QMX_ERR_DTYPE for QMX_F32).
 * Extra requirements: K % 128 == 0; w_packed, x 16-byte aligned.
 */
int qmx_qmm_t(const uint32_t* w_packed, const void* scales, const void* biases,
              const void* x, void* out, int M, int N, int K, int bits, int group_size,
              int dtype, void* stream);

/* qmx_qmm_t_splitk -- qmx_qmm_t with K split into `splits` partitions
 * (page "mlx PR 4682": split-K kernel writing float32 partials that a
 * separate accumulate kernel sums, rounding once).  K is cut into segments
 * of 256 columns (of 128 columns when K is not a multiple of 256), and
 * partition p covers segments [floor(p*nseg/splits), floor((p+1)*nseg/splits))
 * with nseg = K/segment; each partition must hold at least 256 columns, so
 * 2 <= splits <= min(QMX_MAX_SPLITS, K/256).  The first kernel writes
 * workspace[p][m][n] (float32); the second sums p = 0..splits-1 in that
 * order and rounds once to `dtype`.  workspace: device memory of at least
 * qmx_splitk_workspace_bytes(M, N, splits) bytes, 16-byte aligned, owned by
 * the caller, overwritten by the call (its contents on entry do not
 * matter); calls that share one workspace must be ordered on one stream.
 * Other requirements as qmx_qmm_t.
 */
int qmx_qmm_t_splitk(const uint32_t* w_packed, const void* scales, const void* biases,
                     const void* x, void* out, int M, int N, int K, int bits, int group_size,
                     int dtype, int splits, void* workspace, size_t workspace_bytes,
                     void* stream);

/* qmx_qmm_t_partials -- the first kernel of qmx_qmm_t_splitk on its own:
 * writes partition p's float32 sums into workspace[p][m][n] for
 * p = 0..splits-1 (the split-K partial kernel of page "mlx PR 4682") and
 * touches nothing else.  Arguments, partitions and requirements are those
 * of qmx_qmm_t_splitk without `out`; a NULL or short workspace is
 * QMX_ERR_WORKSPACE. */
int qmx_qmm_t_partials(const uint32_t* w_packed, const void* scales, const void* biases,
                       const void* x, int M, int N, int K, int bits, int group_size,
                       int dtype, int splits, void* workspace, size_t workspace_bytes,
                       void* stream);

/* qmx_splitk_accumulate -- the second kernel of qmx_qmm_t_splitk on its own
 * (the separate accumulate kernel of page "mlx PR 4682"):
 * out[m][n] = round(sum over p = 0..splits-1, in that order, of
 * workspace[p][m][n]), float32 sums rounded once to `dtype` (QMX_F16 or
 * QMX_BF16).  workspace: splits*M*N float32, 16-byte aligned; out: M*N
 * elements.  2 <= splits <= QMX_MAX_SPLITS. */
int qmx_splitk_accumulate(const void* workspace, void* out, int M, int N, int splits, int dtype,
                          void* stream);

/* Bytes of float32 partials qmx_qmm_t_splitk needs: splits * M * N * 4
 * (0 for negative arguments). */
size_t qmx_splitk_workspace_bytes(int M, int N, int splits);

/* Size of the per-device scratch array of qmx_qmm_t_splitk_noalloc. */
#define QMX_NOALLOC_SCRATCH_BYTES (16u << 20)

/* qmx_qmm_t_splitk_noalloc -- qmx_qmm_t_splitk for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc).  Same arguments, partitions, results and
 * errors as qmx_qmm_t_splitk without the workspace: the float32 partials go
 * into a scratch array of QMX_NOALLOC_SCRATCH_BYTES that this library holds
 * on each device it runs on until the process ends (16 MiB covers every
 * split qmx_plan picks on a 256-CU device: splits * tiles <= CUs, a tile at
 * most 128 x 128 floats).  QMX_ERR_SCRATCH when splits * M * N * 4 exceeds
 * it.  Nothing is allocated or freed: the array's device address is looked
 * up once per device (QMX_ERR_DEVICE if that fails).  Every call on one
 * device shares that device's array and nothing in it needs clearing; calls
 * that overlap on one device (e.g. on two streams) race on it and must be
 * ordered by the caller. */
int qmx_qmm_t_splitk_noalloc(const uint32_t* w_packed, const void* scales, const void* biases,
                             const void* x, void* out, int M, int N, int K, int bits, int group_size,
                             int dtype, int splits, void* stream);

/* qmx_matvec_q8_0 -- Q8_0 block matvec, M = 1 (page "hanzo-kernel
 * src/quant.rs": Q8_0 matvec and its packed layout).
 * w_blocks: uint32 [N, K/32*9]; each 32-weight block is 9 words, the f16
 * scale d in the low 16 bits of word 0 and 32 signed int8 quants in words
 * 1..8 (quant i at byte i%4 of word 1+i/4).  x: float32 [K]; out: float32
 * [N];  out[n] = sum_blocks d * sum_i q_i * x[32*block+i].
 * Requirements: K % 32 == 0; w_blocks and x 16-byte aligned.
 */
int qmx_matvec_q8_0(const uint32_t* w_blocks, const float* x, float* out, int N, int K,
                    void* stream);

/* qmx_matvec_q4_k -- Q4_K super-block matvec, M = 1 (page "hanzo-kernel
 * src/quant.rs": Q4_K block comment, scale/min unpack and kernel).
 * w_blocks: uint32 [N, K/256*36]; each 144-byte super-block holds f16 d
 * (bytes 0-1), f16 dmin (bytes 2-3), 12 bytes of packed 6-bit scales and
 * mins (bytes 4-15) and 128 bytes of 4-bit quants (bytes 16-143).  Quant
 * byte 32g+i gives element 64g+i (low nibble, sub-block 2g) and element
 * 64g+32+i (high nibble, sub-block 2g+1); the weight of code q in sub-block
 * j is d*sc_j*q - dmin*m_j.  x: float32 [K]; out: float32 [N].
 * Requirements: K % 256 == 0; w_blocks and x 16-byte aligned.
 */
int qmx_matvec_q4_k(const uint32_t* w_blocks, const float* x, float* out, int N, int K,
                    void* stream);

/* qmx_matvec_q8_i8 -- integer-activation matvec (page "hanzo-kernel
 * src/quant.rs", packed-int8 dp4a matvec and its block-per-row form):
 *   out[n] = sum_b wd[n*K/32 + b] * sum_{i in block b} wq[n][i] * xq[i]
 * wq: int8 weights [N][K] packed four to a uint32 (element i at byte i % 4,
 * two's complement); xq: int8 activations [K] packed the same way; wd:
 * float32 [N][K/32], one scale per 32-element block of a row; out: float32
 * [N].  Each block's integer sum is exact (4-way integer dot instructions);
 * the scaled blocks are summed in float32.  Requirements: K % 32 == 0
 * (QMX_ERR_GROUP), wq and xq 16-byte aligned, wd and out 4-byte aligned
 * (QMX_ERR_ALIGN); K = 0 writes zeros.  Device pointers, caller-owned,
 * asynchronous on `stream`.
 */
int qmx_matvec_q8_i8(const uint32_t* wq, const uint32_t* xq, const float* wd, float* out,
                     int N, int K, void* stream);

/* qmx_plan -- the dispatch policy as a pure host function (page "mlx PR
 * 4682", dispatch table and split rule; page "metaltile-std
 * src/mlx/quantized.rs", M-based kernel selector).  Writes the route
 * (qmx_route) and split count (1 when unsplit) that qmx_qmm would use for
 * this problem on a device with `num_cus` compute units (num_cus <= 0:
 * 256).  Routes: float32 activations, K % 128 != 0 and M = 1 take qmx_qmv;
 * M = 2..7 takes qmx_qmv unless a cost estimate (qmv's vector work grows
 * with M, the matrix route with the weight bytes) favours the matrix cores;
 * otherwise qmx_qmm_t, split along K when its tiles leave compute units idle
 * (tiles of 128 columns by up to 64 rows of x; above M = 192 by up to 128
 * rows when those fill the device or launch more work-groups after the
 * split; for 2-, 4- and 8-bit codes split tiles of 64 columns at half the
 * partitions where they fit one round of the device, and unsplit tiles of
 * 16 or 32 columns for M <= 32 where few columns would leave compute units
 * idle).  Performs no HIP call.  Returns QMX_OK or a validation status.
 * route/splits: host pointers.
 */
int qmx_plan(int M, int N, int K, int bits, int group_size, int dtype, int num_cus,
             int* route, int* splits);

/* Workspace bytes qmx_qmm needs for this problem (0 unless the plan picks
 * split-K) on the current device.  Host function; may query the device's
 * compute-unit count once. */
size_t qmx_qmm_workspace_bytes(int M, int N, int K, int bits, int group_size, int dtype);

/* qmx_qmm -- the policy-dispatched entry: runs qmx_qmv, qmx_qmm_t or
 * qmx_qmm_t_splitk as qmx_plan decides for the current device.  workspace
 * may be NULL when qmx_qmm_workspace_bytes() is 0; otherwise it must be at
 * least that large (QMX_ERR_WORKSPACE if not). */
int qmx_qmm(const uint32_t* w_packed, const void* scales, const void* biases,
            const void* x, void* out, int M, int N, int K, int bits, int group_size,
            int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Static, NUL-terminated description of a status code. */
const char* qmx_strerror(int status);

/* QMX_API_VERSION of the built library. */
int qmx_api_version(void);

/* qmx_qmm_batched -- qmx_qmm over a batch of independent problems of one
 * shape: 3-D (batched) quantized weights, strided activations and
 * activations at any element offset (page "mlx PR 4682": the batched
 * transposed qmm, its test of 3-D quantized weights with strided and
 * odd-offset activations, and activations that are not suitably aligned
 * being copied first).
 *   out[i][m][n] = sum_k x_i[m][k] * (s_i[n,k/gs] * q_i[n,k] + b_i[n,k/gs])
 * for i < batch, where
 *   weights i  : w_packed + i*w_batch_stride words (0 shares one matrix;
 *                a multiple of 4, so every matrix is 16-byte aligned),
 *   scales/biases i : + i*sb_batch_stride elements (0 shares them),
 *   x_i rows   : x + i*x_batch_stride + m*x_row_stride elements
 *                (x_row_stride >= K; any element offset),
 *   out        : contiguous [batch][M][N] in `dtype`.
 * Each matrix has the layout of the unbatched calls.  Routes and splits
 * follow qmx_plan_batched (one launch for the whole batch; split-K partials
 * are [S][batch][M][N]).  When x, x_batch_stride or x_row_stride is not
 * 16-byte aligned, x is first copied into the workspace as a contiguous
 * [batch][M][K] array.  workspace: at least
 * qmx_qmm_batched_workspace_bytes(...) bytes, 256-byte aligned, may be NULL
 * when that is 0; contents on entry do not matter; calls sharing one
 * workspace must be ordered on one stream.
 * Errors: as qmx_qmm; QMX_ERR_SHAPE for batch outside [0, 65535], a
 * negative stride or x_row_stride < K; QMX_ERR_ALIGN for a weight stride
 * that is not a multiple of 4 words.
 */
int qmx_qmm_batched(const uint32_t* w_packed, const void* scales, const void* biases,
                    const void* x, void* out, int batch, int M, int N, int K,
                    long long w_batch_stride, long long sb_batch_stride,
                    long long x_batch_stride, long long x_row_stride, int bits,
                    int group_size, int dtype, void* workspace, size_t workspace_bytes,
                    void* stream);

/* Workspace bytes qmx_qmm_batched needs (split-K partials as planned on the
 * current device, plus the copy of x when x or its strides are not 16-byte
 * aligned; x is only inspected, never dereferenced).  0 on invalid input. */
size_t qmx_qmm_batched_workspace_bytes(int batch, int M, int N, int K, int bits, int group_size,
                                       int dtype, const void* x, long long x_batch_stride,
                                       long long x_row_stride);

/* qmx_qmm_gather -- qmx_qmm_batched where problem i takes weight matrix
 * w_index[i] (of num_w) and activation matrix x_index[i] (of num_x) instead
 * of matrix i (page "mlx PR 4682": gathered qmm, the batched route with
 * per-problem weight selection, as mixture-of-experts layers use it).
 *   out[i] = x_{x_index[i]} * dequant(W_{w_index[i]})^T,  i < batch
 * w_index, x_index: device arrays of `batch` int32, 4-byte aligned, owned by
 * the caller and read by the kernels (so not checked on the host): a value
 * outside [0, count - 1] is clamped to that range.  Either may be NULL for
 * the identity (then that operand has `batch` matrices).  Strides, layouts,
 * routes, workspace (qmx_qmm_gather_workspace_bytes; a misaligned x is
 * copied as num_x matrices) and errors as qmx_qmm_batched; QMX_ERR_SHAPE
 * also for num_w or num_x < 1 with a non-empty batch.
 */
int qmx_qmm_gather(const uint32_t* w_packed, const void* scales, const void* biases,
                   const void* x, void* out, const int32_t* w_index, const int32_t* x_index,
                   int num_w, int num_x, int batch, int M, int N, int K,
                   long long w_batch_stride, long long sb_batch_stride,
                   long long x_batch_stride, long long x_row_stride, int bits, int group_size,
                   int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes qmx_qmm_gather needs (num_x: the activation matrices, or
 * `batch` when x_index is NULL). */
size_t qmx_qmm_gather_workspace_bytes(int batch, int num_x, int M, int N, int K, int bits,
                                      int group_size, int dtype, const void* x,
                                      long long x_batch_stride, long long x_row_stride);

/* qmx_qmm_gather_sorted -- qmx_qmm_gather for a w_index that holds runs of
 * equal values, as a mixture-of-experts router's output does once the
 * problems are ordered by expert (the gathered qmm of page "mlx PR 4682";
 * the grouping below is this library's).  Arguments, workspace
 * (qmx_qmm_gather_workspace_bytes), results within the same tolerance, and
 * errors as qmx_qmm_gather, for any index arrays: sortedness only decides
 * how much work is shared, never what is computed.
 * At M = 1 on the vector route, one work-group serves up to g consecutive
 * problems whose clamped w_index values are equal, as the x rows of one tile,
 * so a run of problems on one weight matrix streams those weights once
 * rather than once per problem.  g = 1, 2 or 4 is the run length that
 * batch / num_w suggests (rounded up; 4 from 3 on).  Runs are cut at
 * multiples of g.  Other shapes, and x matrices spanning 2 GiB or more, run
 * as qmx_qmm_gather.  Reruns with the same inputs are bit-identical; the
 * float32 summation order can differ from qmx_qmm_gather's.
 */
int qmx_qmm_gather_sorted(const uint32_t* w_packed, const void* scales, const void* biases,
                          const void* x, void* out, const int32_t* w_index,
                          const int32_t* x_index, int num_w, int num_x, int batch, int M, int N,
                          int K, long long w_batch_stride, long long sb_batch_stride,
                          long long x_batch_stride, long long x_row_stride, int bits,
                          int group_size, int dtype, void* workspace, size_t workspace_bytes,
                          void* stream);

/* qmx_plan for a batch: the tiles of all problems share the device, so a
 * batch needs fewer K partitions.  Pure host function. */
int qmx_plan_batched(int batch, int M, int N, int K, int bits, int group_size, int dtype,
                     int num_cus, int* route, int* splits);

/* ------------------------------------------------------------------------
 * Paged key/value cache held in 4 bits.
 *
 * The affine format of the weights above, at 4 bits, for what an attention
 * layer keeps of its tokens: a token's keys (and values) of one head are cut
 * into groups of group_size elements, a group has a scale s and a bias b in
 * `dtype`, and an element with code c stands for c * s + b.  Writing takes
 * lo and hi, the group's least and greatest element: b = lo,
 * s = (hi - lo) / 15 rounded to `dtype`, c = (x - b) / s rounded to nearest
 * even and kept within 0..15 (0 where s is 0).  A group that holds a NaN or
 * whose hi - lo is infinite reads back as NaN or infinite, whole.
 *
 * Tokens live in pages of page_size; token `at` of page p has the slot
 * p * page_size + at.  With D = head_dim and G = D / group_size:
 *   k_codes, v_codes : uint32 [num_pages, kv_heads, page_size * D / 8]
 *   k_sb, v_sb       : [num_pages, kv_heads, page_size, G, 2] in `dtype`,
 *                      scale then bias.
 * A page and head holds page_size / 16 blocks of 16 tokens, 2 * D words each:
 *   keys:   word (h * 16 + token) * (D / 32) + j holds elements
 *           32j + 8h + e, e = 0..7, element e at bit 4 * (e / 2) + 16 * (e % 2)
 *           (h = 0..3);
 *   values: 16-bit half ((h * 16 + n) * (D / 64) + a) * 4 + i holds token
 *           4h + i's elements 16 * (4a + f) + n, f = 0..3, at bit 4f
 *           (n = 0..15),
 * which is how the matrix cores take them: a lane's operand is one load.
 *
 * Supported: dtype QMX_F16 or QMX_BF16; head_dim 64, 128 or 256; group_size
 * 32, 64 or 128, at most head_dim; page_size 16, 32, ..., a power of two up
 * to 1024.  The four arrays are 16-byte aligned.
 */
typedef struct qmx_kv4_cache {
    uint32_t* k_codes;
    void* k_sb;
    uint32_t* v_codes;
    void* v_sb;
    int num_pages, kv_heads, head_dim, page_size, group_size, dtype;
} qmx_kv4_cache;

/* qmx_kv_maps -- block table entries and slot maps of one step, from the
 * requests' lengths, in one launch.  Request r has past[r] tokens in its
 * pages and gets fresh[r] more (negative lengths count as 0):
 *   query_offsets [requests + 1] : running sum of fresh, held to `tokens`;
 *   kv_lens [requests]           : past[r] + its tokens within `tokens`;
 *   block_table [requests, columns], rows table_stride apart: the pages that
 *       request r lacks, ceil(kv_lens[r] / page_size) - ceil(past[r] /
 *       page_size), are taken from free_pages in order, request after
 *       request, and entered behind those it has (-1 where free_pages ends;
 *       nothing is entered past `columns`); other entries stay;
 *   slots, positions, request_ids [tokens] : of each new token, request after
 *       request; slot -1 where its page is missing (an entry below 0, a column
 *       past the table, a slot past 2^31 - 1), and all three -1 behind the last
 *       token;
 *   counts [2] : the sum of fresh, and the pages wanted (a caller sees here
 *       that `tokens` or num_free was too small).
 * page_size: any size of at least 1.  requests * columns is at most 2^31 - 1.
 * Groups of the launch read the lengths while others write: no output may
 * overlap past, fresh, free_pages, the table's rows or another output, nor the
 * rows an input (QMX_ERR_OVERLAP; kv_lens are not the next step's past in
 * place). */
int qmx_kv_maps(const int32_t* past, const int32_t* fresh, int32_t* block_table,
                const int32_t* free_pages, int requests, int columns, long long table_stride,
                int num_free, int page_size, int tokens, int32_t* query_offsets, int32_t* kv_lens,
                int32_t* slots, int32_t* positions, int32_t* request_ids, int32_t* counts,
                void* stream);

/* qmx_kv4_write -- quantises new tokens into the cache.  k, v: [tokens,
 * kv_heads, head_dim] in the cache's dtype with unit element stride, tokens
 * and heads *_token_stride and *_head_stride elements apart (any alignment
 * of whole elements; 16-byte aligned rows are read faster).  slots: int32
 * [tokens]; a slot below 0 or past the cache is skipped.  Slots of one call
 * are distinct. */
int qmx_kv4_write(const qmx_kv4_cache* cache, const void* k, const void* v, long long k_token_stride,
                  long long k_head_stride, long long v_token_stride, long long v_head_stride,
                  const int32_t* slots, int tokens, void* stream);

/* qmx_kv4_read -- the values that cached tokens stand for, c * s + b rounded
 * to dtype: k_out, v_out [tokens, kv_heads, head_dim], 16-byte aligned; zeros
 * where the slot is below 0 or past the cache. */
int qmx_kv4_read(const qmx_kv4_cache* cache, void* k_out, void* v_out, const int32_t* slots,
                 int tokens, void* stream);

/* qmx_kv4_attention -- causal attention of new tokens over the cache, which
 * holds them already:
 *   out[t, a] = sum_j softmax_j(scale * q[t, a] . k_j) v_j
 * over the keys j of t's request that t sees.  Request r has the tokens
 * query_offsets[r] .. query_offsets[r + 1] - 1, the last of its kv_lens[r]
 * cached ones: the token at position p sees positions 0..p, with window > 0
 * only the last `window` of them; a position whose block_table entry is
 * outside 0..num_pages - 1, or past max_kv_len, is not seen.  Head a reads key
 * head a / (heads / kv_heads).  A token that sees nothing, or belongs to no
 * request (before the first offset or from the last on), gets zeros.  What is not seen may hold anything, NaN included.
 *   q     : [tokens, heads, head_dim], unit element stride, other strides in
 *           elements; out: contiguous, 16-byte aligned; both in the cache's
 *           dtype.
 *   lse   : float32 [tokens, heads] or NULL: log of the sum of exp of the
 *           scaled scores (-inf where nothing is seen).
 *   max_query_len, max_kv_len : at least the longest request's new and cached
 *           tokens (host numbers: they size the launch; queries of a request
 *           past max_query_len are left unwritten); max_query_len is at most
 *           `tokens`.
 *   scale : finite and above 0.
 *   workspace : qmx_kv4_attention_workspace_bytes bytes, 16-byte aligned (NULL
 *           where that is 0), overwritten; calls that share it are ordered.
 * Scores and sums are float32 on exact codes; elements of queries count down
 * to 2^-40 of their row's largest, with more than 64 query rows a key head
 * those of bfloat16 keys to 2^-31 of their token's. What the value codes are
 * multiplied by, a probability times a scale, is held in two bfloat16
 * numbers, to 2^-16 of itself; with more than 64 query rows a key head
 * (max_query_len * heads / kv_heads), values and, in a bfloat16 cache,
 * probabilities are rounded to float16 instead, to 2^-11 of themselves,
 * values also to 2^-18 of their token's largest, and the product of both to
 * 2^-26 of the largest finite value that the query sees. How the keys are cut
 * among work-groups follows the lengths and these arguments, so reruns with
 * the same are bit-identical. */
int qmx_kv4_attention(const qmx_kv4_cache* cache, const void* q, long long q_token_stride,
                      long long q_head_stride, void* out, float* lse, const int32_t* block_table,
                      int columns, long long table_stride, const int32_t* kv_lens,
                      const int32_t* query_offsets, int requests, int tokens, int heads,
                      int max_query_len, int max_kv_len, int window, float scale, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Workspace bytes qmx_kv4_attention needs (0 for arguments it refuses; a
 * max_query_len above `tokens`, which the call does not take, is taken as
 * `tokens`).  Depends on the compute units of the current device. */
size_t qmx_kv4_attention_workspace_bytes(int kv_heads, int head_dim, int requests, int tokens,
                                         int heads, int max_query_len, int max_kv_len, int window);

#ifdef __cplusplus
}
#endif

#endif /* QMX_H */
