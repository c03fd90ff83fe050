// kv4.h -- host-side launchers of the paged 4-bit key/value cache, shared by
// its kernel sources and the C ABI in kv4_api.cpp.  Arguments are validated
// by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qmx {

// The cache as the kernels see it.  Blocks are 16 tokens of one head and hold
// 2 * dim words of codes; block b of page p and head h is number
// (p * heads + h) << page_shift + b, page_shift = log2(page_size / 16).
struct Kv4View {
    uint32_t* kc;
    uint32_t* ks;  // (scale, bias) pairs, the scale in the low half
    uint32_t* vc;
    uint32_t* vs;
    int num_pages, heads, dim, page_shift, group, dt;
};

struct KvMapsArgs {
    const int* past;
    const int* fresh;
    int* table;
    const int* free_pages;
    long long table_stride;
    int requests, columns, num_free, page_size, tokens;
    int *offsets, *kv_lens, *slots, *positions, *request_ids, *counts;
};

// How an attention call is cut up.  A unit is a tile of `rows` rows of one
// request and key head; a row is one (query, head).  With `lines` == 0 a
// work-group takes a unit whole.  Otherwise the steps of a head's units, 32 keys
// each, are laid end to end and cut into `lines` equal parts (of at least `least`
// steps), a work-group each: what is long is shared, what is short is not alone,
// and the cut follows the lengths, which the host does not know.  A unit in two
// parts or more leaves partial sums that a second kernel joins.
struct Kv4AttnPlan {
    int rows;     // 16: kv4_attn_kernel, else kv4_prompt_kernel
    int waves;    // of a work-group
    int tiles;    // units of a request and head
    int lines, least;
    int cost;     // what a unit costs beside its steps, in steps: on a line, units stand this far apart
};
// Waves of a work-group that takes few rows' units whole, by head size: eight of
// 256 would leave a CU one work-group (138 KB of LDS).
constexpr int few_row_waves(int dim) { return dim == 256 ? 4 : 8; }
// Most units of a head that can be laid end to end, by a work-group's waves.
constexpr int kv4_line_units(int waves) { return waves == 4 ? 1024 : 512; }

struct Kv4AttnArgs {
    Kv4View c;
    const void* q;
    void* out;
    float* lse;    // or null
    const int* table;
    const int* kv_lens;
    const int* offsets;
    long long q_ts, q_hs, table_stride;
    int requests, tokens, heads, each, columns, max_query, max_kv, window;
    float scale_log2;      // softmax scale * log2(e)
    Kv4AttnPlan p;
    // Workspace, with lines > 0.  A part has two places: 2w + 1 for the unit that
    // starts in it and goes on, 2w for one that came from before.
    float* part;   // [2 * lines][kv heads][rows][dim]; rows > 16: over the part's sum
    float* stat;   // [2 * lines][kv heads][rows] pairs (max, sum)
    int* pos;      // the parts' length in steps, then where each unit begins and ends
};

Kv4AttnPlan kv4_attn_plan(int requests, int heads, int kv_heads, int dim, int max_query, int max_kv, int window,
                          int cus);
// Bytes of workspace of such a plan.
inline size_t kv4_attn_workspace(const Kv4AttnPlan& p, int requests, int kv_heads, int dim) {
    if (!p.lines) return 0;
    return (size_t)2 * p.lines * kv_heads * p.rows * (dim + 2) * sizeof(float) +
           (2 * (size_t)requests * p.tiles + 1) * sizeof(int);
}

hipError_t launch_kv_maps(const KvMapsArgs& a, hipStream_t st);
hipError_t launch_kv4_write(const Kv4View& c, const void* k, const void* v, long long k_ts, long long k_hs,
                            long long v_ts, long long v_hs, const int* slots, int tokens, hipStream_t st);
hipError_t launch_kv4_read(const Kv4View& c, void* k, void* v, const int* slots, int tokens, hipStream_t st);
hipError_t launch_kv4_attn(const Kv4AttnArgs& a, hipStream_t st);

}  // namespace qmx
