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

struct Kv4AttnArgs {
    Kv4View c;
    const void* q;
    void* out;
    float* lse;    // or null
    float* part;   // split partial sums [splits][tokens][heads][dim], then (max, sum) pairs
    const int* table;
    const int* kv_lens;
    const int* offsets;
    long long q_ts, q_hs, table_stride;
    int requests, tokens, heads, each, columns, max_query, max_kv, window;
    int splits, chunk;     // key range of a split in tokens (a multiple of 32)
    int tiles;             // row tiles of a request and key head
    float scale_log2;      // softmax scale * log2(e)
};

// How an attention call is cut up.
struct Kv4AttnPlan {
    int rt, wm, wk;   // 16-row tiles a wave, waves along rows, waves along keys
    int tiles, splits, chunk;
};
Kv4AttnPlan kv4_attn_plan(int requests, int heads, int kv_heads, int dim, int max_query, int max_kv, int window,
                          int cus);

hipError_t launch_kv_maps(const KvMapsArgs& a, hipStream_t st);
hipError_t launch_kv4_write(const Kv4View& c, const void* k, const void* v, long long k_ts, long long k_hs,
                            long long v_ts, long long v_hs, const int* slots, int tokens, hipStream_t st);
hipError_t launch_kv4_read(const Kv4View& c, void* k, void* v, const int* slots, int tokens, hipStream_t st);
hipError_t launch_kv4_attn(const Kv4AttnArgs& a, const Kv4AttnPlan& p, hipStream_t st);

}  // namespace qmx
