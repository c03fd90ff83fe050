// kv4_api.cpp -- the C ABI of the paged 4-bit key/value cache: host-side
// validation, how an attention call is cut up, and the launches.  Every check
// runs before any launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "kv4.h"
#include "kv4_attn_launch.h"
#include "qmx.h"
#include "qmx_internal.h"

namespace {

bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int launch_status(hipError_t e) { return e == hipSuccess ? QMX_OK : QMX_ERR_LAUNCH; }

int check_cache(const qmx_kv4_cache* c) {
    if (!c) return QMX_ERR_NULL;
    if (c->dtype != QMX_F16 && c->dtype != QMX_BF16) return QMX_ERR_DTYPE;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return QMX_ERR_SHAPE;
    if ((c->group_size != 32 && c->group_size != 64 && c->group_size != 128) || c->group_size > c->head_dim)
        return QMX_ERR_GROUP;
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return QMX_ERR_SHAPE;
    if (c->num_pages < 0 || c->kv_heads < 1 || c->kv_heads > 1024) return QMX_ERR_SHAPE;
    if (c->num_pages > 0) {
        if (!c->k_codes || !c->k_sb || !c->v_codes || !c->v_sb) return QMX_ERR_NULL;
        if (!is_aligned(c->k_codes, 16) || !is_aligned(c->k_sb, 16) || !is_aligned(c->v_codes, 16) ||
            !is_aligned(c->v_sb, 16))
            return QMX_ERR_ALIGN;
    }
    return QMX_OK;
}

qmx::Kv4View view(const qmx_kv4_cache* c) {
    int shift = 0;
    while ((16 << shift) < c->page_size) ++shift;
    return {c->k_codes, static_cast<uint32_t*>(c->k_sb), c->v_codes, static_cast<uint32_t*>(c->v_sb),
            c->num_pages, c->kv_heads, c->head_dim, shift, c->group_size, c->dtype};
}

// Where the ints of an argument are: `n` of them, `rows` times, `stride` apart.
struct Span {
    const int32_t* p;
    long long n, rows = 1, stride = 0;
};

// Whether `x`, of one row, shares an int with `y`.
bool overlap(const Span& x, const Span& y) {
    if (x.n <= 0 || y.n <= 0 || y.rows <= 0) return false;
    typedef __int128 wide;   // rows may be any distance apart
    const wide row = 4 * (wide)y.n, step = 4 * (wide)y.stride, to = 4 * (wide)x.n;
    const wide from = (wide)reinterpret_cast<uintptr_t>(x.p) - reinterpret_cast<uintptr_t>(y.p);
    if (from + to <= 0 || from >= (y.rows - 1) * step + row) return false;
    if (from < row) return true;
    return ((from - row) / step + 1) * step < from + to;   // the first row that ends behind x's start
}

bool good_heads(int heads, int kv_heads) {
    return kv_heads >= 1 && kv_heads <= 1024 && heads >= kv_heads && heads <= 65536 && heads % kv_heads == 0;
}

// How a call is cut up; the one rule of the call and of its workspace's size.
qmx::Kv4AttnPlan plan_for(int requests, int heads, int kv_heads, int dim, int max_query, int max_kv, int window) {
    const int cus = qmx::device_cu_count();
    return qmx::kv4_attn_plan(requests, heads, kv_heads, dim, std::max(1, max_query), max_kv, window,
                              cus > 0 ? cus : 256);
}

}  // namespace

namespace qmx {

Kv4AttnPlan kv4_attn_plan(int requests, int heads, int kv_heads, int dim, int max_query, int max_kv, int window,
                          int cus) {
    Kv4AttnPlan p;
    const long long rows = (long long)max_query * (heads / kv_heads);
    const long long keys = window ? std::min((long long)max_kv, (long long)window + max_query) : (long long)max_kv;
    // Few rows or many: 8 requests over 4000 keys (8 key heads of 128, bfloat16) take
    // 44 us by units of 16 rows and 61 by the prompt kernel at 48 rows, 53 and 62 at
    // 64, 71 and 65 at 96; heads of 64: 40 and 46 at 64, 51 and 48 at 96; of 256: 99
    // and 109, 141 and 112.
    const bool prompt = rows > 64;
    p.rows = prompt ? kv4::PROMPT_ROWS : 16;
    p.tiles = (int)((rows + p.rows - 1) / p.rows);
    const long long units = (long long)requests * p.tiles, groups = units * kv_heads;
    // Units whole or on a line.  Few rows: joining costs some 5 us, which a walk of
    // 1000 to 1500 keys more costs too (one token of 32 heads on 8 key heads of 128: 12.8
    // us whole and on a line over 1000 keys, 16.6 and 12.8 over 1500, 24 and 13 over
    // 2500; 64 such requests of one length are the same, whose parts are units).
    // Prompts: units enough even each other out, and parts are written and joined in
    // 32 bits (4096 tokens: 197 us whole, 233 on a line); behind a long prefix
    // requests differ (12 of up to 512 tokens over up to 4000, heads of 256: 547 and
    // 220; 3 of up to 300 over 20000: 704 and 185).  Few prompt rows take the same
    // limit of keys, though a line is faster for one request from some 700 on (100
    // tokens: 25 whole and 30 us over 300 keys, 49 and 39 over 1000, 64 and 48 over
    // 1500; 8 requests 26 and 44, 51 and 58, 67 and 69).
    const bool uneven = !prompt || groups < cus * 3 / 4 || (keys > 2ll * max_query && groups < 4ll * cus);
    const bool line = keys > 1536 && uneven && units > 0 && units <= kv4_line_units(prompt ? kv4::PROMPT_WAVES : 4) &&
                      units * (keys / 32 + 32) <= INT_MAX;
    p.waves = prompt ? kv4::PROMPT_WAVES : line ? 4 : few_row_waves(dim);
    p.lines = line ? std::max(1, (prompt ? 1 : 2) * cus / kv_heads) : 0;
    // A unit's queries, first loads and joining waves wait on memory about four
    // times, as long as its work-group takes for some 8 steps (48 tokens over up to
    // 8000, joined: 33.3 us with 8, 34.4 with 16, 39.5 with 32).
    p.cost = 8;
    p.least = 8;
    return p;
}

hipError_t launch_kv4_attn(const Kv4AttnArgs& a, hipStream_t st) {
    const bool half = a.c.dt == DT_F16;
    switch (a.c.dim) {
        case 64: return half ? kv4::launch_dim<64, DT_F16>(a, st) : kv4::launch_dim<64, DT_BF16>(a, st);
        case 128: return half ? kv4::launch_dim<128, DT_F16>(a, st) : kv4::launch_dim<128, DT_BF16>(a, st);
        default: return half ? kv4::launch_dim<256, DT_F16>(a, st) : kv4::launch_dim<256, DT_BF16>(a, st);
    }
}

}  // namespace qmx

extern "C" {

int qmx_kv_maps(const int32_t* past, const int32_t* fresh, int32_t* block_table, const int32_t* free_pages,
                int requests, int columns, long long table_stride, int num_free, int page_size, int tokens,
                int32_t* query_offsets, int32_t* kv_lens, int32_t* slots, int32_t* positions,
                int32_t* request_ids, int32_t* counts, void* stream) {
    if (requests < 0 || columns < 0 || num_free < 0 || tokens < 0 || page_size < 1) return QMX_ERR_SHAPE;
    if ((long long)requests * columns > INT_MAX || requests == INT_MAX) return QMX_ERR_SHAPE;
    if (requests > 1 && table_stride < columns) return QMX_ERR_SHAPE;
    if (!query_offsets || !counts) return QMX_ERR_NULL;
    if (requests > 0 && (!past || !fresh || !kv_lens)) return QMX_ERR_NULL;
    if (requests > 0 && columns > 0 && !block_table) return QMX_ERR_NULL;
    if (num_free > 0 && !free_pages) return QMX_ERR_NULL;
    if (tokens > 0 && (!slots || !positions || !request_ids)) return QMX_ERR_NULL;
    for (const void* p : {(const void*)past, (const void*)fresh, (const void*)block_table, (const void*)free_pages,
                          (const void*)query_offsets, (const void*)kv_lens, (const void*)slots,
                          (const void*)positions, (const void*)request_ids, (const void*)counts})
        if (!is_aligned(p, 4)) return QMX_ERR_ALIGN;
    const Span table = {block_table, columns, requests, table_stride};
    const Span in[] = {{past, requests}, {fresh, requests}, {free_pages, num_free}};
    const Span out[] = {{query_offsets, requests + 1}, {kv_lens, requests}, {slots, tokens},
                        {positions, tokens}, {request_ids, tokens}, {counts, 2}};
    for (const Span& x : in)
        if (overlap(x, table)) return QMX_ERR_OVERLAP;
    for (const Span& x : out) {
        if (overlap(x, table)) return QMX_ERR_OVERLAP;
        for (const Span& y : in)
            if (overlap(x, y)) return QMX_ERR_OVERLAP;
        for (const Span& y : out)
            if (&x != &y && overlap(x, y)) return QMX_ERR_OVERLAP;
    }
    const qmx::KvMapsArgs a = {past, fresh, block_table, free_pages, table_stride, requests, columns, num_free,
                               page_size, tokens, query_offsets, kv_lens, slots, positions, request_ids, counts};
    return launch_status(qmx::launch_kv_maps(a, static_cast<hipStream_t>(stream)));
}

int qmx_kv4_write(const qmx_kv4_cache* cache, const void* k, const void* v, long long k_token_stride,
                  long long k_head_stride, long long v_token_stride, long long v_head_stride,
                  const int32_t* slots, int tokens, void* stream) {
    const int rc = check_cache(cache);
    if (rc) return rc;
    if (tokens < 0 || (long long)tokens * cache->kv_heads > (1ll << 31)) return QMX_ERR_SHAPE;
    if (tokens == 0 || cache->num_pages == 0) return QMX_OK;
    if (!k || !v || !slots) return QMX_ERR_NULL;
    if (!is_aligned(k, 2) || !is_aligned(v, 2) || !is_aligned(slots, 4)) return QMX_ERR_ALIGN;
    return launch_status(qmx::launch_kv4_write(view(cache), k, v, k_token_stride, k_head_stride, v_token_stride,
                                               v_head_stride, slots, tokens, static_cast<hipStream_t>(stream)));
}

int qmx_kv4_read(const qmx_kv4_cache* cache, void* k_out, void* v_out, const int32_t* slots, int tokens,
                 void* stream) {
    const int rc = check_cache(cache);
    if (rc) return rc;
    if (tokens < 0 || (long long)tokens * cache->kv_heads > (1ll << 31)) return QMX_ERR_SHAPE;
    if (tokens == 0) return QMX_OK;
    if (!k_out || !v_out || !slots) return QMX_ERR_NULL;
    if (!is_aligned(k_out, 16) || !is_aligned(v_out, 16) || !is_aligned(slots, 4)) return QMX_ERR_ALIGN;
    return launch_status(qmx::launch_kv4_read(view(cache), k_out, v_out, slots, tokens,
                                              static_cast<hipStream_t>(stream)));
}

size_t qmx_kv4_attention_workspace_bytes(int kv_heads, int head_dim, int requests, int tokens, int heads,
                                         int max_query_len, int max_kv_len, int window) {
    if (!good_heads(heads, kv_heads) || (head_dim != 64 && head_dim != 128 && head_dim != 256) || requests < 0 ||
        tokens < 0 || max_query_len < 0 || max_kv_len < 0 || max_kv_len > INT_MAX - 64 || window < 0)
        return 0;
    const int queries = std::min(max_query_len, tokens);
    return qmx::kv4_attn_workspace(plan_for(requests, heads, kv_heads, head_dim, queries, max_kv_len, window),
                                   requests, kv_heads, head_dim);
}

int qmx_kv4_attention(const qmx_kv4_cache* cache, const void* q, long long q_token_stride, long long q_head_stride,
                      void* out, float* lse, const int32_t* block_table, int columns, long long table_stride,
                      const int32_t* kv_lens, const int32_t* query_offsets, int requests, int tokens, int heads,
                      int max_query_len, int max_kv_len, int window, float scale, void* workspace,
                      size_t workspace_bytes, void* stream) {
    const int rc = check_cache(cache);
    if (rc) return rc;
    if (!good_heads(heads, cache->kv_heads)) return QMX_ERR_SHAPE;
    if (requests < 0 || tokens < 0 || columns < 0 || max_query_len < 0 || max_kv_len < 0 || window < 0)
        return QMX_ERR_SHAPE;
    if (max_query_len > tokens || max_kv_len > INT_MAX - 64 || requests > (1 << 24)) return QMX_ERR_SHAPE;
    if (!std::isfinite(scale) || scale <= 0.0f) return QMX_ERR_SHAPE;
    if ((long long)columns * cache->page_size > INT_MAX) return QMX_ERR_SHAPE;
    if (requests > 1 && table_stride < columns) return QMX_ERR_SHAPE;
    if (tokens == 0) return QMX_OK;
    if (!q || !out || !query_offsets) return QMX_ERR_NULL;
    if (requests > 0 && (!kv_lens || (columns > 0 && !block_table))) return QMX_ERR_NULL;
    if (!is_aligned(q, 2) || !is_aligned(out, 16) || !is_aligned(lse, 4) || !is_aligned(block_table, 4) ||
        !is_aligned(kv_lens, 4) || !is_aligned(query_offsets, 4))
        return QMX_ERR_ALIGN;
    const int queries = std::max(1, max_query_len);
    const auto p = plan_for(requests, heads, cache->kv_heads, cache->head_dim, max_query_len, max_kv_len, window);
    const size_t need = qmx::kv4_attn_workspace(p, requests, cache->kv_heads, cache->head_dim);
    if (need && (!workspace || !is_aligned(workspace, 16) || workspace_bytes < need)) return QMX_ERR_WORKSPACE;
    if ((long long)(requests + 1) * std::max<long long>((long long)p.tiles * cache->kv_heads,
                                                        (long long)queries * heads) > INT_MAX)
        return QMX_ERR_SHAPE;
    qmx::Kv4AttnArgs a = {};
    a.c = view(cache);
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.p = p;
    if (need) {
        const size_t places = (size_t)2 * p.lines * cache->kv_heads * p.rows;
        a.part = static_cast<float*>(workspace);
        a.stat = a.part + places * cache->head_dim;
        a.pos = reinterpret_cast<int*>(a.stat + 2 * places);
    }
    a.table = block_table;
    a.kv_lens = kv_lens;
    a.offsets = query_offsets;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.table_stride = table_stride;
    a.requests = requests;
    a.tokens = tokens;
    a.heads = heads;
    a.each = heads / cache->kv_heads;
    a.columns = columns;
    a.max_query = queries;
    // With no page in the cache nothing is seen, and no address formed.
    a.max_kv = cache->num_pages > 0 ? max_kv_len : 0;
    a.window = window;
    a.scale_log2 = scale * 1.4426950408889634f;
    return launch_status(qmx::launch_kv4_attn(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
