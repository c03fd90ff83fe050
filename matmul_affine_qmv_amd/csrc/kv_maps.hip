// kv_maps.hip -- block tables and slot maps from the requests' lengths.
//
// Every work-group scans all requests by itself, 4096 at most at a time, so one
// launch suffices and no group waits for another: a token's page is either one
// that its request held before the call (read from the table, which this call
// leaves alone there) or the free page whose place in the list the scan gives.
// A work-group then writes its own range of tokens, or its share of the new
// table entries.
//
// Bound by waits, one after the other (lengths, scan, search, table, stores): 5 us
// for 24 requests, 13 us for 3000 requests with 300000 tokens, where the 3.8 MB
// would take 0.8 us.  Two scans, for tokens and then pages, took 15 us.
#include "kv4.h"
#include "kv_scan.h"

namespace qmx {
namespace {

constexpr int THREADS = 1024;
constexpr int EACH = 4;                // most requests of a thread at a time
constexpr int WAVES = THREADS / 64;

// Numbers up to 2^32 - 1 by the page size.
template <bool SHIFTS>
struct Pages {
    uint32_t size;
    int shift;   // SHIFTS: the size is a power of two
    __device__ __forceinline__ uint32_t whole(uint32_t x) const { return SHIFTS ? x >> shift : x / size; }
    __device__ __forceinline__ uint32_t rest(uint32_t x) const { return SHIFTS ? x & (size - 1) : x % size; }
    __device__ __forceinline__ uint32_t count(uint32_t x) const { return whole(x) + (rest(x) ? 1 : 0); }
};

template <bool SHIFTS>
__global__ __launch_bounds__(THREADS) void kv_maps_kernel(KvMapsArgs a, int per_group, int token_groups, int per,
                                                         int shift) {
    __shared__ int s_end[EACH * THREADS], s_page_end[EACH * THREADS], s_past[EACH * THREADS];
    __shared__ int s_waves[2][WAVES];
    const Pages<SHIFTS> page{(uint32_t)a.page_size, shift};
    const int chunk = per * THREADS;   // requests at a time, `per` a thread
    const int tid = threadIdx.x;
    const bool first = blockIdx.x == 0;
    const int t0 = (int)min((long long)blockIdx.x * per_group, (long long)a.tokens);
    const int t1 = (int)min((long long)t0 + per_group, (long long)a.tokens);
    int sum = 0;     // new tokens of the chunks before, held to 2^31 - 1
    int pages = 0;   // pages handed out before
    if (first && tid == 0) a.offsets[0] = 0;
    int n[EACH], past[EACH];
    auto read = [&](int r0) {
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int r = r0 + per * tid + i;
            const bool there = i < per && r < a.requests;
            n[i] = there ? max(a.fresh[r], 0) : 0;
            past[i] = there ? max(a.past[r], 0) : 0;
        }
    };
    read(0);
    for (int r0 = 0; r0 < a.requests; r0 += chunk) {
        const int count = min(chunk, a.requests - r0);
        const int begin = min(sum, a.tokens);
        // Both sums at once, the pages as if every token had room; where the room
        // ends in this chunk, the pages once more.
        int mine[2] = {0, 0}, total[2], end[EACH], held[EACH], take[EACH];
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            mine[0] = add_held(mine[0], n[i]);
            held[i] = (int)min(page.count((uint32_t)past[i]), (uint32_t)a.columns);
            take[i] = (int)min(page.count((uint32_t)past[i] + (uint32_t)n[i]), (uint32_t)a.columns) - held[i];
            mine[1] += take[i];
        }
        scan_group<WAVES>(mine, s_waves, total);
        int e = add_held(mine[0], sum);
        const bool cut = add_held(sum, total[0]) > a.tokens;
        int cut_takes = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int start = min(e, a.tokens);
            e = add_held(e, n[i]);
            end[i] = min(e, a.tokens);
            const uint32_t kv = (uint32_t)past[i] + (uint32_t)(end[i] - start);
            if (cut) {
                take[i] = (int)min(page.count(kv), (uint32_t)a.columns) - held[i];
                cut_takes += take[i];
            }
            const int r = per * tid + i;
            if (first && i < per && r < count) {
                a.offsets[r0 + r + 1] = end[i];
                a.kv_lens[r0 + r] = (int)min(kv, 0x7fffffffu);
            }
        }
        int chunk_pages = total[1], takes[1] = {mine[1]};
        if (cut) {
            int pages_total[1];
            takes[0] = cut_takes;
            scan_group<WAVES>(takes, s_waves, pages_total);
            chunk_pages = pages_total[0];
        }
        int page_end = pages + takes[0];
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int r = per * tid + i;
            page_end += take[i];
            if (i < per) {
                s_end[r] = end[i];
                s_page_end[r] = page_end;
                s_past[r] = past[i];
            }
        }
        if (r0 + chunk < a.requests) read(r0 + chunk);
        __syncthreads();
        const int stop = s_end[count - 1];
        // unsigned: a step may pass 2^31 - 1
        for (uint32_t i = (uint32_t)max(t0, begin) + tid; i < (uint32_t)min(t1, stop); i += THREADS) {
            const int t = (int)i, r = first_after(s_end, count, t);
            const int start = r ? s_end[r - 1] : begin;
            const uint32_t before = (uint32_t)s_past[r], at = before + (uint32_t)(t - start);
            const uint32_t col = page.whole(at), held = min(page.count(before), (uint32_t)a.columns);
            long long slot = -1;
            if (col < (uint32_t)a.columns) {
                long long p;
                if (col < held) {
                    p = a.table[(r0 + r) * a.table_stride + col];
                } else {
                    const long long place = (long long)(r ? s_page_end[r - 1] : pages) + (int)(col - held);
                    p = place < a.num_free ? a.free_pages[place] : -1;
                }
                if (p >= 0) slot = p * a.page_size + page.rest(at);
                if (slot > 0x7fffffffll) slot = -1;
            }
            a.slots[t] = (int)slot;
            a.positions[t] = (int)min(at, 0x7fffffffu);
            a.request_ids[t] = r0 + r;
        }
        const int turn = (int)blockIdx.x - token_groups;   // groups behind those of the tokens enter the pages
        long long p = turn >= 0 ? (long long)pages + turn * THREADS + tid : (long long)pages + chunk_pages;
        for (; p < (long long)pages + chunk_pages; p += (long long)(gridDim.x - token_groups) * THREADS) {
            const int r = first_after(s_page_end, count, (int)p);
            const int j = (int)p - (r ? s_page_end[r - 1] : pages);
            const int held = (int)min(page.count((uint32_t)s_past[r]), (uint32_t)a.columns);
            a.table[(r0 + r) * a.table_stride + held + j] = p < a.num_free ? a.free_pages[p] : -1;
        }
        sum = add_held(sum, total[0]);
        pages += chunk_pages;
        __syncthreads();
    }
    for (uint32_t t = (uint32_t)max(t0, min(sum, a.tokens)) + tid; t < (uint32_t)t1; t += THREADS) {
        a.slots[t] = -1;
        a.positions[t] = -1;
        a.request_ids[t] = -1;
    }
    if (first && tid == 0) {
        a.counts[0] = sum;
        a.counts[1] = pages;
    }
}

}  // namespace

hipError_t launch_kv_maps(const KvMapsArgs& a, hipStream_t st) {
    long long groups = ((long long)a.tokens + THREADS - 1) / THREADS;
    groups = groups < 1 ? 1 : groups > 512 ? 512 : groups;
    const int per_group = (int)(((long long)a.tokens + groups - 1) / groups);
    const int per = a.requests > EACH * THREADS ? EACH : a.requests > THREADS ? (a.requests + THREADS - 1) / THREADS : 1;
    // entries past the free pages are written too, so their number is only a guide
    const int page_groups = 1 + (a.num_free < 64 * THREADS ? a.num_free / THREADS : 63);
    const unsigned all = (unsigned)groups + page_groups;
    int shift = 0;
    while (shift < 30 && (1 << shift) < a.page_size) ++shift;
    if ((1 << shift) == a.page_size)
        kv_maps_kernel<true><<<all, THREADS, 0, st>>>(a, per_group, (int)groups, per, shift);
    else
        kv_maps_kernel<false><<<all, THREADS, 0, st>>>(a, per_group, (int)groups, per, 0);
    return hipGetLastError();
}

}  // namespace qmx
