// kv_maps.hip -- block tables and slot maps from the requests' lengths.
//
// Every work-group scans all requests by itself, CHUNK at a time, so one
// launch suffices and no group waits for another: a token's page is either one
// that its request held before the call (read from the table, which this call
// leaves alone there) or the free page whose place in the list the scan gives.
// A work-group then writes its own range of tokens, and its share of the new
// table entries.
#include "kv4.h"
#include "kv_scan.h"

namespace qmx {
namespace {

constexpr int THREADS = 512;
constexpr int EACH = 4;                // requests of a thread at a time
constexpr int CHUNK = EACH * THREADS;
constexpr int WAVES = THREADS / 64;

// Numbers up to 2^32 - 1 by the page size: a shift where that is a power of two.
struct Pages {
    uint32_t size;
    int shift;   // or -1
    __device__ __forceinline__ uint32_t whole(uint32_t x) const { return shift >= 0 ? x >> shift : x / size; }
    __device__ __forceinline__ uint32_t count(uint32_t x) const { return whole(x) + (whole(x) * size != x ? 1 : 0); }
};

__global__ __launch_bounds__(THREADS) void kv_maps_kernel(KvMapsArgs a, int per_group, int shift) {
    __shared__ int s_end[CHUNK], s_page_end[CHUNK], s_past[CHUNK], s_held[CHUNK];
    __shared__ int s_waves[2][WAVES];
    const Pages page{(uint32_t)a.page_size, shift};
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
            const int r = r0 + EACH * tid + i;
            n[i] = r < a.requests ? max(a.fresh[r], 0) : 0;
            past[i] = r < a.requests ? max(a.past[r], 0) : 0;
        }
    };
    read(0);
    for (int r0 = 0; r0 < a.requests; r0 += CHUNK) {
        const int count = min(CHUNK, a.requests - r0);
        const int begin = min(sum, a.tokens);
        int mine = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) mine = add_held(mine, n[i]);
        int chunk_sum;
        const int upto = scan_group<WAVES>(mine, s_waves[0], chunk_sum);
        // exclusive, from the inclusive sum of the thread before (a difference of held sums would not do)
        int e = __shfl_up(upto, 1, 64);
        if ((tid & 63) == 0) {
            e = 0;
            for (int w = 0; w < tid >> 6; ++w) e = add_held(e, s_waves[0][w]);
        }
        e = add_held(e, sum);
        int take[EACH], takes = 0, end[EACH], held[EACH];
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int start = min(e, a.tokens);
            e = add_held(e, n[i]);
            end[i] = min(e, a.tokens);
            const uint32_t kv = (uint32_t)past[i] + (uint32_t)(end[i] - start);
            held[i] = (int)min(page.count((uint32_t)past[i]), (uint32_t)a.columns);
            take[i] = (int)min(page.count(kv), (uint32_t)a.columns) - held[i];
            takes += take[i];
            const int r = EACH * tid + i;
            if (first && r < count) {
                a.offsets[r0 + r + 1] = end[i];
                a.kv_lens[r0 + r] = (int)min(kv, 0x7fffffffu);
            }
        }
        int chunk_pages;
        int page_end = pages + scan_group<WAVES>(takes, s_waves[1], chunk_pages) - takes;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int r = EACH * tid + i;
            page_end += take[i];
            s_end[r] = end[i];
            s_page_end[r] = page_end;
            s_past[r] = past[i];
            s_held[r] = held[i];
        }
        if (r0 + CHUNK < a.requests) read(r0 + CHUNK);
        __syncthreads();
        const int stop = s_end[count - 1];
        for (int t = max(t0, begin) + tid; t < min(t1, stop); t += THREADS) {
            const int r = first_after(s_end, count, t);
            const int start = r ? s_end[r - 1] : begin;
            const uint32_t at = (uint32_t)s_past[r] + (uint32_t)(t - start);
            const uint32_t col = page.whole(at);
            long long slot = -1;
            if (col < (uint32_t)a.columns) {
                long long p;
                if ((int)col < s_held[r]) {
                    p = a.table[(r0 + r) * a.table_stride + col];
                } else {
                    const long long place = (long long)(r ? s_page_end[r - 1] : pages) + ((int)col - s_held[r]);
                    p = place < a.num_free ? a.free_pages[place] : -1;
                }
                if (p >= 0) slot = p * a.page_size + (at - col * page.size);
                if (slot > 0x7fffffffll) slot = -1;
            }
            a.slots[t] = (int)slot;
            a.positions[t] = (int)min(at, 0x7fffffffu);
            a.request_ids[t] = r0 + r;
        }
        for (long long p = (long long)pages + blockIdx.x * THREADS + tid; p < (long long)pages + chunk_pages;
             p += gridDim.x * THREADS) {
            const int r = first_after(s_page_end, count, (int)p);
            const int j = (int)p - (r ? s_page_end[r - 1] : pages);
            a.table[(r0 + r) * a.table_stride + s_held[r] + j] = p < a.num_free ? a.free_pages[p] : -1;
        }
        sum = add_held(sum, chunk_sum);
        pages += chunk_pages;
        __syncthreads();
    }
    for (int t = max(t0, min(sum, a.tokens)) + tid; t < t1; t += THREADS) {
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
    long long groups = ((long long)a.tokens + 2 * THREADS - 1) / (2 * THREADS);
    groups = groups < 1 ? 1 : groups > 512 ? 512 : groups;
    int shift = -1;
    if ((a.page_size & (a.page_size - 1)) == 0)
        for (shift = 0; (1 << shift) < a.page_size;) ++shift;
    const int per_group = (int)(((long long)a.tokens + groups - 1) / groups);
    kv_maps_kernel<<<dim3((unsigned)groups), dim3(THREADS), 0, st>>>(a, per_group, shift);
    return hipGetLastError();
}

}  // namespace qmx
