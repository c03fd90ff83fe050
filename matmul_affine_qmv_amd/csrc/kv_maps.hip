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
constexpr int CHUNK = 2 * THREADS;   // requests scanned at a time, two a thread
constexpr int WAVES = THREADS / 64;

__global__ __launch_bounds__(THREADS) void kv_maps_kernel(KvMapsArgs a, int per_group) {
    __shared__ int s_end[CHUNK], s_page_end[CHUNK], s_past[CHUNK], s_held[CHUNK];
    __shared__ long long s_waves64[WAVES];
    __shared__ int s_waves32[WAVES];
    const int tid = threadIdx.x;
    const bool first = blockIdx.x == 0;
    const int t0 = (int)min((long long)blockIdx.x * per_group, (long long)a.tokens);
    const int t1 = (int)min((long long)t0 + per_group, (long long)a.tokens);
    long long sum = 0;   // new tokens of the chunks before, not held to the room for them
    int pages = 0;       // pages handed out before
    if (first && tid == 0) a.offsets[0] = 0;
    for (int r0 = 0; r0 < a.requests; r0 += CHUNK) {
        const int count = min(CHUNK, a.requests - r0);
        const int begin = (int)min(sum, (long long)a.tokens);
        long long n[2];
        int past[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * tid + i;
            n[i] = r < count ? max(a.fresh[r0 + r], 0) : 0;
            past[i] = r < count ? max(a.past[r0 + r], 0) : 0;
        }
        long long chunk_sum;
        const long long upto = sum + scan_group<WAVES>(n[0] + n[1], s_waves64, chunk_sum);
        int take[2], held[2], end[2];
        long long e = upto - n[1] - n[0];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int start = (int)min(e, (long long)a.tokens);
            e += n[i];
            end[i] = (int)min(e, (long long)a.tokens);
            const long long kv = (long long)past[i] + (end[i] - start);
            const long long h = ((long long)past[i] + a.page_size - 1) / a.page_size;
            const long long h2 = (kv + a.page_size - 1) / a.page_size;
            held[i] = (int)min(h, (long long)a.columns);
            take[i] = (int)min(h2, (long long)a.columns) - held[i];
            const int r = 2 * tid + i;
            if (first && r < count) {
                a.offsets[r0 + r + 1] = end[i];
                a.kv_lens[r0 + r] = (int)min(kv, 0x7fffffffll);
            }
        }
        int chunk_pages;
        const int page_upto = pages + scan_group<WAVES>(take[0] + take[1], s_waves32, chunk_pages);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * tid + i;
            s_end[r] = end[i];
            s_page_end[r] = page_upto - (i == 0 ? take[1] : 0);
            s_past[r] = past[i];
            s_held[r] = held[i];
        }
        __syncthreads();
        const int stop = s_end[count - 1];
        for (int t = max(t0, begin) + tid; t < min(t1, stop); t += THREADS) {
            const int r = first_after(s_end, count, t);
            const int start = r ? s_end[r - 1] : begin;
            const long long at = (long long)s_past[r] + (t - start);
            const long long col = at / a.page_size;
            long long slot = -1;
            if (col < a.columns) {
                long long page;
                if (col < s_held[r]) {
                    page = a.table[(r0 + r) * a.table_stride + col];
                } else {
                    const long long p = (r ? s_page_end[r - 1] : pages) + col - s_held[r];
                    page = p < a.num_free ? a.free_pages[p] : -1;
                }
                if (page >= 0) slot = page * a.page_size + at % a.page_size;
                if (slot > 0x7fffffffll) slot = -1;
            }
            a.slots[t] = (int)slot;
            a.positions[t] = (int)min(at, 0x7fffffffll);
            a.request_ids[t] = r0 + r;
        }
        for (int p = pages + blockIdx.x * THREADS + tid; p < pages + chunk_pages; p += gridDim.x * THREADS) {
            const int r = first_after(s_page_end, count, p);
            const int j = p - (r ? s_page_end[r - 1] : pages);
            a.table[(r0 + r) * a.table_stride + s_held[r] + j] = p < a.num_free ? a.free_pages[p] : -1;
        }
        sum += chunk_sum;
        pages += chunk_pages;
        __syncthreads();
    }
    const int end = (int)min(sum, (long long)a.tokens);
    for (int t = max(t0, end) + tid; t < t1; t += THREADS) {
        a.slots[t] = -1;
        a.positions[t] = -1;
        a.request_ids[t] = -1;
    }
    if (first && tid == 0) {
        a.counts[0] = (int)min(sum, 0x7fffffffll);
        a.counts[1] = pages;
    }
}

}  // namespace

hipError_t launch_kv_maps(const KvMapsArgs& a, hipStream_t st) {
    long long groups = ((long long)a.tokens + 2 * THREADS - 1) / (2 * THREADS);
    groups = groups < 1 ? 1 : groups > 512 ? 512 : groups;
    const int per_group = (int)(((long long)a.tokens + groups - 1) / groups);
    kv_maps_kernel<<<dim3((unsigned)groups), dim3(THREADS), 0, st>>>(a, per_group);
    return hipGetLastError();
}

}  // namespace qmx
