// kv4_units.h -- which rows and keys a work-group of an attention call takes,
// and the kernel that joins what was cut (kv4.h describes the cut).
#pragma once

#include "kv4.h"
#include "kv_scan.h"
#include "qmx_device.h"

namespace qmx {
namespace kv4 {

constexpr float LN2 = 0.69314718055994530942f;

typedef float f32x2 __attribute__((ext_vector_type(2)));

// The number of block `blk` of a request's tokens, which is in the page given.  32
// bits hold it: 2^32 blocks of the smallest head would be 4 TB.
__device__ __forceinline__ uint32_t block_number(const Kv4View& c, int page, int head, int blk) {
    return (((uint32_t)page * c.heads + head) << c.page_shift) + (blk & ((1 << c.page_shift) - 1));
}

// Rows and keys of one unit, or of the part of it that a work-group takes.
struct Unit {
    int req;
    int start, back;          // the request's first token, and that token's position
    int row0, rows;           // of the request's rows
    int end;                  // keys from here on are not there
    int step, steps;          // the keys, 32 a step
    int full_lo, full_hi;     // keys that every row sees
    int place;                // of the partial sums, or -1: the unit is whole
};

// Unit `v` of a head, from what memory holds: steps is 0 where no key is seen.
__device__ __forceinline__ Unit unit_of(const Kv4AttnArgs& a, int v) {
    Unit u;
    u.req = v / a.p.tiles;
    const int tile = a.p.tiles - 1 - (v - u.req * a.p.tiles);   // the tiles that see most keys first
    u.start = max(a.offsets[u.req], 0);
    const int stop = a.offsets[u.req + 1], kv = a.kv_lens[u.req];
    const int count = min(min(stop, a.tokens) - u.start, a.max_query);
    u.back = kv - (stop - u.start);
    u.row0 = tile * a.p.rows;
    u.rows = min(count * a.each - u.row0, a.p.rows);
    u.place = -1;
    u.step = u.steps = 0;
    u.end = u.full_lo = u.full_hi = 0;
    if (u.rows > 0) {
        const int pos0 = u.back + u.row0 / a.each, pos1 = u.back + (u.row0 + u.rows - 1) / a.each;
        u.end = min(min(kv, a.max_kv), pos1 + 1);
        const int first = a.window ? max(0, pos0 - a.window + 1) : 0;
        u.step = first >> 5;
        u.steps = max(0, ((u.end + 31) >> 5) - u.step);
        u.full_lo = a.window ? pos1 - a.window + 1 : 0;
        u.full_hi = min(pos0, u.end - 1);
    }
    return u;
}

// Zeros for the tokens of no request, before the first offset and from the last
// on, and for a request's tokens past max_query: group `id` of `of`.  In each group a
// wave looks at 64 requests at a time and clears with the others' same wave what is
// past the bound (8191 tokens of 40 heads of 128 take 50 us so, and 138 ms by one lane;
// all waves for each run, which every wave then has to look for, 28 us, but calls
// without such tokens took up to 4 % longer).
__device__ __forceinline__ void clear_rest(const Kv4AttnArgs& a, int id, int of) {
    const long long thread = (long long)id * blockDim.x + threadIdx.x, threads = (long long)of * blockDim.x;
    const int first = min(max(a.offsets[0], 0), a.tokens), begin = max(a.offsets[a.requests], 0);
    auto clear = [&](long long from, long long to, long long at, long long step) {
        const int per = a.heads * (a.c.dim / 8);
        for (long long i = from * per + at; i < to * per; i += step)
            reinterpret_cast<u32x4*>(a.out)[i] = u32x4{0, 0, 0, 0};
        if (a.lse)
            for (long long i = from * a.heads + at; i < to * a.heads; i += step) a.lse[i] = -INFINITY;
    };
    clear(0, first, thread, threads);
    clear(begin, a.tokens, thread, threads);
    const int lane = threadIdx.x & 63;
    for (int r0 = threadIdx.x & ~63; r0 < a.requests; r0 += blockDim.x) {
        const int r = min(r0 + lane, a.requests - 1);
        const int from = min(max(a.offsets[r], 0), a.tokens - a.max_query) + a.max_query;
        const int to = min(a.offsets[r + 1], a.tokens);
        for (unsigned long long which = __ballot(r == r0 + lane && from < to); which; which &= which - 1) {
            const int owner = __ffsll(which) - 1;
            clear(__shfl(from, owner, 64), __shfl(to, owner, 64), 64 * id + lane, 64ll * of);
        }
    }
}

// Whether work-group `id` of a head is the one behind the units, which clears.
__device__ __forceinline__ bool clears(const Kv4AttnArgs& a, int id, int head) {
    if (a.p.lines || id < a.requests * a.p.tiles) return false;
    clear_rest(a, head, a.c.heads);
    return true;
}

// The units of work-group `id` of a head, one after the other.
template <int THREADS>
class Units {
    int id_, count_, at_, stop_;
    int *begin_, *end_;   // LDS: a unit's steps on the line

  public:
    __device__ __forceinline__ Units(const Kv4AttnArgs& a, int id, int head) : id_(id), count_(a.requests * a.p.tiles) {
        constexpr int MOST = kv4_line_units(THREADS / 64);
        __shared__ int s_begin[MOST], s_end[MOST];
        __shared__ int s_waves[1][THREADS / 64];
        begin_ = s_begin;
        end_ = s_end;
        at_ = 0;
        stop_ = 1;
        if (!a.p.lines) return;
        constexpr int EACH = MOST / THREADS;
        int n[EACH], sum = 0;
        const int per = (count_ + THREADS - 1) / THREADS;   // units a thread, at most EACH
        const int v0 = (int)threadIdx.x * per;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const bool there = i < per && v0 + i < count_;
            n[i] = there ? unit_of(a, v0 + i).steps : 0;
            sum += n[i] ? n[i] + a.p.cost : 0;
        }
        int ends[1] = {sum}, totals[1];
        scan_group<THREADS / 64>(ends, s_waves, totals);
        int upto = ends[0];
        const int total = totals[0];
        const int length = max(a.p.least, (total + a.p.lines - 1) / a.p.lines);
        const bool tell = id == 0 && head == 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            if (i < per && v0 + i < count_) {
                const int begin = upto + (n[i] ? a.p.cost : 0);
                upto = begin + n[i];
                s_begin[v0 + i] = begin;
                s_end[v0 + i] = upto;
                if (tell) {
                    a.pos[1 + 2 * (v0 + i)] = begin;
                    a.pos[2 + 2 * (v0 + i)] = upto;
                }
            }
        }
        if (tell && threadIdx.x == 0) a.pos[0] = length;
        __syncthreads();
        at_ = (int)min((long long)id * length, (long long)total);
        stop_ = (int)min((long long)at_ + length, (long long)total);
    }

    // Whether there is another; uniform over the work-group.
    __device__ __forceinline__ bool next(const Kv4AttnArgs& a, Unit& u) {
        if (at_ >= stop_) return false;
        if (!a.p.lines) {
            at_ = stop_;
            u = unit_of(a, id_);
            return u.rows > 0;
        }
        const int v = __builtin_amdgcn_readfirstlane(first_after(end_, count_, at_));
        const int begin = __builtin_amdgcn_readfirstlane(begin_[v]), end = __builtin_amdgcn_readfirstlane(end_[v]);
        if (stop_ <= begin) return false;   // only the gap before the unit
        u = unit_of(a, v);
        const int first = max(at_, begin), last = min(end, stop_);
        u.step += first - begin;
        u.steps = last - first;
        if (first > begin) u.place = 2 * id_;
        else if (last < end) u.place = 2 * id_ + 1;
        at_ = last;
        return true;
    }
};

// Work-groups of a call: the units of a head and one for the rest, or the lines.
inline long long kv4_groups(const Kv4AttnArgs& a) {
    return (long long)a.c.heads * (a.p.lines ? a.p.lines : (long long)a.requests * a.p.tiles + 1);
}

// The parts of a unit's row, in the order of the line: their places, and what
// they add up to.
struct Parts {
    int first, last;   // parts of the line; last < first: no key is seen
    long long row;     // of all rows of a part
    long long all;
    __device__ __forceinline__ long long place(int w) const {
        return (2ll * w + (w == first ? 1 : 0)) * all + row;
    }
};
__device__ __forceinline__ Parts parts_of(const Kv4AttnArgs& a, int v, int kv_head, int row) {
    const int length = a.pos[0], p0 = a.pos[1 + 2 * v], p1 = a.pos[2 + 2 * v];
    const int first = p0 / length;
    return {first, p1 > p0 ? (p1 - 1) / length : first - 1, (long long)kv_head * a.p.rows + row,
            (long long)a.c.heads * a.p.rows};
}

// A finished row's four values of a thread, and its log-sum-exp.
template <int D, int DT>
__device__ __forceinline__ void store_row(const Kv4AttnArgs& a, long long at, int lane, f32x4 o, float l, float safe) {
    o *= l != 0.0f ? 1.0f / l : 0.0f;
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = DT == DT_F16 ? f32_to_f16_bits(o[e]) : f32_to_bf16_bits(o[e]);
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at * D + 4 * lane) =
        u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
    if (a.lse && lane == 0) a.lse[at] = l != 0.0f ? (safe + __builtin_amdgcn_logf(l)) * LN2 : -INFINITY;
}

// Joins the parts of few rows' units, writes zeros where no key is seen, and
// leaves alone what is whole.  A work-group takes a row (token of a request,
// head), which may have as many parts as there are lines: D / 4 threads side by
// side, and as many such sets as there are, each every so many parts.
template <int D, int DT>
__global__ __launch_bounds__(256) void kv4_join_kernel(Kv4AttnArgs a) {
    constexpr int LANES = D / 4, SETS = 256 / LANES;
    __shared__ f32x4 s_o[256];
    __shared__ float s_l[SETS];
    const int own = a.requests * a.max_query * a.heads;   // the groups behind these take the tokens of no request
    if ((int)blockIdx.x >= own) {
        clear_rest(a, blockIdx.x - own, gridDim.x - own);
        return;
    }
    const int lane = threadIdx.x % LANES, set = threadIdx.x / LANES;
    const int head = blockIdx.x % a.heads, t = blockIdx.x / a.heads, req = t / a.max_query, i = t - req * a.max_query;
    const int start = max(a.offsets[req], 0);
    if (i >= a.offsets[req + 1] - start || start + i >= a.tokens) return;
    const int row = i * a.each + head % a.each, tile = row / a.p.rows;
    const Parts parts = parts_of(a, req * a.p.tiles + a.p.tiles - 1 - tile, head / a.each, row - tile * a.p.rows);
    if (parts.first == parts.last) return;
    const f32x2* stat = reinterpret_cast<const f32x2*>(a.stat);
    // the largest maximum first: the sets' sums then just add
    float m = -INFINITY, l = 0.0f;
    for (int w = parts.first + (int)(threadIdx.x & 63); w <= parts.last; w += 64) m = fmaxf(m, stat[parts.place(w)][0]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    const float safe = m > -INFINITY ? m : 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int w = parts.first + set; w <= parts.last; w += SETS) {
        const long long p = parts.place(w);
        const f32x2 st = stat[p];
        const float f = __builtin_amdgcn_exp2f(st[0] - safe);
        l += st[1] * f;
        o += *reinterpret_cast<const f32x4*>(a.part + p * D + 4 * lane) * f;
    }
    s_o[threadIdx.x] = o;
    if (lane == 0) s_l[set] = l;
    __syncthreads();
    if (set) return;
#pragma unroll
    for (int s = 1; s < SETS; ++s) {
        o += s_o[s * LANES + lane];
        l += s_l[s];
    }
    store_row<D, DT>(a, ((long long)start + i) * a.heads + head, lane, o, l, safe);
}

// The same for the many rows of a prompt's units, which have few parts: a
// work-group takes JOIN_ROWS rows of a unit, so that one look tells it that they
// are whole.
constexpr int JOIN_ROWS = 32;
template <int D, int DT>
__global__ __launch_bounds__(256) void kv4_join_prompt_kernel(Kv4AttnArgs a) {
    constexpr int LANES = D / 4, ABREAST = 256 / LANES;
    const int slices = a.p.rows / JOIN_ROWS, own = a.requests * a.p.tiles * a.c.heads * slices;
    if ((int)blockIdx.x >= own) {
        clear_rest(a, blockIdx.x - own, gridDim.x - own);
        return;
    }
    const int slice = blockIdx.x % slices, kv_head = blockIdx.x / slices % a.c.heads;
    const int v = blockIdx.x / slices / a.c.heads, req = v / a.p.tiles;
    const int tile = a.p.tiles - 1 - (v - req * a.p.tiles), lane = threadIdx.x % LANES;
    const int start = max(a.offsets[req], 0);
    const int count = min(min(a.offsets[req + 1], a.tokens) - start, a.max_query);
    const int rows = min(count * a.each - tile * a.p.rows, a.p.rows);
    Parts parts = parts_of(a, v, kv_head, 0);
    if (parts.first == parts.last) return;
    const f32x2* stat = reinterpret_cast<const f32x2*>(a.stat);
    const long long row0 = parts.row;
#pragma unroll 4
    for (int r = slice * JOIN_ROWS + threadIdx.x / LANES; r < min(rows, (slice + 1) * JOIN_ROWS); r += ABREAST) {
        parts.row = row0 + r;
        float m = -INFINITY, l = 0.0f;
        for (int w = parts.first; w <= parts.last; ++w) m = fmaxf(m, stat[parts.place(w)][0]);
        const float safe = m > -INFINITY ? m : 0.0f;
        f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int w = parts.first; w <= parts.last; ++w) {
            const long long p = parts.place(w);
            const f32x2 st = stat[p];
            const float f = st[1] * __builtin_amdgcn_exp2f(st[0] - safe);   // the part is over its sum
            l += f;
            o += *reinterpret_cast<const f32x4*>(a.part + p * D + 4 * lane) * f;
        }
        const int row = tile * a.p.rows + r, i = row / a.each;
        store_row<D, DT>(a, ((long long)start + i) * a.heads + kv_head * a.each + row - i * a.each, lane, o, l, safe);
    }
}

template <int D, int DT>
hipError_t launch_join(const Kv4AttnArgs& a, hipStream_t st) {
    const long long rest = 1 + ((long long)a.tokens * a.heads * (D / 8) >> 12);   // 16 stores a thread
    const unsigned behind = (unsigned)(rest < 64 ? rest : 64);
    if (a.p.rows > 16)
        kv4_join_prompt_kernel<D, DT><<<(unsigned)(a.requests * a.p.tiles * a.c.heads * (a.p.rows / JOIN_ROWS)) + behind,
                                        256, 0, st>>>(a);
    else
        kv4_join_kernel<D, DT><<<(unsigned)(a.requests * a.max_query * a.heads) + behind, 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace kv4
}  // namespace qmx
