// Page tables, slots and positions of a step's new tokens from the requests'
// lengths (nvfp4_kv_plan).
//
//   total_b = cached_b + new_b,  held_b = ceil(cached_b / p),  want_b = ceil(total_b / p)
//   end_b = sum_{a <= b} new_a,  need_b = want_b - held_b (0 for a request that cannot fit)
//   request b gets the entries held_b .. want_b - 1 from
//   free_pages[head + sum_{a < b} need_a ..]; row end_{b-1} + i holds its token
//   cached_b + i, whose slot is table[b][pos / p] * p + pos % p.
//
// A request is granted when its lengths are not negative, its pages fit the
// table's row, its rows fit the step and its pages the list, in the requests'
// order: pages of requests that are refused for the list's end still count, so
// every request after the first refused one that needs a page is refused too
// and the granted ones are a scan's prefix.
//
// What bounds it is latency: loads, two scans over the requests, a search and
// one table entry a row.  Up to kPlanLds requests every workgroup makes the
// scans for itself and then writes its rows from LDS (k_plan with ROWS), which
// costs less than the second launch that sharing them would.  Where an output
// is an input's memory only one workgroup may run, or a launch for the scans and
// one for the rows (k_plan, k_plan_rows); the latter also for more requests.
// Measured in a graph: 16 requests of a token each 3.9 us, 257 with 16384 rows
// 7.5, 600 prompts with 131072 rows 7.8 (1.7 MB: 0.2 TB/s).
// Sums are 32 bits wide and saturate above all limits (T, F < 2^30), divisions
// by the page size are multiplications.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

constexpr int kPlanItems = 4;                    // requests a thread and round of the scans
constexpr int kPlanMaxThreads = 1024;
constexpr int kPlanLds = kPlanMaxThreads * kPlanItems;   // requests whose ends are searched in LDS
constexpr int kPlanRows = 256;                   // rows of a workgroup of k_plan_rows
constexpr uint32_t kPlanMost = 0x7FFFFFFFu;      // where sums saturate

struct PlanArgs {
    const int32_t* cached;
    const int32_t* fresh;
    int32_t* table;
    int64_t ld_table;
    const int32_t* free_pages;
    const int32_t* head;
    int32_t* slots;
    int32_t* positions;
    int32_t* requests;
    int32_t* lengths;    // may be cached
    int32_t* offsets;
    int32_t* head_out;   // may be head
    int2* seen;          // [B] workspace: (a request's first place in free_pages or -1 if refused, its cached tokens)
    int64_t F;
    int64_t page_limit;  // pages below it have slots below 2^31
    int B, width, page, T;
    uint32_t page_magic;   // t / page = umulhi(t, magic) >> shift for t < 2^31; magic 0: page 1
    int page_shift;
    __device__ __forceinline__ int pages_of(int t) const {
        return page_magic ? (int)(__umulhi((uint32_t)t, page_magic) >> page_shift) : t;
    }
};

__device__ __forceinline__ uint32_t plan_add(uint32_t a, uint32_t b) {
    const uint32_t s = a + b;   // both at most kPlanMost
    return s < kPlanMost ? s : kPlanMost;
}

// Saturating scan over the workgroup's threads: the sum of the v before this
// one's; total in all of them.  Ends with a barrier, so that sums may be used again at once.
template <int THREADS>
__device__ __forceinline__ uint32_t plan_scan(uint32_t v, uint32_t* sums, uint32_t& total) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(v, d);
        if (lane >= d) v = plan_add(v, o);
    }
    if (lane == 63) sums[w] = v;
    v = __shfl_up(v, 1);
    if (lane == 0) v = 0;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) {
        const uint32_t s = sums[i];
        before = i < w ? plan_add(before, s) : before;
        total = plan_add(total, s);
    }
    __syncthreads();
    return plan_add(before, v);
}

// Row t: its request by a search of ends (ends[b] = offsets[b + 1], ascending),
// then its slot and position; the first token of a page enters the page into
// the table.  A page begun by a new token is new: pages that are held begin
// with cached tokens.
__device__ __forceinline__ void plan_row(const PlanArgs& a, int t, const int32_t* ends, const int2* seen) {
    int lo = 0, hi = a.B;   // the first request whose end is past t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > t) hi = mid;
        else lo = mid + 1;
    }
    int slot = -1, pos = 0, request = -1;
    if (lo < a.B) {
        const int2 s = seen[lo];
        if (s.x >= 0) {
            const int begin = lo ? ends[lo - 1] : 0;
            pos = s.y + (t - begin);
            request = lo;
            const int entry = a.pages_of(pos), in = pos - entry * a.page;
            const int held = a.pages_of(s.y + a.page - 1);
            int32_t* at = a.table + (int64_t)lo * a.ld_table + entry;
            int page;
            if (entry < held) {
                page = *at;
            } else {
                page = a.free_pages[(int64_t)s.x + (entry - held)];
                if (in == 0) *at = page;
            }
            if (page >= 0 && page < a.page_limit) slot = page * a.page + in;
        }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
    a.requests[t] = request;
}

// ROWS: the rows too (B <= THREADS * kPlanItems), all workgroups' together; else
// they are k_plan_rows's.
template <int THREADS, bool ROWS>
__global__ void __launch_bounds__(THREADS) k_plan(PlanArgs a) {
    constexpr int kChunk = THREADS * kPlanItems;
    __shared__ uint32_t sums[THREADS / 64];
    __shared__ int32_t s_ends[ROWS ? kChunk : 1];
    __shared__ int2 s_seen[ROWS ? kChunk : 1];
    __shared__ uint32_t s_given;   // pages granted: they are a prefix of what is wanted
    const int tid = threadIdx.x;
    const int32_t start = a.head[0];
    const uint32_t head = start > 0 ? (uint32_t)start : 0u;
    if (tid == 0) s_given = 0;
    uint32_t tokens = 0, pages = 0;   // of the rounds before
    for (int b0 = 0; b0 < a.B; b0 += kChunk) {
        int32_t cached[kPlanItems], fresh[kPlanItems];
        uint32_t need[kPlanItems], end[kPlanItems];
        bool fits[kPlanItems];
        uint32_t sum = 0, total;
#pragma unroll
        for (int i = 0; i < kPlanItems; ++i) {
            const int b = b0 + tid * kPlanItems + i;
            cached[i] = b < a.B ? a.cached[b] : 0;
            fresh[i] = b < a.B ? a.fresh[b] : 0;
        }
#pragma unroll
        for (int i = 0; i < kPlanItems; ++i) sum = plan_add(sum, fresh[i] > 0 ? (uint32_t)fresh[i] : 0u);
        uint32_t run = plan_add(tokens, plan_scan<THREADS>(sum, sums, total));
        tokens = plan_add(tokens, total);
        sum = 0;
#pragma unroll
        for (int i = 0; i < kPlanItems; ++i) {
            run = plan_add(run, fresh[i] > 0 ? (uint32_t)fresh[i] : 0u);
            end[i] = run;
            // a table's row holds fewer than 2^30 tokens
            const uint32_t all = (uint32_t)cached[i] + (uint32_t)fresh[i];
            fits[i] = cached[i] >= 0 && fresh[i] >= 0 && all < (1u << 30) && run <= (uint32_t)a.T;
            const int want = fits[i] ? a.pages_of((int)all + a.page - 1) : 0;
            fits[i] = fits[i] && want <= a.width;
            need[i] = fits[i] ? (uint32_t)(want - a.pages_of(cached[i] + a.page - 1)) : 0u;
            sum = plan_add(sum, need[i]);
        }
        run = plan_add(pages, plan_scan<THREADS>(sum, sums, total));
        pages = plan_add(pages, total);
        uint32_t given = 0;
#pragma unroll
        for (int i = 0; i < kPlanItems; ++i) {
            const int b = b0 + tid * kPlanItems + i;
            const uint32_t first = plan_add(head, run);
            run = plan_add(run, need[i]);
            const bool granted = fits[i] && (need[i] == 0 || plan_add(head, run) <= (uint32_t)a.F);
            if (granted && need[i]) given = run;
            if (b < a.B) {
                const int e = end[i] < (uint32_t)a.T ? (int)end[i] : a.T;
                const int2 s = make_int2(granted ? (need[i] ? (int)first : 0) : -1, granted ? cached[i] : 0);
                if (blockIdx.x == 0) {
                    a.offsets[b + 1] = e;
                    a.lengths[b] = granted ? cached[i] + fresh[i] : cached[i] > 0 ? cached[i] : 0;
                }
                if (ROWS) {
                    s_ends[b] = e;
                    s_seen[b] = s;
                } else {
                    a.seen[b] = s;
                }
            }
        }
        if (given) atomicMax(&s_given, given);
    }
    __syncthreads();   // every thread has read head; the lists in LDS
    if (blockIdx.x == 0 && tid == 0) {
        a.offsets[0] = 0;
        a.head_out[0] = (int32_t)(head + s_given);
    }
    if (ROWS)
        for (int64_t t = (int64_t)blockIdx.x * THREADS + tid; t < a.T; t += (int64_t)gridDim.x * THREADS)
            plan_row(a, (int)t, s_ends, s_seen);
}

__global__ void __launch_bounds__(kPlanRows) k_plan_rows(PlanArgs a) {
    __shared__ int32_t s_ends[kPlanLds];
    const bool near = a.B <= kPlanLds;   // the ends in LDS: a search costs 12 of its reads, not 12 of the L2's
    if (near) {
        for (int b = threadIdx.x; b < a.B; b += kPlanRows) s_ends[b] = a.offsets[b + 1];
        __syncthreads();
    }
    const int t = blockIdx.x * kPlanRows + threadIdx.x;
    if (t < a.T) plan_row(a, t, near ? s_ends : a.offsets + 1, a.seen);
}

}  // namespace nvfp4
