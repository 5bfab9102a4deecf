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
// What bounds it is latency: two scans over the requests, a search and one
// table entry a row.  One workgroup does the scans (k_plan); with few rows it
// goes on to write them in the same launch, from LDS, and with more a second
// launch of a workgroup per kPlanRows rows does (k_plan_rows), which no
// barrier across workgroups could do faster than the launch's 2 us.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

constexpr int kPlanThreads = 1024;
constexpr int kPlanItems = 4;                             // requests a thread and round of the scans
constexpr int kPlanChunk = kPlanThreads * kPlanItems;
constexpr int kPlanLds = kPlanChunk;                      // requests whose ends are searched in LDS
constexpr int kPlanRows = 1024;                           // rows of a workgroup of k_plan_rows

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
};

// Inclusive scan of v over the workgroup's threads; total in all of them.  Ends
// with a barrier, so that sums may be used again at once.
__device__ __forceinline__ int64_t plan_scan(int64_t v, int64_t* sums, int64_t& total) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    if (lane == 63) sums[w] = v;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kPlanThreads / 64; ++i) {
        const int64_t s = sums[i];
        before += i < w ? s : 0;
        total += s;
    }
    __syncthreads();
    return before + v;
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
            const int entry = pos / a.page, in = pos - entry * a.page;
            const int held = (s.y + a.page - 1) / a.page;
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

// ROWS: the rows too (B <= kPlanLds); else they are k_plan_rows's.
template <bool ROWS>
__global__ void __launch_bounds__(kPlanThreads) k_plan(PlanArgs a) {
    __shared__ int64_t sums[kPlanThreads / 64];
    __shared__ int32_t s_ends[ROWS ? kPlanLds : 1];
    __shared__ int2 s_seen[ROWS ? kPlanLds : 1];
    const int tid = threadIdx.x;
    int64_t head = a.head[0];
    if (head < 0) head = 0;
    int64_t tokens = 0, pages = 0, given = 0;   // rows and pages of the rounds before, pages granted
    for (int b0 = 0; b0 < a.B; b0 += kPlanChunk) {
        int64_t cached[kPlanItems], fresh[kPlanItems], end[kPlanItems], need[kPlanItems];
        bool fits[kPlanItems];
        int64_t sum = 0;
#pragma unroll
        for (int i = 0; i < kPlanItems; ++i) {
            const int b = b0 + tid * kPlanItems + i;
            cached[i] = b < a.B ? a.cached[b] : 0;
            fresh[i] = b < a.B ? a.fresh[b] : 0;
            fits[i] = cached[i] >= 0 && fresh[i] >= 0;
            sum += fresh[i] > 0 ? fresh[i] : 0;
        }
        int64_t total;
        int64_t run = tokens + plan_scan(sum, sums, total) - sum;
        tokens += total;
        sum = 0;
#pragma unroll
        for (int i = 0; i < kPlanItems; ++i) {
            run += fresh[i] > 0 ? fresh[i] : 0;
            end[i] = run;
            // below 2^30 where it counts: the table holds fewer tokens
            const int64_t want = (cached[i] + fresh[i] + a.page - 1) / a.page;
            fits[i] = fits[i] && want <= a.width && run <= a.T;
            need[i] = fits[i] ? want - (cached[i] + a.page - 1) / a.page : 0;
            sum += need[i];
        }
        run = pages + plan_scan(sum, sums, total) - sum;
        pages += total;
        int64_t mine = 0;
#pragma unroll
        for (int i = 0; i < kPlanItems; ++i) {
            const int b = b0 + tid * kPlanItems + i;
            const int64_t first = head + run;
            run += need[i];
            const bool granted = fits[i] && (need[i] == 0 || head + run <= a.F);
            if (granted) mine += need[i];
            if (b < a.B) {
                const int e = (int)(end[i] < a.T ? end[i] : a.T);
                // a granted request without new pages has no place in the list: 0 stands for it
                const int2 s = make_int2(granted ? (need[i] ? (int)first : 0) : -1, granted ? (int)cached[i] : 0);
                a.offsets[b + 1] = e;
                a.lengths[b] = (int)(granted ? cached[i] + fresh[i] : cached[i] > 0 ? cached[i] : 0);
                if (ROWS) {
                    s_ends[b] = e;
                    s_seen[b] = s;
                } else {
                    a.seen[b] = s;
                }
            }
        }
        plan_scan(mine, sums, total);
        given += total;
    }
    __syncthreads();   // every thread has read head
    if (tid == 0) {
        a.offsets[0] = 0;
        a.head_out[0] = (int32_t)(head + given);
    }
    if (ROWS)
        for (int t = tid; t < a.T; t += kPlanThreads) plan_row(a, t, s_ends, s_seen);
}

__global__ void __launch_bounds__(256) k_plan_rows(PlanArgs a) {
    __shared__ int32_t s_ends[kPlanLds];
    const bool near = a.B <= kPlanLds;   // the ends in LDS: a search costs 12 of its reads, not 12 of the L2's
    if (near) {
        for (int b = threadIdx.x; b < a.B; b += 256) s_ends[b] = a.offsets[b + 1];
        __syncthreads();
    }
    const int64_t t0 = (int64_t)blockIdx.x * kPlanRows;
    for (int i = threadIdx.x; i < kPlanRows && t0 + i < a.T; i += 256)
        plan_row(a, (int)(t0 + i), near ? s_ends : a.offsets + 1, a.seen);
}

}  // namespace nvfp4
