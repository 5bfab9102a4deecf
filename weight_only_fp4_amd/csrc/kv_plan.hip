// C ABI of the page tables and slots of a step (include/nvfp4_w4a16.h).
#include <hip/hip_runtime.h>

#include "../../include/nvfp4_w4a16.h"
#include "kernels_plan.h"
#include "plan.h"

using namespace nvfp4;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMost = (int64_t)1 << 30;   // requests, rows and tokens of a table's row stay below

// Rows that one workgroup writes alone where an output is an input's memory (16
// rows: 3.9 us, by two launches 5.5; 1024: 5.8 and 5.9; 4096: 11.2 and 5.9).
constexpr int64_t kPlanAlone = 1024;

// Whether the call may take two launches, by its sizes alone (the workspace
// is for them).
bool may_share(int64_t B, int64_t T) { return B > kPlanLds || T > kPlanAlone; }

template <int THREADS>
void launch_whole(const PlanArgs& a, bool alone, hipStream_t st) {
    // two rows a thread: half as many scans as with one
    const int64_t groups = ((int64_t)a.T + 2 * THREADS - 1) / (2 * THREADS);
    hipLaunchKernelGGL((k_plan<THREADS, true>), dim3(alone || groups < 1 ? 1u : (unsigned)groups), dim3(THREADS), 0, st, a);
}

}  // namespace

extern "C" {

int64_t nvfp4_kv_plan_workspace_bytes(int64_t B, int64_t T) {
    if (B < 0 || B >= kMost || T < 0 || T >= kMost) {
        fail(NVFP4_ERR_INVALID_ARG, "nvfp4_kv_plan_workspace_bytes: B = %lld, T = %lld", (long long)B, (long long)T);
        return -1;
    }
    return may_share(B, T) ? B * (int64_t)sizeof(int2) : 0;
}

nvfp4_status nvfp4_kv_plan(const int32_t* cached, const int32_t* fresh, int64_t B, int32_t* page_table, int64_t ld_table,
                           int64_t max_pages, int64_t page_size, const int32_t* free_pages, int64_t F, const int32_t* head,
                           int64_t T, int32_t* slots, int32_t* positions, int32_t* requests, int32_t* lengths,
                           int32_t* offsets, int32_t* head_out, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "nvfp4_kv_plan";
    if (B < 0 || B >= kMost || T < 0 || T >= kMost)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: B = %lld, T = %lld must be in [0, 2^30)", fn, (long long)B, (long long)T);
    if (page_size < 1 || page_size >= kMost || max_pages < 0 || max_pages >= kMost || max_pages * page_size >= kMost)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: max_pages = %lld of page_size = %lld: a table's row must hold fewer than 2^30 tokens",
                    fn, (long long)max_pages, (long long)page_size);
    if (ld_table < max_pages || ld_table >= (int64_t)1 << 40)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: ld_table = %lld < max_pages = %lld or too large", fn, (long long)ld_table,
                    (long long)max_pages);
    if (F < 0 || F >= kMost) return fail(NVFP4_ERR_INVALID_ARG, "%s: F = %lld free pages", fn, (long long)F);
    if (!head || !head_out || !offsets || (F > 0 && !free_pages) || (B > 0 && (!cached || !fresh || !lengths)) ||
        (B > 0 && max_pages > 0 && !page_table) || (T > 0 && (!slots || !positions || !requests)))
        return fail(NVFP4_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    const void* all[] = {cached, fresh, page_table, free_pages, head, slots, positions, requests, lengths, offsets, head_out};
    for (const void* p : all)
        if (!aligned(p, 4)) return fail(NVFP4_ERR_ALIGNMENT, "%s: int32 arrays must be 4-byte aligned", fn);
    const int64_t need = nvfp4_kv_plan_workspace_bytes(B, T);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(NVFP4_ERR_BUFFER_TOO_SMALL, "%s: workspace of %lld bytes is below the %lld bytes this call needs", fn,
                        (long long)workspace_bytes, (long long)need);
        if (!aligned(workspace, 8)) return fail(NVFP4_ERR_ALIGNMENT, "%s: workspace must be 8-byte aligned", fn);
    }
    PlanArgs a;
    a.cached = cached;
    a.fresh = fresh;
    a.table = page_table;
    a.ld_table = ld_table;
    a.free_pages = free_pages;
    a.head = head;
    a.slots = slots;
    a.positions = positions;
    a.requests = requests;
    a.lengths = lengths;
    a.offsets = offsets;
    a.head_out = head_out;
    a.seen = static_cast<int2*>(workspace);
    a.F = F;
    a.page_limit = ((int64_t)1 << 31) / page_size;
    a.B = (int)B;
    a.width = (int)max_pages;
    a.page = (int)page_size;
    a.T = (int)T;
    // umulhi(t, ceil(2^(32 + s) / page_size)) >> s is t / page_size for t < 2^31 with 2^s < page_size <= 2^(s + 1)
    a.page_shift = 0;
    while ((int64_t)2 << a.page_shift < page_size) ++a.page_shift;
    a.page_magic = page_size == 1 ? 0u
                   : (uint32_t)((((uint64_t)1 << (32 + a.page_shift)) + (uint64_t)page_size - 1) / (uint64_t)page_size);
    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool in_place = lengths == cached || head_out == head;
    if (B <= kPlanLds && (!in_place || T <= kPlanAlone)) {
        // few requests: fewer waves to wait for at each barrier (16 requests 3.9
        // us with 64 threads, 4.2 with 256; 64: 4.15 and 4.35; 200: 5.4 and 4.7)
        if (B <= 64 && T <= 256) launch_whole<64>(a, in_place, st);
        else if (B <= 256 * kPlanItems) launch_whole<256>(a, in_place, st);
        else launch_whole<kPlanMaxThreads>(a, in_place, st);
        return launched(fn);
    }
    // offsets and the workspace are written here, for the rows' launch
    if (B <= 256 * kPlanItems) hipLaunchKernelGGL((k_plan<256, false>), dim3(1), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_plan<kPlanMaxThreads, false>), dim3(1), dim3(kPlanMaxThreads), 0, st, a);
    const nvfp4_status s = launched(fn);
    if (s != NVFP4_OK || T == 0) return s;
    hipLaunchKernelGGL(k_plan_rows, dim3((unsigned)((T + kPlanRows - 1) / kPlanRows)), dim3(kPlanRows), 0, st, a);
    return launched(fn);
}

}  // extern "C"
