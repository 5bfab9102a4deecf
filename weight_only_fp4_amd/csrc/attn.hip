// Single-token attention kernels of one cache format (NVFP4_KV_FMT: 0 bf16,
// 1 fp16, 2 E4M3, 3 NVFP4).
#include "attn_plan.h"

#ifndef NVFP4_KV_FMT
#error "compile with -DNVFP4_KV_FMT=0 .. 3"
#endif

namespace nvfp4 {

namespace {

template <int DT, bool FAST>
void launch(const AttnArgs& a, int64_t workgroups, hipStream_t st) {
    const int nh = a.G < kAttnHeads ? a.G : kAttnHeads;
    const size_t out = (size_t)kAttnWaves * nh * ((DT < kAttnOutCols ? DT : kAttnOutCols) + 4) * sizeof(float);
    const size_t join = (size_t)kAttnMaxWorkgroups * nh * sizeof(float);   // factors of every partial result
    hipLaunchKernelGGL((k_paged_attn<NVFP4_KV_FMT, DT, FAST>), dim3((unsigned)workgroups), dim3(kAttnThreads),
                       out > join ? out : join, st, a);
}

template <int DT>
void launch_dt(const AttnArgs& a, bool fast, int64_t workgroups, hipStream_t st) {
    if (fast && a.shape.D == DT) launch<DT, true>(a, workgroups, st);
    else launch<DT, false>(a, workgroups, st);
}

}  // namespace

#if NVFP4_KV_FMT == 0
#define NVFP4_ATTN_LAUNCHER launch_attn_bf16
#elif NVFP4_KV_FMT == 1
#define NVFP4_ATTN_LAUNCHER launch_attn_f16
#elif NVFP4_KV_FMT == 2
#define NVFP4_ATTN_LAUNCHER launch_attn_e4m3
#else
#define NVFP4_ATTN_LAUNCHER launch_attn_nvfp4
#endif

void NVFP4_ATTN_LAUNCHER(const AttnArgs& a, bool fast, int64_t workgroups, hipStream_t st) {
    if (a.shape.D <= 64) launch_dt<64>(a, fast, workgroups, st);
    else if (a.shape.D <= 128) launch_dt<128>(a, fast, workgroups, st);
    else launch_dt<256>(a, fast, workgroups, st);
}

}  // namespace nvfp4
