// Single-token attention kernels of one cache format (NVFP4_KV_FMT: 0 bf16,
// 1 fp16, 2 E4M3, 3 NVFP4).
#include "attn_plan.h"

#ifndef NVFP4_KV_FMT
#error "compile with -DNVFP4_KV_FMT=0 .. 3"
#endif

namespace nvfp4 {

namespace {

template <int DT, bool FULL>
void launch(const AttnArgs& a, int64_t B, int64_t Hk, hipStream_t st) {
    const int nh = a.G < kAttnHeads ? a.G : kAttnHeads;
    const size_t lds = (size_t)kAttnWaves * nh * (DT / attn_out_passes(DT) + 4) * sizeof(float);
    const dim3 grid((unsigned)a.S, (unsigned)(Hk * a.head_tiles), (unsigned)B);
    hipLaunchKernelGGL((k_paged_attn<NVFP4_KV_FMT, DT, FULL>), grid, dim3(kAttnWaves * 64), lds, st, a);
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

void NVFP4_ATTN_LAUNCHER(const AttnArgs& a, int64_t B, int64_t Hk, hipStream_t st) {
    const int D = a.shape.D;
    if (D == 64) launch<64, true>(a, B, Hk, st);
    else if (D < 64) launch<64, false>(a, B, Hk, st);
    else if (D == 128) launch<128, true>(a, B, Hk, st);
    else if (D < 128) launch<128, false>(a, B, Hk, st);
    else if (D == 256) launch<256, true>(a, B, Hk, st);
    else launch<256, false>(a, B, Hk, st);
}

}  // namespace nvfp4
