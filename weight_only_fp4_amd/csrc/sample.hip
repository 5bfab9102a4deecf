// C ABI of the choice of the next token (include/nvfp4_w4a16.h).
#include <hip/hip_runtime.h>

#include "../../include/nvfp4_w4a16.h"
#include "kernels_sample.h"
#include "plan.h"

using namespace nvfp4;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMostVocab = (int64_t)1 << 23;   // the steps of a row fit k_sample_row's counters

bool sizes(const char* fn, int64_t B, int64_t V) {
    if (B >= 0 && B < (int64_t)1 << 22 && V >= 1 && V <= kMostVocab) return true;
    fail(NVFP4_ERR_INVALID_ARG, "%s: B = %lld must be in [0, 2^22), V = %lld in [1, 2^23]", fn, (long long)B, (long long)V);
    return false;
}

}  // namespace

extern "C" {

int64_t nvfp4_sample_workspace_bytes(int64_t B, int64_t V) {
    if (!sizes("nvfp4_sample_workspace_bytes", B, V)) return -1;
    return 0;
}

nvfp4_status nvfp4_sample(const void* logits, int64_t ld, int type, int64_t B, int64_t V, const float* u,
                          const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                          int32_t* tokens, float* logprobs, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "nvfp4_sample";
    if (!sizes(fn, B, V)) return NVFP4_ERR_INVALID_ARG;
    if (type < NVFP4_LOGITS_BF16 || type > NVFP4_LOGITS_F32) return fail(NVFP4_ERR_INVALID_ARG, "%s: unknown logits type %d", fn, type);
    if (ld < 0 || ld >= (int64_t)1 << 40)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: ld = %lld is negative or too large", fn, (long long)ld);
    if (B == 0) return ok();
    if (!logits || !u || !tokens) return fail(NVFP4_ERR_INVALID_ARG, "%s: NULL logits, u or tokens", fn);
    if (!aligned(logits, type == NVFP4_LOGITS_F32 ? 4 : 2)) return fail(NVFP4_ERR_ALIGNMENT, "%s: misaligned logits", fn);
    const void* all[] = {u, temperature, top_k, top_p, min_p, tokens, logprobs};
    for (const void* p : all)
        if (!aligned(p, 4)) return fail(NVFP4_ERR_ALIGNMENT, "%s: settings and outputs must be 4-byte aligned", fn);
    SampleArgs a;
    a.logits = logits;
    a.ld = ld;
    a.u = u;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.tokens = tokens;
    a.logprobs = logprobs;
    a.B = (int)B;
    a.V = (int)V;
    int bits = 0;
    while ((int64_t)1 << bits < V) ++bits;
    a.shift = 62 - bits < 52 ? 62 - bits : 52;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const dim3 grid((unsigned)B), block(kSampleThreads);
    if (type == NVFP4_LOGITS_BF16) hipLaunchKernelGGL((k_sample_row<kLogitBf16>), grid, block, 0, st, a);
    else if (type == NVFP4_LOGITS_F16) hipLaunchKernelGGL((k_sample_row<kLogitF16>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_sample_row<kLogitF32>), grid, block, 0, st, a);
    return launched(fn);
}

}  // extern "C"
