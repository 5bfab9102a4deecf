// C ABI of the choice of the next token (include/nvfp4_w4a16.h).
#include <hip/hip_runtime.h>

#include "../../include/nvfp4_w4a16.h"
#include "kernels_sample.h"
#include "plan.h"

using namespace nvfp4;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMostVocab = (int64_t)1 << 23;   // the steps of a row fit sample_slow's counters
constexpr int64_t kMostRows = 65535;               // rows are a grid's second axis

// Slices of a row: of 1024 16-byte pieces, which a workgroup holds in LDS
// (2 a thread), or of more where rows are long or so many that 1024 workgroups
// are there without.
struct SampleShape {
    int S, slice, bits;   // bits: 2^bits logits a slice at most
};
SampleShape sample_shape(int64_t B, int64_t V, int type) {
    const int64_t each = type == NVFP4_LOGITS_F32 ? 4 : 8;
    const int64_t pieces = (V + 2 * (each - 1)) / each;   // of a row that starts anywhere
    constexpr int64_t kHeld = kSampleHeld * kSampleScanThreads;
    int64_t least = pieces * B / 1024;   // of a slice, for 1024 workgroups
    if (least < pieces / kSampleMaxSlices + 1) least = pieces / kSampleMaxSlices + 1;
    SampleShape s;
    s.slice = (int)(least <= kHeld ? kHeld : round_up(least, kHeld));
    s.S = (int)((pieces + s.slice - 1) / s.slice);
    s.bits = 0;
    while ((int64_t)1 << s.bits < s.slice * each) ++s.bits;
    return s;
}

bool sizes(const char* fn, int64_t B, int64_t V) {
    if (B >= 0 && B <= kMostRows && V >= 1 && V <= kMostVocab) return true;
    fail(NVFP4_ERR_INVALID_ARG, "%s: B = %lld must be in [0, 65535], V = %lld in [1, 2^23]", fn, (long long)B, (long long)V);
    return false;
}

template <int DT>
void launch(const SampleArgs& a, hipStream_t st) {
    hipLaunchKernelGGL((k_sample_scan<DT>), dim3((unsigned)a.S, (unsigned)a.B), dim3(kSampleScanThreads), 0, st, a);
    hipLaunchKernelGGL((k_sample_pick<DT>), dim3((unsigned)a.B), dim3(kSampleThreads), 0, st, a);
}

}  // namespace

extern "C" {

int64_t nvfp4_sample_workspace_bytes(int64_t B, int64_t V) {
    if (!sizes("nvfp4_sample_workspace_bytes", B, V)) return -1;
    // 32-bit logits have the most slices
    const int64_t S = sample_shape(B, V, NVFP4_LOGITS_F32).S, half = sample_shape(B, V, NVFP4_LOGITS_BF16).S;
    return B * (S > half ? S : half) * (int64_t)sizeof(SampleSlice);
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
    const int64_t need = nvfp4_sample_workspace_bytes(B, V);
    if (!workspace || workspace_bytes < need)
        return fail(NVFP4_ERR_BUFFER_TOO_SMALL, "%s: workspace of %lld bytes is below the %lld bytes this call needs", fn,
                    (long long)workspace_bytes, (long long)need);
    if (!aligned(workspace, 256)) return fail(NVFP4_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", fn);
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
    a.shift = 62 - bits < 45 ? 62 - bits : 45;
    const SampleShape sh = sample_shape(B, V, type);
    a.slices = static_cast<SampleSlice*>(workspace);
    a.S = sh.S;
    a.slice = sh.slice;
    a.slice_shift = 62 - sh.bits < 49 ? 62 - sh.bits : 49;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (type == NVFP4_LOGITS_BF16) launch<kLogitBf16>(a, st);
    else if (type == NVFP4_LOGITS_F16) launch<kLogitF16>(a, st);
    else launch<kLogitF32>(a, st);
    return launched(fn);
}

}  // extern "C"
