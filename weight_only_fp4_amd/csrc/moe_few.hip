// C ABI of the mixture-of-experts layer for a few tokens (include/nvfp4_w4a16.h).
#include <hip/hip_runtime.h>

#include "../../include/nvfp4_w4a16.h"
#include "kernels_moe_few.h"
#include "plan.h"

using namespace nvfp4;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kFewCounters = NVFP4_MOE_LAYER_COUNTER_BYTES / 4;   // units whose columns may be split
constexpr int64_t kFewLd = (int64_t)1 << 21;                          // offsets of a part's 512 rows fit 32 bits

struct FewShape {
    int S;
    int64_t a_at, list_at, part_at, total;   // workspace: counters, a, FC2's list, partial sums
};

FewShape few_shape(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
    FewShape s;
    const int64_t P = T * k, NU = (H + kUnitN - 1) / kUnitN, KC = (I + kChunkK - 1) / kChunkK;
    // enough workgroups of FC2 for two a compute unit, while a wave still has two
    // chunks (16 tokens of the figures in kernels_moe_few.h: 41.5 us with 512
    // workgroups and with 256, 46.6 with 1024)
    int64_t S = NU <= kFewCounters ? (512 + NU - 1) / NU : 1;
    const int64_t chunks = (P < E ? P : E) * KC;
    const int64_t most = chunks / (kFewWaves * 2);
    if (S > most) S = most;
    if (S > 16) S = 16;
    s.S = S < 1 ? 1 : (int)S;
    s.a_at = NVFP4_MOE_LAYER_COUNTER_BYTES;
    s.list_at = s.a_at + P * KC * kChunkK * kFewParts * 2;
    s.part_at = s.list_at + round_up((int64_t)sizeof(FewList), 256);
    s.total = s.part_at + (s.S > 1 ? (int64_t)s.S * NU * T * kUnitN * 4 : 0);
    return s;
}

nvfp4_status sizes(const char* fn, int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, int mx) {
    if (T < 0 || T > kFewTokens || k < 1 || k > kFewPairs || T * k > kFewPairs)
        return fail(NVFP4_ERR_INVALID_ARG,
                    "%s: T = %lld, k = %lld: up to %d tokens and %d (token, slot) pairs (more rows go by nvfp4_moe_route, "
                    "nvfp4_moe_fc1, the grouped GEMM and nvfp4_moe_combine)",
                    fn, (long long)T, (long long)k, kFewTokens, kFewPairs);
    if (E < 1 || E > kMaxExperts) return fail(NVFP4_ERR_INVALID_ARG, "%s: E = %lld must be in [1, %d]", fn, (long long)E, kMaxExperts);
    const int64_t unit = mx ? 32 : 16;
    if (H < unit || I < unit || H % unit != 0 || I % unit != 0 || H >= kFewLd || I >= kFewLd)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: H = %lld, I = %lld must be multiples of %lld below 2^21", fn, (long long)H,
                    (long long)I, (long long)unit);
    return NVFP4_OK;
}

template <bool F16, bool PRE, int ACT>
void launch_fc1(const FewArgs& f, hipStream_t st) {
    constexpr int NT = ACT == kActSiluGlu ? 2 : 1;
    hipLaunchKernelGGL((k_moe_few_fc1<F16, PRE, ACT>), dim3((unsigned)((f.NU1 + NT - 1) / NT), (unsigned)f.P + 1),
                       dim3(kFewWaves1 * 64), 0, st, f);
}
template <bool F16>
void launch_fc2(const FewArgs& f, hipStream_t st) {
    hipLaunchKernelGGL((k_moe_few_fc2<F16>), dim3((unsigned)f.NU2, (unsigned)f.sk.S), dim3(kFewWaves * 64),
                       (size_t)kFewWaves * f.T * 16 * sizeof(float), st, f);
}
template <bool F16>
void launch(const FewArgs& f, int act, hipStream_t st) {
    if (act == kActSiluGlu) f.pre1 ? launch_fc1<F16, true, kActSiluGlu>(f, st) : launch_fc1<F16, false, kActSiluGlu>(f, st);
    else f.pre1 ? launch_fc1<F16, true, kActRelu2>(f, st) : launch_fc1<F16, false, kActRelu2>(f, st);
    launch_fc2<F16>(f, st);
}

}  // namespace

extern "C" {

int64_t nvfp4_moe_layer_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
    if (sizes("nvfp4_moe_layer_workspace_bytes", T, k, E, H, I, 0) != NVFP4_OK) return -1;
    return T == 0 ? 0 : few_shape(T, k, E, H, I).total;
}

nvfp4_status nvfp4_moe_layer(const void* x, int64_t ld_x, const int32_t* topk_ids, const float* topk_weights, int64_t T,
                             int64_t k, const void* pre_scale1, const void* w_fc1, const float* global_scales1,
                             const void* pre_scale2, const void* w_fc2, const float* global_scales2,
                             int global_scale_is_divisor, int activation, void* out, int64_t ld_o, int64_t E, int64_t H,
                             int64_t I, void* workspace, int64_t workspace_bytes, int f16, int mx, void* stream) {
    const char* fn = "nvfp4_moe_layer";
    if (mx != 0 && mx != 1) return fail(NVFP4_ERR_INVALID_ARG, "%s: mx must be 0 or 1", fn);
    int act;
    if (activation == NVFP4_MOE_SILU_GLU) act = kActSiluGlu;
    else if (activation == NVFP4_MOE_RELU2) act = kActRelu2;
    else return fail(NVFP4_ERR_INVALID_ARG, "%s: activation %d is not NVFP4_MOE_SILU_GLU or NVFP4_MOE_RELU2", fn, activation);
    nvfp4_status s = sizes(fn, T, k, E, H, I, mx);
    if (s != NVFP4_OK) return s;
    if (ld_x < H || ld_o < H || ld_x >= kFewLd || ld_o >= (int64_t)1 << 40)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: ld_x = %lld or ld_o = %lld is below H = %lld or too large", fn, (long long)ld_x,
                    (long long)ld_o, (long long)H);
    if (!w_fc1 || !w_fc2) return fail(NVFP4_ERR_INVALID_ARG, "%s: w_fc1 or w_fc2 is NULL", fn);
    if (mx ? global_scales1 || global_scales2 : !global_scales1 || !global_scales2)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: %s", fn, mx ? "MXFP4 weights take no global scales" : "global scales are NULL");
    if (T == 0) return ok();
    if (!x || !out || !topk_ids || !topk_weights) return fail(NVFP4_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(x, 16) || ld_x % 8 != 0)
        return fail(NVFP4_ERR_ALIGNMENT, "%s: x must be 16-byte aligned with ld_x %% 8 == 0 (ld_x = %lld)", fn, (long long)ld_x);
    if (!aligned(w_fc1, 16) || !aligned(w_fc2, 16) || !aligned(pre_scale1, 16) || !aligned(pre_scale2, 16))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: weights and pre-scales must be 16-byte aligned", fn);
    if (!aligned(out, 2) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) || !aligned(global_scales1, 4) ||
        !aligned(global_scales2, 4))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: misaligned pointer", fn);
    const FewShape sh = few_shape(T, k, E, H, I);
    if (!workspace || workspace_bytes < sh.total)
        return fail(NVFP4_ERR_BUFFER_TOO_SMALL, "%s: workspace of %lld bytes is below the %lld bytes this call needs", fn,
                    (long long)workspace_bytes, (long long)sh.total);
    if (!aligned(workspace, 256)) return fail(NVFP4_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", fn);
    FewArgs f;
    f.x = static_cast<const uint16_t*>(x);
    f.ld_x = ld_x;
    f.ids = topk_ids;
    f.weights = topk_weights;
    f.F = (int)(act == kActSiluGlu ? 2 * I : I);
    const Layout L1 = make_layout(E, f.F, H, mx), L2 = make_layout(E, H, I, mx);
    f.w1 = make_view(L1, static_cast<const uint8_t*>(w_fc1));
    f.w2 = make_view(L2, static_cast<const uint8_t*>(w_fc2));
    f.g1 = global_scales1;
    f.g2 = global_scales2;
    f.pre1 = static_cast<const uint16_t*>(pre_scale1);
    f.pre2 = static_cast<const uint16_t*>(pre_scale2);
    char* ws = static_cast<char*>(workspace);
    f.a = reinterpret_cast<uint16_t*>(ws + sh.a_at);
    f.P = (int)(T * k);
    f.list = reinterpret_cast<FewList*>(ws + sh.list_at);
    f.out = static_cast<uint16_t*>(out);
    f.ld_o = ld_o;
    f.sk = SplitK{sh.S, reinterpret_cast<float*>(ws + sh.part_at), reinterpret_cast<int*>(ws)};
    f.g_div = global_scale_is_divisor != 0;
    f.T = (int)T;
    f.k = (int)k;
    f.E = (int)E;
    f.H = (int)H;
    f.I = (int)I;
    f.NU1 = (int)L1.NU;
    f.KC1 = (int)L1.KC;
    f.NU2 = (int)L2.NU;
    f.KC2 = (int)L2.KC;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (f16) launch<true>(f, act, st);
    else launch<false>(f, act, st);
    return launched(fn);
}

}  // extern "C"
