// C ABI of the low-rank adapters (include/nvfp4_w4a16.h).
#include <hip/hip_runtime.h>

#include "../../include/nvfp4_w4a16.h"
#include "kernels_lora.h"
#include "plan.h"

using namespace nvfp4;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kFar = (int64_t)1 << 40;
constexpr int64_t kMostRows = 1048560;
static_assert(kMostRows / kLoraTile < 65535, "tiles fit a grid");

bool sizes(const char* fn, int64_t T, int64_t K, int64_t N, int64_t R) {
    // tiles of rows are the grid's second axis
    if (T < 0 || T > kMostRows || K < 8 || K >= (int64_t)1 << 24 || K % 8 != 0 || N < 0 || N >= (int64_t)1 << 24) {
        fail(NVFP4_ERR_INVALID_ARG, "%s: T = %lld must be in [0, 1048560], K = %lld a multiple of 8 in [8, 2^24), N = %lld in [0, 2^24)",
             fn, (long long)T, (long long)K, (long long)N);
        return false;
    }
    if (R < 8 || R > kLoraMaxRank || R % 8 != 0) {
        fail(NVFP4_ERR_INVALID_ARG, "%s: rank %lld must be a multiple of 8 up to %d", fn, (long long)R, kLoraMaxRank);
        return false;
    }
    return true;
}

struct LoraShape {
    int slices, slice, places, groups;   // groups: the grid's second axis
};
LoraShape lora_shape(int64_t T, int64_t K, int64_t L) {
    LoraShape s;
    s.places = T <= kLoraLists ? (int)(L < T ? (L < 1 ? 1 : L) : T) : 0;
    s.groups = s.places ? s.places : (int)((T + kLoraTile - 1) / kLoraTile);
    // K slices of at least a chunk for each wave, as many as make about 512
    // workgroups; k_lora_up reads them all for each of its column blocks (4099
    // prompt rows, rank 32: 48.4 us in all with 4, 52 with 8, 53 with 2; 133 rows
    // of 12 adapters, rank 64: 17.7 with 8, 19.8 with 4)
    int64_t want = (512 + s.groups - 1) / s.groups;
    const int64_t most = (K + 511) / 512;
    if (want > most) want = most;
    if (want > (s.places ? 8 : 4)) want = s.places ? 8 : 4;
    s.slice = (int)round_up((K + want - 1) / want, 128);
    s.slices = (int)((K + s.slice - 1) / s.slice);
    return s;
}

// The grid's third axis.  Shares of a list, where adapters have few workgroups
// otherwise: up to one for every `rows` rows, which a workgroup takes at a time
// (60 rows of one adapter of rank 128, 4096 columns: 21 us, 37 with one share for
// 64 rows; 128 of 4: 23 and 28; 133 rows of 12, rank 64: 17.7 with either).
// Tiles: two turns, so that where one prompt ends and the next begins both
// adapters go at once (2048 prompt rows of 6 adapters: 24 us, one turn 27), and up
// to eight while there are few workgroups (2048 rows of 16 adapters in any order:
// 47 us, two turns 50).
unsigned shares(int64_t T, const LoraShape& s, int64_t blocks, int rows) {
    const int64_t want = (s.places ? 1024 : 2048) / (blocks * s.groups);
    if (!s.places) return (unsigned)(want < 2 ? 2 : want < 8 ? want : 8);
    const int64_t most = (T + rows - 1) / rows;
    return (unsigned)(want < 1 ? 1 : want < most ? want : most);
}

template <int RT, int MT, bool F16>
void launch_down(const LoraArgs& a, const LoraShape& s, hipStream_t st) {
    hipLaunchKernelGGL((k_lora_down<RT, MT, F16>), dim3((unsigned)a.slices, (unsigned)s.groups, shares(a.T, s, a.slices, MT * kLoraRows)),
                       dim3(kLoraThreads), 0, st, a);
}
template <int KT, bool F16>
void launch_up(LoraArgs a, const LoraShape& s, hipStream_t st) {
    // as many columns a wave as leave 512 workgroups (tiles: 1024, but 64 columns
    // at least), up to 256: B's fragments are asked for once a step of 32, a
    // list's rows' sums made once a workgroup (133 rows, rank 64: 17.6 us with
    // 512, 21 with 1024; tiles of 4099 rows: 48.2 with 1024, 50.6 with 512; of
    // 2048 rows of 16 adapters: 50 with 64 columns, 63 with 32)
    const int64_t enough = s.places ? 512 : 1024;
    int64_t blocks;
    a.cols = 8 * kLoraCols;
    for (;; a.cols /= 2) {
        blocks = (a.N + kLoraWaves * a.cols - 1) / (kLoraWaves * a.cols);
        if (a.cols == (s.places ? kLoraCols : 2 * kLoraCols) || blocks * s.groups >= enough) break;
    }
    hipLaunchKernelGGL((k_lora_up<KT, F16>), dim3((unsigned)blocks, (unsigned)s.groups, shares(a.T, s, blocks, kLoraTile)),
                       dim3(kLoraThreads), 0, st, a);
}
template <bool F16>
void launch(const LoraArgs& a, const LoraShape& s, hipStream_t st) {
    if (a.R <= 16) launch_down<1, 4, F16>(a, s, st);
    else if (a.R <= 32) launch_down<2, 4, F16>(a, s, st);
    else if (a.R <= 64) launch_down<4, 2, F16>(a, s, st);
    else launch_down<8, 1, F16>(a, s, st);
    if (a.R <= 32) launch_up<1, F16>(a, s, st);
    else if (a.R <= 64) launch_up<2, F16>(a, s, st);
    else launch_up<4, F16>(a, s, st);
}

}  // namespace

extern "C" {

int64_t nvfp4_lora_workspace_bytes(int64_t T, int64_t K, int64_t N, int64_t R) {
    if (!sizes("nvfp4_lora_workspace_bytes", T, K, N, R)) return -1;
    // one adapter has the most slices
    return T == 0 || N == 0 ? 0 : (int64_t)lora_shape(T, K, 1).slices * T * R * 4;
}

nvfp4_status nvfp4_lora_add(const void* x, int64_t ld_x, const void* a, int64_t a_l, int64_t a_r, const void* b, int64_t b_l,
                            int64_t b_n, const int32_t* adapter, const float* scale, const void* y, int64_t ld_y, void* out,
                            int64_t ld_o, int64_t T, int64_t K, int64_t N, int64_t R, int64_t L, void* workspace,
                            int64_t workspace_bytes, int f16, void* stream) {
    const char* fn = "nvfp4_lora_add";
    if (!sizes(fn, T, K, N, R)) return NVFP4_ERR_INVALID_ARG;
    if (L < 0 || L >= (int64_t)1 << 31) return fail(NVFP4_ERR_INVALID_ARG, "%s: L = %lld adapters", fn, (long long)L);
    if (T == 0 || N == 0) return ok();
    if (ld_x < K || ld_y < N || ld_o < N || ld_x >= kFar || ld_y >= kFar || ld_o >= kFar)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: a leading dimension is below its row's length or too large", fn);
    if (out == y && T > 1 && ld_o != ld_y)   // rows without an adapter are not copied then
        return fail(NVFP4_ERR_INVALID_ARG, "%s: out is y with another leading dimension", fn);
    if (a_l < 0 || a_r < 0 || b_l < 0 || b_n < 0 || a_l >= kFar || a_r >= kFar || b_l >= kFar || b_n >= kFar)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: strides of a or b are out of range", fn);
    if (!x || !y || !out || !adapter || (L > 0 && (!a || !b))) return fail(NVFP4_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(x, 16) || ld_x % 8 != 0 || !aligned(a, 16) || a_l % 8 != 0 || a_r % 8 != 0 || !aligned(b, 16) ||
        b_l % 8 != 0 || b_n % 8 != 0)
        return fail(NVFP4_ERR_ALIGNMENT, "%s: rows of x, a and b must be 16-byte aligned", fn);
    if (!aligned(y, 2) || !aligned(out, 2) || !aligned(adapter, 4) || !aligned(scale, 4))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: misaligned pointer", fn);
    const int64_t need = nvfp4_lora_workspace_bytes(T, K, N, R);
    if (!workspace || workspace_bytes < need)
        return fail(NVFP4_ERR_BUFFER_TOO_SMALL, "%s: workspace of %lld bytes is below the %lld bytes this call needs", fn,
                    (long long)workspace_bytes, (long long)need);
    if (!aligned(workspace, 16)) return fail(NVFP4_ERR_ALIGNMENT, "%s: workspace must be 16-byte aligned", fn);
    const LoraShape s = lora_shape(T, K, L);
    LoraArgs g;
    g.x = static_cast<const uint16_t*>(x);
    g.a = static_cast<const uint16_t*>(a);
    g.b = static_cast<const uint16_t*>(b);
    g.y = static_cast<const uint16_t*>(y);
    g.out = static_cast<uint16_t*>(out);
    g.adapter = adapter;
    g.scale = scale;
    g.h = static_cast<float*>(workspace);
    g.ld_x = ld_x;
    g.ld_y = ld_y;
    g.ld_o = ld_o;
    g.a_l = a_l;
    g.a_r = a_r;
    g.b_l = b_l;
    g.b_n = b_n;
    g.T = (int)T;
    g.K = (int)K;
    g.N = (int)N;
    g.R = (int)R;
    g.L = (int)L;
    g.slices = s.slices;
    g.slice = s.slice;
    g.places = s.places;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (f16) launch<true>(g, s, st);
    else launch<false>(g, s, st);
    return launched(fn);
}

}  // extern "C"
