// Host side of the single-token attention: launch shape, workspace layout and
// the launchers of its translation units (one per cache format).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels_attn.h"

namespace nvfp4 {

struct AttnShape {
    int64_t pairs;       // (sequence, key-value head, tile of 16 query heads)
    int S;               // splits of the longest sequence
    int64_t part_floats; // fp32 of one split's partial result
    int64_t total;       // workspace bytes: the counters' fixed region, then every pair's partial results
};

// Splits.  The lengths are on the device, so the grid holds S workgroups for
// every pair and a pair with fewer tokens than S chunks leaves the rest of
// them at once; the split length itself is taken on the device from the
// sequence's own length.
constexpr int64_t kAttnWorkgroups = 2048;
constexpr int kAttnMaxSplits = 64;
// Only calls of fewer than kAttnWorkgroups pairs are split, so the counters of
// every call fit this region at the workspace's start, which partial results
// of calls of other sizes never reach.
constexpr int64_t kAttnCounterBytes = kAttnWorkgroups * 4;
inline AttnShape attn_shape(int64_t B, int64_t Hk, int64_t G, int64_t D, int64_t max_tokens) {
    AttnShape s;
    s.pairs = B * Hk * ((G + kAttnHeads - 1) / kAttnHeads);
    const int64_t chunks = (max_tokens + kAttnChunk - 1) / kAttnChunk;
    int64_t S = s.pairs > 0 ? (kAttnWorkgroups + s.pairs - 1) / s.pairs : 1;
    if (S > kAttnMaxSplits) S = kAttnMaxSplits;
    if (S > chunks) S = chunks;
    if (S < 1) S = 1;
    s.S = (int)S;
    s.part_floats = (G < kAttnHeads ? G : kAttnHeads) * (D + 2);
    s.total = S > 1 ? kAttnCounterBytes + s.pairs * S * s.part_floats * 4 : 0;
    return s;
}

// Defined by attn.hip, once per cache format (0 bf16, 1 fp16, 2 E4M3, 3 NVFP4).
void launch_attn_bf16(const AttnArgs& a, int64_t B, int64_t Hk, hipStream_t st);
void launch_attn_f16(const AttnArgs& a, int64_t B, int64_t Hk, hipStream_t st);
void launch_attn_e4m3(const AttnArgs& a, int64_t B, int64_t Hk, hipStream_t st);
void launch_attn_nvfp4(const AttnArgs& a, int64_t B, int64_t Hk, hipStream_t st);

}  // namespace nvfp4
