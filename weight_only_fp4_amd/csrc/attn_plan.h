// Host side of the single-token attention: launch shape, workspace layout and
// the launchers of its translation units (one per cache format).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/nvfp4_w4a16.h"
#include "kernels_attn.h"

namespace nvfp4 {

struct AttnShape {
    int64_t pairs;        // (sequence, key-value head, tile of 16 query heads)
    int64_t workgroups;
    bool split;           // stretches of units; else one workgroup per pair
    int64_t part_floats;  // fp32 of one partial result
    int64_t total;        // workspace bytes: the counters' fixed region, then two partial results a workgroup
};

// A split call's counters, one a workgroup, at the workspace's start: partial
// results of calls of other sizes never reach them.
constexpr int64_t kAttnCounterBytes = kAttnMaxWorkgroups * 4;
static_assert(kAttnCounterBytes == NVFP4_ATTENTION_COUNTER_BYTES, "the header's figure");
// Two workgroups per compute unit where the kernel's registers let eight waves
// fit it: one works while the other ends a segment.  They do up to D = 128 and
// with E4M3 at 256 (151 .. 250 registers); D = 256 with 16 bits (253 + 48
// accumulation registers) and with NVFP4 (256 + 6) runs one workgroup a unit,
// the second 256 after the first (8 x 8192 tokens, 8 heads, by kernel trace: 16
// bits 100 us, 5.4 TB/s; NVFP4 43, 3.5; E4M3 49, 5.5).
// Only places the lengths can give count (kernels_attn.h).
//
// More than kAttnScan sequences are not split: their unit counts would not fit
// LDS, and such batches fill the chip with a workgroup per pair (2048 of 40
// tokens and one of 8192, 8 heads of 128, bf16: 152 us; 2047 and it, split, 249).
// Only one sequence far longer than all others then takes longer (131072: 1716
// us and 328).
inline AttnShape attn_shape(int64_t B, int64_t Hk, int64_t G, int64_t D, int64_t max_tokens) {
    AttnShape s;
    s.pairs = B * Hk * ((G + kAttnHeads - 1) / kAttnHeads);
    s.part_floats = (G < kAttnHeads ? G : kAttnHeads) * (D + 2);
    const int64_t units = (max_tokens + kAttnTile + kAttnUnit - 1) / kAttnUnit;
    const int64_t places = s.pairs * (units + 2);   // at most (kernels_attn.h)
    s.split = B <= kAttnScan && s.pairs * (units + 1) >= 8 && places < ((int64_t)1 << 31);
    s.workgroups = s.pairs;
    if (s.split) {
        int64_t each = units + 1;
        if (each > kAttnPairSplits) each = kAttnPairSplits;
        s.workgroups = s.pairs * each < kAttnMaxWorkgroups ? s.pairs * each : kAttnMaxWorkgroups;
    }
    s.total = s.split && units > 1 ? kAttnCounterBytes + (int64_t)kAttnMaxWorkgroups * 2 * s.part_floats * 4 : 0;
    return s;
}

// Defined by attn.hip, once per cache format (0 bf16, 1 fp16, 2 E4M3, 3
// NVFP4): the launch, `fast` as kernels_attn.h has it.
void launch_attn_bf16(const AttnArgs& a, bool fast, int64_t workgroups, hipStream_t st);
void launch_attn_f16(const AttnArgs& a, bool fast, int64_t workgroups, hipStream_t st);
void launch_attn_e4m3(const AttnArgs& a, bool fast, int64_t workgroups, hipStream_t st);
void launch_attn_nvfp4(const AttnArgs& a, bool fast, int64_t workgroups, hipStream_t st);

}  // namespace nvfp4
