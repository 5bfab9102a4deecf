// A whole mixture-of-experts layer for a few tokens in two kernels
// (nvfp4_moe_layer).  With pairs p = t k + j, e = ids[p]:
//
//   a_p   = RNE16(act(g1_e X'_t W1_e^T))                 k_moe_few_fc1
//   out_t = RNE16(sum_j w_tj g2_e (a'_p W2_e^T))         k_moe_few_fc2
//
// X' and a' with the pre-quant scales applied (RNE16) where given.  The first
// product's sums stay fp32 through the activation, and the second's through
// the weighted sum: a is the only value between x and out that is rounded, to
// the matrix instructions' operand type.
//
// Both kernels contract as the small-M GEMM does (kernels_gemm.h) and read
// each active expert's weights once while it has at most 4 MG rows.  What
// bounds them is HBM, behind a chain of latencies (ids, rows, weights).
//
// There is no routing launch.  k_moe_few_fc1 has a grid row per pair, and the
// workgroups of the first pair of an expert do all of the expert's pairs; its
// first column also writes each pair's group (the first pair of its expert),
// its place in it and the groups' sizes.  k_moe_few_fc2 makes a list of (expert,
// up to 4 MG rows) from them; a workgroup owns 16 columns of out and a share of
// that list's K chunks, cut evenly into one stretch per wave, which a wave's
// ring of loads streams without a stop where an expert ends.  So the sum over a
// token's experts needs no exchange of rows: it is formed where the products
// are, and split workgroups exchange 16 columns of T rows.
//
// Waves add into accumulators of their own and are summed in a fixed order, as
// the splits are: no result depends on timing.
#pragma once
#include "kernels_gemm.h"

namespace nvfp4 {

constexpr int kFewTokens = 64;
constexpr int kFewPairs = 512;
constexpr int kFewWaves = 4;           // of a workgroup of k_moe_few_fc2
constexpr int kFewDepth = 4;           // ring of loads

struct FewArgs {
    const uint16_t* x;
    int64_t ld_x;
    const int32_t* ids;
    const float* weights;
    BlobView w1, w2;
    const float* g1;
    const float* g2;
    const uint16_t* pre1;
    const uint16_t* pre2;
    uint16_t* a;          // [P][ld_a] workspace
    int32_t* group;       // [P]: first pair of the pair's expert, -1 if it has none
    int32_t* place;       // [P]: the pair's place among that expert's pairs
    int32_t* size;        // [P]: the expert's pairs at its first, 0 elsewhere
    uint16_t* out;
    int64_t ld_a, ld_o;
    SplitK sk;            // k_moe_few_fc2's splits: partials [S][units][T * 16], counters [units]
    int g_div;
    int T, k, P, E, H, I, F;   // F: rows of W1 (2 I with a gate)
    int NU1, KC1, NU2, KC2;
};

// Grid: (units of W1 / NT, pairs).  NT = 2 with the gate (a pair of units: gate, up).
template <int MG, int W, bool F16, bool PRE, int ACT>
__global__ void __launch_bounds__(W * 64) k_moe_few_fc1(FewArgs f) {
    constexpr int NT = ACT == kActSiluGlu ? 2 : 1;
    constexpr int RLD = NT * 16;
    __shared__ float red[W][4 * MG * RLD];
    __shared__ float2 lut[256];
    __shared__ int32_t tokens[kFewPairs];
    __shared__ int32_t pairs[kFewPairs];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int p = blockIdx.y, u0 = blockIdx.x * NT;
    const int e = f.ids[p];
    const bool none = e < 0 || e >= f.E;
    // the expert's pairs, in order (every wave makes the same list)
    int count = 0;
    bool first = true;
    for (int q0 = 0; q0 < f.P; q0 += 64) {
        const int q = q0 + lane;
        const bool same = q < f.P && f.ids[q] == e;
        const uint64_t m = __ballot(same);
        if (q0 <= p) {
            const uint64_t before = q0 + 64 <= p ? ~0ull : ((1ull << (p - q0)) - 1);
            if (m & before) first = false;
        }
        if (same) {
            const int at = count + __popcll(m & ((1ull << lane) - 1));
            pairs[at] = q;
            tokens[at] = q / f.k;
        }
        count += __popcll(m);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        f.size[p] = first && !none ? count : 0;
        if (none) f.group[p] = -1;
    }
    if (none || !first) return;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < count; i += W * 64) {
            f.group[pairs[i]] = p;
            f.place[pairs[i]] = i;
        }
    const int c0 = f.KC1 * w / W, c1 = f.KC1 * (w + 1) / W;
    const int64_t blk0 = f.w1.block(e, u0, 0);
    const WaveWeights ww{f.w1.codes + blk0 * kCodeBlock, f.w1.scales + blk0 * kScaleBlock,
                         f.w1.unit_stride * kCodeBlock, f.w1.chunk_stride * kCodeBlock,
                         (f.NU1 - u0) < NT ? (f.NU1 - u0) : NT};
    bool built = false;
    auto mid = [&]() {
        if (built) return;
        build_scale_table(lut, f.w1.mx);
        wait_lgkmcnt0();   // only LDS writes need to be seen (the ring's loads stay in flight)
        asm volatile("s_barrier" ::: "memory");
        built = true;
    };
    const float gv = global_scale_at(f.g1, e, f.g_div);
    for (int r0 = 0; r0 < count; r0 += 4 * MG) {
        const int rows = count - r0 < 4 * MG ? count - r0 : 4 * MG;
        small_m_pass<MG, NT, kFewDepth, false, F16, PRE>(f.x, f.ld_x, rows, f.pre1, ww, c0, c1, f.H, lut, red[w], RLD,
                                                         lane, mid, tokens + r0);
        __syncthreads();
        for (int t = threadIdx.x; t < rows * 16; t += W * 64) {
            const int r = t >> 4, c = t & 15;
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int wi = 0; wi < W; ++wi) {
                s0 += red[wi][r * RLD + c];
                if (NT == 2) s1 += red[wi][r * RLD + (NT - 1) * 16 + c];
            }
            const int n = (int)blockIdx.x * 16 + c;
            const float v = ACT == kActSiluGlu ? silu_times(gv * s0, gv * s1) : relu_squared(gv * s0);
            if (n < f.I) f.a[(int64_t)pairs[r0 + r] * f.ld_a + n] = (uint16_t)round_out<F16>(v);
        }
        __syncthreads();
    }
}

struct FewShared {
    float2 lut[256];
    int32_t pair[kFewPairs];      // pairs by group
    float weight[kFewPairs];
    int32_t item_e[kFewPairs];    // items: up to 4 MG rows of an expert
    int32_t item_first[kFewPairs];
    int32_t item_rows[kFewPairs];
    float item_g[kFewPairs];
    int32_t sums[kFewWaves][2];
    int flag;
};

// Grid: (units of W2, S).  A wave's stretch of the items' chunks is streamed
// by one ring; sums[token][16] of each wave in dynamic LDS.
template <int MG, bool F16, bool PRE>
__global__ void __launch_bounds__(kFewWaves * 64) k_moe_few_fc2(FewArgs f) {
    __shared__ FewShared sh;
    extern __shared__ float sums[];   // [kFewWaves][T * 16]
    constexpr int kThreads = kFewWaves * 64;
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int u = blockIdx.x, S = f.sk.S, s = blockIdx.y;
    const int out_n = f.T * 16;
    build_scale_table(sh.lut, f.w2.mx);
    for (int i = tid; i < kFewWaves * out_n; i += kThreads) sums[i] = 0.f;
    // lists from the groups: thread tid scans pairs tid and tid + 256 by their order
    constexpr int kEach = kFewPairs / kThreads;
    int base_rows = 0, items = 0;
    int first_row[kEach], n_rows[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int p = j * kThreads + tid;
        const int n = p < f.P ? f.size[p] : 0, its = (n + 4 * MG - 1) / (4 * MG);
        int a = n, b = its;   // inclusive scans of rows and items
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int oa = __shfl_up(a, d), ob = __shfl_up(b, d);
            if (lane >= d) a += oa, b += ob;
        }
        __syncthreads();
        if (lane == 63) sh.sums[w][0] = a, sh.sums[w][1] = b;
        __syncthreads();
        int ra = base_rows, rb = items;
#pragma unroll
        for (int i = 0; i < kFewWaves; ++i) {
            if (i < w) ra += sh.sums[i][0], rb += sh.sums[i][1];
            base_rows += sh.sums[i][0];
            items += sh.sums[i][1];
        }
        first_row[j] = ra + a - n;
        n_rows[j] = n;
        if (n > 0) {
            const int e = f.ids[p];
            const float g = global_scale_at(f.g2, e, f.g_div);
            for (int i = 0; i < its; ++i) {
                const int at = rb + b - its + i;
                sh.item_e[at] = e;
                sh.item_first[at] = first_row[j] + 4 * MG * i;
                sh.item_rows[at] = n - 4 * MG * i < 4 * MG ? n - 4 * MG * i : 4 * MG;
                sh.item_g[at] = g;
            }
        }
    }
    // the place of a group's rows, kept where its first pair's weight will not be needed: in weight[]
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int p = j * kThreads + tid;
        if (p < f.P && n_rows[j] > 0) sh.weight[p] = __int_as_float(first_row[j]);
    }
    __syncthreads();
    int at[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int p = j * kThreads + tid;
        at[j] = -1;
        if (p < f.P) {
            const int g = f.group[p];
            if (g >= 0) at[j] = __float_as_int(sh.weight[g]) + f.place[p];
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (at[j] >= 0) {
            const int p = j * kThreads + tid;
            sh.pair[at[j]] = p;
            sh.weight[at[j]] = f.weights[p];
        }
    __syncthreads();

    // this wave's stretch of all chunks
    const int64_t all = (int64_t)items * f.KC2;
    const int64_t part = (int64_t)s * kFewWaves + w, parts = (int64_t)S * kFewWaves;
    const int64_t lo = all * part / parts, n = all * (part + 1) / parts - lo;
    if (n > 0) {
        float* mine = sums + w * out_n;
        const int g = lane >> 4, q = (lane >> 2) & 3, ai = lane & 3;
        const int kpiece = g * 32 + q * 8;
        struct At { int item, chunk; };
        At ld = {(int)(lo / f.KC2), (int)(lo % f.KC2)}, us = ld;
        int64_t ld_i = 0;
        const uint8_t *codes = nullptr, *scales = nullptr;   // the load side's unit
        uint32_t row[MG];
        auto enter = [&]() {   // the load side's item
            const int e = __builtin_amdgcn_readfirstlane(sh.item_e[ld.item]);
            const int first = sh.item_first[ld.item], rows = sh.item_rows[ld.item];
            const int64_t blk = f.w2.block(e, u, 0);
            codes = f.w2.codes + blk * kCodeBlock;
            scales = f.w2.scales + blk * kScaleBlock;
#pragma unroll
            for (int mg = 0; mg < MG; ++mg) {
                const int m = 4 * mg + ai;
                row[mg] = (uint32_t)(sh.pair[first + (m < rows ? m : 0)] * f.ld_a * 2);
            }
        };
        enter();
        f32x4 acc[1][MG];
        auto zero = [&]() {
#pragma unroll
            for (int mg = 0; mg < MG; ++mg) acc[0][mg] = f32x4{0.f, 0.f, 0.f, 0.f};
        };
        zero();
        const uint8_t* ab = reinterpret_cast<const uint8_t*>(f.a);
        auto load = [&](SmallSlot<MG, 1>& slot, int64_t i) {
            if (i > ld_i) {   // i is the last one, or one more
                ld_i = i;
                if (++ld.chunk == f.KC2) {
                    ld.chunk = 0;
                    ++ld.item;
                    enter();
                }
            }
            const int64_t off = (int64_t)ld.chunk * f.w2.chunk_stride;
            slot.cw[0] = load_stream_u4(codes + off * kCodeBlock + (uint32_t)(lane * 16));
            slot.sw[0] = load_scale_dword(scales + off * kScaleBlock, lane);
            const int kk = ld.chunk * kChunkK + kpiece;
            const uint32_t kb = kk < f.I ? (uint32_t)(kk * 2) : 0u;
#pragma unroll
            for (int mg = 0; mg < MG; ++mg) slot.xa[mg] = *reinterpret_cast<const uint4*>(ab + (row[mg] + kb));
            if constexpr (PRE) slot.pa = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(f.pre2) + kb);
        };
        auto use = [&](const SmallSlot<MG, 1>& slot, int64_t i) {
            small_m_chunk<MG, 1, false, F16, PRE>(slot, us.chunk * kChunkK + kpiece < f.I, sh.lut, lane, acc);
            const bool ends = us.chunk == f.KC2 - 1;
            if (ends || i == n - 1) {
                // the item's rows into the tokens' sums: lane l < 16 has column l
                const int first = sh.item_first[us.item], rows = sh.item_rows[us.item];
                const float gv = sh.item_g[us.item];
#pragma unroll
                for (int mg = 0; mg < MG; ++mg)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float v = acc[0][mg][r];
                        v += __shfl_xor(v, 16);
                        v += __shfl_xor(v, 32);
                        if (lane < 16 && 4 * mg + r < rows) {
                            const int at = first + 4 * mg + r;
                            float* to = mine + sh.pair[at] / f.k * 16 + lane;
                            *to = __builtin_fmaf(sh.weight[at] * gv, v, *to);
                        }
                    }
                zero();
            }
            if (ends) ++us.item, us.chunk = 0;
            else ++us.chunk;
        };
        SmallSlot<MG, 1> ring[kFewDepth];
        const int64_t last = n - 1;
#pragma unroll
        for (int d = 0; d < kFewDepth; ++d) {
            load(ring[d], d < last ? d : last);
            __builtin_amdgcn_sched_barrier(0);
        }
        int64_t i = 0;
        for (; i + 2 * kFewDepth <= n; i += kFewDepth) {
#pragma unroll
            for (int d = 0; d < kFewDepth; ++d) {
                use(ring[d], i + d);
                __builtin_amdgcn_sched_barrier(0);
                load(ring[d], i + kFewDepth + d);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int d = 0; d < kFewDepth; ++d) {
            if (i + d < n) use(ring[d], i + d);
            if (i + kFewDepth + d < n) load(ring[d], i + kFewDepth + d);
        }
#pragma unroll
        for (int d = 0; d < kFewDepth; ++d)
            if (i + kFewDepth + d < n) use(ring[d], i + kFewDepth + d);
    }
    __syncthreads();
    auto total = [&](int i) {
        float v = 0.f;
#pragma unroll
        for (int wi = 0; wi < kFewWaves; ++wi) v += sums[wi * out_n + i];
        return v;
    };
    auto store = [&](int i, float v) {
        const int64_t c = (int64_t)u * kUnitN + (i & 15);
        if (c < f.H) f.out[(i >> 4) * f.ld_o + c] = (uint16_t)round_out<F16>(fp32_value(v));
    };
    if (S == 1) {
        for (int i = tid; i < out_n; i += kThreads) store(i, total(i));
        return;
    }
    float* part_at = f.sk.partials + ((int64_t)s * f.NU2 + u) * out_n;
    for (int i = tid; i < out_n; i += kThreads) store_partial(part_at + i, total(i));
    if (!split_arrive(f.sk.counters, u, S, &sh.flag)) return;
    for (int i = tid; i < out_n; i += kThreads) {
        float v = 0.f;   // in the splits' order, whichever arrived last
        for (int ss = 0; ss < S; ++ss) v += load_partial(f.sk.partials + ((int64_t)ss * f.NU2 + u) * out_n + i);
        store(i, v);
    }
}

}  // namespace nvfp4
