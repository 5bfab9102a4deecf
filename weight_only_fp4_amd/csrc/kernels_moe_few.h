// A whole mixture-of-experts layer for a few tokens in two kernels
// (nvfp4_moe_layer).  With pairs p = t k + j, e = ids[p]:
//
//   a_p   = act(g1_e X'_t W1_e^T) (* the second pre-quant scale)   k_moe_few_fc1
//   out_t = RNE16(sum_j w_tj g2_e (a_p W2_e^T))                    k_moe_few_fc2
//
// X' with the first pre-quant scale applied (RNE16) where given.  Sums stay fp32
// from x to out, and a is handed on whole: as three bf16 parts of 8 bits, which
// are multiplied one after another into the same sums.  In both types: bf16 has
// fp32's range, and bare E2M1 values are exact in it.  (Below 2^-110 the last part
// is a bf16 denormal or nothing.)  Two parts of the layer's own type were 16 bits
// in bf16, 22 in fp16 for values near one only, and none beyond 65504; 1 / 16 / 5
// wide tokens (as below) took 13.9 / 49.5 / 104 us.  Tried for three: a row of the
// product for each part, items of two pairs 14.1 / 53.8 / 120, of four 15.8 / 59 /
// 118 (registers spill); two fp16 parts with a power of two for every 16 values
// 15.4 / 56 / 119 (two more loads a chunk).
//
// Both kernels contract as the small-M GEMM does (kernels_gemm.h) and read
// each active expert's weights once for every four of its rows.  What
// bounds them is HBM, behind a chain of latencies (ids, rows, weights).
//
// There is no routing launch.  k_moe_few_fc1 has a grid row per pair, and every
// fourth pair of an expert has workgroups, which do it and those after it up
// to the next.  (With an expert's pairs in one workgroup, one pass after another,
// the busiest expert decides.)  One more workgroup makes the second kernel's
// list meanwhile: items of an expert and up to four of its pairs.  A workgroup
// of k_moe_few_fc2 owns 16 columns of out and a share of the items' K chunks,
// cut evenly into one stretch per wave, which a wave's ring of loads streams
// without a stop where an expert ends.  So the sum over a token's experts needs
// no exchange of rows: it is formed where the products are, and split workgroups
// exchange 16 columns of T rows.
//
// Measured in a graph, over sets of inputs beyond the last cache: 1 token of 128
// experts, top-8, 2048 x 768 (21.2 MB of weights): 13.7 us (1.5 TB/s; the chain of
// latencies is most of it); 16 tokens of it: 51 with NVFP4 weights (4.0 TB/s); 5
// tokens of 8 experts, top-2, 4096 x 14336 (0.6 GB, six experts, on average): 110
// (5.5 of the 7 TB/s that a plain read reaches).
//
// Waves add into accumulators of their own and are summed in a fixed order, as
// the splits are: no result depends on timing.  Where a token's sum is cut depends
// on the number of pairs and of items, so its last bits may on the other tokens'
// experts.
#pragma once
#include "kernels_gemm.h"

namespace nvfp4 {

constexpr int kFewTokens = 64;
constexpr int kFewPairs = 512;
// Pairs that a workgroup of the first product does at most: its rows.  An expert
// with more has its weights read again, which the caches answer: 8 or 16 rows
// cost more in registers and empty rows than they save (with a in one part, 64
// tokens of 128 experts, top-8, 2048 x 768: 128 us with 4, 145 with 8, 174 with
// 16; 64 of 8, top-2, 4096 x 2048, where each has 16 rows: 94, 88, 95).
constexpr int kFewRows = 4;
// Pairs of an item of the second product, a row of the matrix instruction each.
constexpr int kFewItem = 4;
constexpr int kFewParts = 3;
// Shapes (us of the layer in a graph: 1 token of 128 experts, top-8, 2048 x 768;
// 16 tokens of it; 5 tokens of 8 experts, top-2, 4096 x 14336):
//   FC1, waves and depth of their rings: 4 and 2 13.6 / 40.8 / 89.1; 4 and 4 13.7
//   / 44.2 / 90.5; 2 and 4 14.8 / 41.5 / 87.4; 1 and 4 15.5 / 43.2 / 87.0; 8 and 2
//   13.8 / 49.0 / 93.2 (with a in one part);
//   FC2: 8 and 2 13.7 / 51.4 / 110; 8 and 3 17.2 / 54.2 / 112 (more than 128
//   registers: one workgroup a compute unit); 4 and 2 14.2 / 51.1 / 110, and 64
//   tokens of 4 experts, top-1, 26.5 for 24.5.
constexpr int kFewWaves1 = 4, kFewDepth1 = 2;
constexpr int kFewWaves = 8, kFewDepth = 2;

// Up to kFewItem pairs of one expert: places first .. first + rows - 1 of the list.
struct FewItem {
    int32_t e, first, rows;
    float g;   // the expert's global scale
};
struct FewList {
    int32_t items, reserved[3];
    FewItem item[kFewPairs];
    int32_t pair[kFewPairs];      // pairs by expert, in the order of the experts' first ones
    float weight[kFewPairs];
};

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
    uint16_t* a;          // [kFewParts][P][KC2 * 128] workspace: bf16 parts of a, zeros behind I
    FewList* list;        // workspace
    uint16_t* out;
    int64_t ld_o;
    SplitK sk;            // k_moe_few_fc2's splits: partials [S][units][T * 16], counters [units]
    int g_div;
    int T, k, P, E, H, I, F;   // F: rows of W1 (2 I with a gate)
    int NU1, KC1, NU2, KC2;
};

// The second kernel's list, by one workgroup: a pair's place is that of its
// expert's first pair, plus the pairs of the expert before it.
template <int THREADS>
__device__ __forceinline__ void few_list(const FewArgs& f, int32_t* ids, int32_t* place) {
    __shared__ int32_t s_sums[THREADS / 64][2];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    for (int p = tid; p < f.P; p += THREADS) ids[p] = f.ids[p];
    __syncthreads();
    int rows = 0, items = 0;   // of the rounds before
    for (int p0 = 0; p0 < f.P; p0 += THREADS) {
        const int p = p0 + tid, e = p < f.P ? ids[p] : -1;
        const bool valid = e >= 0 && e < f.E;
        int before = 0, all = 0;
        if (valid)
            for (int q = 0; q < f.P; ++q) {
                const bool same = ids[q] == e;
                all += same;
                before += same && q < p;
            }
        const bool first = valid && before == 0;
        const int n = first ? all : 0, its = (n + kFewItem - 1) / kFewItem;
        int a = n, b = its;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int oa = __shfl_up(a, d), ob = __shfl_up(b, d);
            if (lane >= d) a += oa, b += ob;
        }
        if (lane == 63) s_sums[w][0] = a, s_sums[w][1] = b;
        __syncthreads();
        int ra = rows, rb = items;
#pragma unroll
        for (int i = 0; i < THREADS / 64; ++i) {
            if (i < w) ra += s_sums[i][0], rb += s_sums[i][1];
            rows += s_sums[i][0];
            items += s_sums[i][1];
        }
        ra += a - n;
        rb += b - its;
        if (first) {
            place[p] = ra;
            const float g = global_scale_at(f.g2, e, f.g_div);
            for (int i = 0; i < its; ++i)
                f.list->item[rb + i] = FewItem{e, ra + kFewItem * i, n - kFewItem * i < kFewItem ? n - kFewItem * i : kFewItem, g};
        }
        __syncthreads();
    }
    for (int p = tid; p < f.P; p += THREADS) {
        const int e = ids[p];
        if (e < 0 || e >= f.E) continue;
        int before = 0, q = 0;
        while (ids[q] != e) ++q;   // ends at p
        const int first = q;
        for (; q < p; ++q) before += ids[q] == e;
        f.list->pair[place[first] + before] = p;
        f.list->weight[place[first] + before] = f.weights[p];
    }
    if (tid == 0) f.list->items = items;
}

// v as three bf16 values whose sum it is, `stride` apart: its upper 8 bits, the 8
// after them, the last 8.  (An fp32 value less its own upper part is exact.)
__device__ __forceinline__ void few_split(float v, uint16_t* to, int64_t stride) {
    const bool finite = fabsf(v) < __builtin_inff();
#pragma unroll
    for (int part = 0; part < kFewParts; ++part) {
        const uint32_t bits = __float_as_uint(v);
        to[part * stride] = v != v ? (uint16_t)0x7FC0u : (uint16_t)(bits >> 16);
        v = finite ? v - __uint_as_float(bits & 0xFFFF0000u) : 0.f;   // an infinity or NaN leaves nothing over
    }
}

// Grid: (units of W1 / NT, pairs + 1).  NT = 2 with the gate (a pair of units: gate, up).
template <bool F16, bool PRE, int ACT>
__global__ void __launch_bounds__(kFewWaves1 * 64) k_moe_few_fc1(FewArgs f) {
    constexpr int W = kFewWaves1;
    constexpr int NT = ACT == kActSiluGlu ? 2 : 1;
    constexpr int RLD = NT * 16;
    __shared__ float red[W][kFewRows * RLD];
    __shared__ float2 lut[256];
    __shared__ int32_t tokens[kFewPairs];   // (few_list's first)
    __shared__ int32_t pairs[kFewPairs];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int p = (int)blockIdx.y - 1, u0 = blockIdx.x * NT;
    if (p < 0) {   // first in the grid: it is not what the launch waits for in the end
        if (blockIdx.x == 0) few_list<W * 64>(f, tokens, pairs);
        return;
    }
    const int e = f.ids[p];
    if (e < 0 || e >= f.E) return;
    // the pair's place among its expert's pairs, and the pairs from it on (every
    // wave makes the same list)
    int place = 0, upto = 0;
    for (int q0 = 0; q0 < f.P; q0 += 64) {
        const int q = q0 + lane;
        const uint64_t same = __ballot(q < f.P && f.ids[q] == e);
        if (q0 <= p) place += __popcll(same & (q0 + 64 <= p ? ~0ull : (1ull << (p - q0)) - 1));
        if (q0 + 64 > p && (same >> lane) & 1ull) {
            const int at = upto + __popcll(same & ((1ull << lane) - 1)) - place;
            if (at >= 0 && at < kFewRows) {
                pairs[at] = q;
                tokens[at] = q / f.k;
            }
        }
        upto += __popcll(same);
    }
    if (place % kFewRows != 0) return;
    const int rows = upto - place < kFewRows ? upto - place : kFewRows;
    const int c0 = f.KC1 * w / W, c1 = f.KC1 * (w + 1) / W;
    const int64_t blk0 = f.w1.block(e, u0, 0);
    const WaveWeights ww{f.w1.codes + blk0 * kCodeBlock, f.w1.scales + blk0 * kScaleBlock,
                         f.w1.unit_stride * kCodeBlock, f.w1.chunk_stride * kCodeBlock,
                         (f.NU1 - u0) < NT ? (f.NU1 - u0) : NT};
    auto mid = [&]() {
        build_scale_table(lut, f.w1.mx);
        wait_lgkmcnt0();   // only LDS writes need to be seen (the ring's loads stay in flight)
        asm volatile("s_barrier" ::: "memory");
    };
    const float gv = global_scale_at(f.g1, e, f.g_div);
    small_m_pass<1, NT, kFewDepth1, false, F16, PRE>(f.x, f.ld_x, rows, f.pre1, ww, c0, c1, f.H, lut, red[w], RLD, lane,
                                                     mid, tokens);
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
        float v = ACT == kActSiluGlu ? silu_times(gv * s0, gv * s1) : relu_squared(gv * s0);
        if (n < f.I) {
            if (f.pre2) v = fp32_value(v * act_to_f32<F16>(f.pre2[n]));
            const int64_t row = f.KC2 * kChunkK;
            uint16_t* to = f.a + pairs[r] * row + n;
            few_split(v, to, f.P * row);
            if ((int)blockIdx.x * 16 + 16 == f.I)   // the last columns' workgroup: zeros to the chunk's end
                for (int past = 16; n + past < row; past += 16) few_split(0.f, to + past, f.P * row);
        }
    }
}

// What a wave of k_moe_few_fc2 has on its way of a chunk.
struct FewSlot {
    uint4 cw, xa[kFewParts];
    uint32_t sw;
};

// One chunk of an item: the small-M GEMM's contraction (kernels_gemm.h) with a's
// parts one after another into the same sums.  The weights enter as bare E2M1
// values, their scales multiply the sums of 16 columns.
__device__ __forceinline__ void few_chunk(const FewSlot& s, const float* lut, int lane, f32x4& acc) {
    const uint32_t sp = scale_pair(s.sw, lane);
    const float s0 = lut[sp & 0xFFu], s1 = lut[(sp >> 8) & 0xFFu];
    const s16x4 b0 = decode4_pow2<false, 0>(s.cw.x, 1.f), b1 = decode4_pow2<false, 2>(s.cw.x, 1.f);
    const s16x4 b2 = decode4_pow2<false, 0>(s.cw.y, 1.f), b3 = decode4_pow2<false, 2>(s.cw.y, 1.f);
    const s16x4 b4 = decode4_pow2<false, 0>(s.cw.z, 1.f), b5 = decode4_pow2<false, 2>(s.cw.z, 1.f);
    const s16x4 b6 = decode4_pow2<false, 0>(s.cw.w, 1.f), b7 = decode4_pow2<false, 2>(s.cw.w, 1.f);
    f32x4 p = {0.f, 0.f, 0.f, 0.f}, r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int part = kFewParts - 1; part >= 0; --part) {   // the smallest first
        const s16x4 lo = dwords_to_s16x4(s.xa[part].x, s.xa[part].y), hi = dwords_to_s16x4(s.xa[part].z, s.xa[part].w);
        p = mma4<false, 2, 0>(lo, b0, p);
        r = mma4<false, 2, 2>(lo, b4, r);
        p = mma4<false, 2, 0>(hi, b1, p);
        r = mma4<false, 2, 2>(hi, b5, r);
        p = mma4<false, 2, 1>(lo, b2, p);
        r = mma4<false, 2, 3>(lo, b6, r);
        p = mma4<false, 2, 1>(hi, b3, p);
        r = mma4<false, 2, 3>(hi, b7, r);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(s1, r[i], __builtin_fmaf(s0, p[i], acc[i]));
}

struct FewShared {
    float lut[256];   // the weights' scales
    FewItem item[kFewPairs];
    int32_t pair[kFewPairs];
    float weight[kFewPairs];
    int flag;
};

// Grid: (units of W2, S).  A wave's stretch of the items' chunks is streamed
// by one ring; sums[token][16] of each wave in dynamic LDS.
template <bool F16>
__global__ void __launch_bounds__(kFewWaves * 64) k_moe_few_fc2(FewArgs f) {
    __shared__ FewShared sh;
    extern __shared__ float sums[];   // [kFewWaves][T * 16]
    constexpr int kThreads = kFewWaves * 64;
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int u = blockIdx.x, S = f.sk.S, s = blockIdx.y;
    const int out_n = f.T * 16;
    const int items = f.list->items;
    for (int i = tid; i < f.P; i += kThreads) {   // (what is past the items and their pairs is not read)
        sh.item[i] = f.list->item[i];
        sh.pair[i] = f.list->pair[i];
        sh.weight[i] = f.list->weight[i];
    }
    for (int b = tid; b < 256; b += kThreads) sh.lut[b] = f.w2.mx ? e8m0_to_f32((uint32_t)b) : e4m3_to_f32((uint32_t)b);
    for (int i = tid; i < kFewWaves * out_n; i += kThreads) sums[i] = 0.f;
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
        uint32_t row = 0;   // the byte offset of this lane's piece of its pair's row
        auto enter = [&]() {   // the load side's item
            const int e = __builtin_amdgcn_readfirstlane(sh.item[ld.item].e);
            const int first = sh.item[ld.item].first, rows = sh.item[ld.item].rows;
            const int64_t blk = f.w2.block(e, u, 0);
            codes = f.w2.codes + blk * kCodeBlock;
            scales = f.w2.scales + blk * kScaleBlock;
            row = (uint32_t)(sh.pair[first + (ai < rows ? ai : 0)] * f.KC2 * kChunkK + kpiece) * 2;
        };
        enter();
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        const uint8_t* ab = reinterpret_cast<const uint8_t*>(f.a);
        const int64_t part_bytes = (int64_t)f.P * f.KC2 * kChunkK * 2;
        auto load = [&](FewSlot& slot, int64_t i) {
            if (i > ld_i) {   // i is the last one, or one more
                ld_i = i;
                if (++ld.chunk == f.KC2) {
                    ld.chunk = 0;
                    ++ld.item;
                    enter();
                }
            }
            const int64_t off = (int64_t)ld.chunk * f.w2.chunk_stride;
            slot.cw = load_stream_u4(codes + off * kCodeBlock + (uint32_t)(lane * 16));
            slot.sw = load_scale_dword(scales + off * kScaleBlock, lane);
            const uint8_t* ac = ab + ld.chunk * (kChunkK * 2);
#pragma unroll
            for (int part = 0; part < kFewParts; ++part)
                slot.xa[part] = *reinterpret_cast<const uint4*>(ac + part * part_bytes + row);
        };
        auto use = [&](const FewSlot& slot, int64_t i) {
            few_chunk(slot, sh.lut, lane, acc);
            const bool ends = us.chunk == f.KC2 - 1;
            if (ends || i == n - 1) {
                // the item's rows into the tokens' sums: lane l < 16 has column l
                const int first = sh.item[us.item].first, rows = sh.item[us.item].rows;
                const float gv = sh.item[us.item].g;
#pragma unroll
                for (int r = 0; r < kFewItem; ++r) {
                    float v = acc[r];
                    v += __shfl_xor(v, 16);
                    v += __shfl_xor(v, 32);
                    if (lane < 16 && r < rows) {
                        float* to = mine + sh.pair[first + r] / f.k * 16 + lane;
                        *to = __builtin_fmaf(sh.weight[first + r] * gv, v, *to);
                    }
                }
                acc = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            if (ends) ++us.item, us.chunk = 0;
            else ++us.chunk;
        };
        FewSlot ring[kFewDepth];
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
