// Attention of one new token per sequence over the paged key-value cache,
// split over the cache's length and joined.
#pragma once
#include "decode.h"
#include "kernels_gemm.h"
#include "kernels_kv.h"

namespace nvfp4 {

struct AttnArgs {
    const uint16_t* q;           // [B][Hq][D]
    int64_t q_b, q_h;            // strides in elements
    KvSide kc, vc;
    KvShape shape;
    const int32_t* table;        // [B][ld_table], `width` entries used
    int64_t ld_table;
    int width;
    const int32_t* lengths;      // [B]
    int G;                       // query heads per key-value head
    int head_tiles;              // ceil(G / 16)
    int Hq;
    int window;                  // 0: all tokens
    float scale_log2;            // softmax scale * log2(e)
    uint16_t* out;
    int64_t o_b, o_h;
    float* lse;                  // [B][Hq] or NULL
    int f16;                     // q and out are fp16 (else bf16)
    int S;                       // splits (grid x)
    float* partials;             // [B * Hk * head_tiles][S][min(G, 16) * (D + 2)]: sums, then (maximum, sum) pairs
    int* counters;               // [B * Hk * head_tiles], zero between calls
};

constexpr int kAttnWaves = 4;
constexpr int kAttnTile = 32;                               // tokens a wave takes at a time
constexpr int kAttnChunk = kAttnWaves * kAttnTile;          // a split takes a multiple of this
constexpr int kAttnHeads = 16;                              // query heads of one workgroup

// Passes in which a workgroup's accumulators go through LDS.
constexpr int attn_out_passes(int DT) { return DT > 128 ? 2 : 1; }

// Tokens of one split of a sequence of n tokens over S splits.
__device__ __forceinline__ int attn_split_tokens(int n, int S) {
    const int per = (int)(((int64_t)n + S - 1) / S);
    return (per + kAttnChunk - 1) / kAttnChunk * kAttnChunk;
}

// Workgroup (s, h, b): split s of key-value head h / head_tiles of sequence
// b, for up to 16 of that head's query heads.  Its waves take tiles of 32
// tokens in turn, each with its own running maximum, sum and accumulators,
// so the loop has no barrier.
//
// A wave's tile:
//   S^T = K Q^T       mfma 16x16x32, rows = tokens, columns = heads: lane (g, c)
//                     (g = lane / 16, c = lane % 16) loads 16-byte pieces of
//                     token c's key row straight into the A operand, and gets
//                     the scores of head c for tokens 4 g .. 4 g + 3;
//   softmax           all of a lane's values belong to head c; the four lanes
//                     of a head exchange maxima only (two steps);
//   O^T += V^T P^T    rows = columns of V, columns = heads: the contraction
//                     slots are numbered so that lane (g, c) holds in slots
//                     0..3 / 4..7 the tokens 4 g .. of the tile's two halves,
//                     which are the tokens whose weights it just computed, so
//                     P goes from the scores to the B operand inside the lane.
//                     V's rows are loaded as stored (lane c: columns c VD ..
//                     c VD + VD - 1, VD = DT / 16) and transposed in
//                     registers, one byte permute per two values; MFMA e takes
//                     the columns c VD + e.
// Nothing passes through LDS but the tile's 32 row offsets (each wave its own).
//
// Quantised caches are decoded to fp16, which holds E4M3 and E2M1 x E4M3
// exactly; q is scaled to [1, 2) by a power of two per head so that it fits,
// and the weights p <= 1 are rounded to fp16 (bf16 with a bf16 cache) for the
// second product; the sum of the weights is taken in fp32 before that.  The
// heads' key scale goes into the softmax scale, the value scale into the
// final normalisation.
//
// Tokens past the length, and tokens of pages whose table entry is outside
// the cache, get the weight 0 and their value rows are replaced by zeros, so
// nothing in them (an infinity, a NaN) reaches the result; their rows are not
// read either (the address falls back to the cache's first row).
template <int FMT, int DT, bool FULL>
struct AttnTile {
    static constexpr bool F16 = FMT != 0;                   // type of the products: 0 is a bf16 cache
    static constexpr int KV = FMT <= 1 ? kKv16 : FMT == 2 ? kKvE4m3 : kKvNvfp4;
    static constexpr int KSTEPS = DT / 32;                  // 32-column steps of the first product
    static constexpr int VD = DT / 16;                      // value columns of a lane
};

// fp16 pair of two E4M3 bytes / two E2M1 codes
template <bool HI>
__device__ __forceinline__ uint32_t f16_of_e4m3(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
}
__device__ __forceinline__ uint32_t f16_times(uint32_t a, f16x2v s) {
    return __builtin_bit_cast(uint32_t, (f16x2v)(__builtin_bit_cast(f16x2v, a) * s));
}
// eight E2M1 codes times an E4M3 group scale, exact in fp16 (at most 6
// significant bits, magnitudes 2^-10 .. 2688 or 0)
__device__ __forceinline__ uint4 f16_of_nvfp4(uint32_t codes, f16x2v s) {
    return make_uint4(
        f16_times(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0)), s),
        f16_times(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1)), s),
        f16_times(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2)), s),
        f16_times(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3)), s));
}
__device__ __forceinline__ f16x2v f16_group_scale(uint32_t pair_bytes, bool second) {
    const uint32_t p = f16_of_e4m3<false>(pair_bytes);
    const uint32_t h = second ? (p >> 16) : (p & 0xFFFFu);
    return __builtin_bit_cast(f16x2v, h | (h << 16));
}

template <int FMT, int DT, bool FULL>
__global__ void __launch_bounds__(kAttnWaves * 64) k_paged_attn(AttnArgs a) {
    using X = AttnTile<FMT, DT, FULL>;
    constexpr int KSTEPS = X::KSTEPS, VD = X::VD, KV = X::KV;
    constexpr bool F16 = X::F16;
    const int D = FULL ? DT : a.shape.D;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
    const int s = blockIdx.x, b = blockIdx.z;
    const int hk = blockIdx.y / a.head_tiles, ht = blockIdx.y - hk * a.head_tiles;
    const int nh = a.G - ht * kAttnHeads < kAttnHeads ? a.G - ht * kAttnHeads : kAttnHeads;
    const int head0 = hk * a.G + ht * kAttnHeads;

    __shared__ uint32_t s_off[kAttnWaves][3][kAttnTile];
    __shared__ float s_m[kAttnWaves][kAttnHeads], s_l[kAttnWaves][kAttnHeads];
    __shared__ int s_flag;
    // the waves' accumulators on their way out: [waves][nh][OS], in two passes of half the columns for DT = 256
    // (one pass would take 65 KB at 16 heads)
    extern __shared__ float s_o[];
    constexpr int PASSES = attn_out_passes(DT), RP = 4 / PASSES;   // accumulator rows of a lane per pass
    constexpr int LD = DT / PASSES, OS = LD + 4;                   // 16-byte aligned rows, spread over the banks

    int len = a.lengths[b];
    const int64_t most = (int64_t)a.width * a.shape.page_size;
    len = len < 0 ? 0 : ((int64_t)len > most ? (int)most : len);
    const int first = a.window > 0 && len > a.window ? len - a.window : 0;
    const int n = len - first;
    const int per = n > 0 ? attn_split_tokens(n, a.S) : kAttnChunk;
    const int parts = n > 0 ? (n + per - 1) / per : 1;
    if (s >= parts) return;
    const int t_end = first + (n < (s + 1) * (int64_t)per ? n : (s + 1) * per);   // one past the split's last token
    const int t_begin = first + s * per;

    // q of head c as the B operand of each 32-column step: the columns of step
    // j are the ones key pieces deliver (see key_columns below)
    uint4 qf[KSTEPS];
    float qk_log2 = a.scale_log2;
    auto key_column = [&](int j) {   // first of the 8 columns lane (g, c) holds in step j
        if constexpr (KV == kKv16) return j * 32 + g * 8;
        else if constexpr (KV == kKvE4m3) return (j >> 1) * 64 + g * 16 + (j & 1) * 8;
        else if constexpr (DT == 64) return g * 16 + j * 8;
        else return (j >> 2) * 128 + g * 32 + (j & 3) * 8;
    };
    {
        const uint16_t* qr = a.q + b * a.q_b + (int64_t)(head0 + (c < nh ? c : 0)) * a.q_h;
#pragma unroll
        for (int j = 0; j < KSTEPS; ++j) {
            const int col = key_column(j);
            const bool in = c < nh && (FULL || col < D);
            qf[j] = in ? *reinterpret_cast<const uint4*>(qr + col) : make_uint4(0u, 0u, 0u, 0u);
        }
        if constexpr (KV != kKv16) {
            uint32_t top = 0u;
            float f[KSTEPS][8];
#pragma unroll
            for (int j = 0; j < KSTEPS; ++j) {
                if (a.f16) unpack8<true>(qf[j], f[j]);
                else unpack8<false>(qf[j], f[j]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t u = __float_as_uint(f[j][e]) & 0x7FFFFFFFu;
                    top = u > top ? u : top;
                }
            }
            uint32_t o = __shfl_xor(top, 16);
            top = o > top ? o : top;
            o = __shfl_xor(top, 32);
            top = o > top ? o : top;
            int ex = (int)(top >> 23);
            ex = ex < 1 ? 1 : (ex > 253 ? 253 : ex);
            const float down = __uint_as_float((uint32_t)(254 - ex) << 23);   // 2^(127 - ex)
#pragma unroll
            for (int j = 0; j < KSTEPS; ++j) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[j][e] *= down;
                qf[j] = pack8<true>(f[j]);
            }
            qk_log2 *= __uint_as_float((uint32_t)ex << 23);
            if (a.kc.scale) qk_log2 *= a.kc.scale[hk];
        }
    }

    f32x4 acc[VD];
#pragma unroll
    for (int e = 0; e < VD; ++e) acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;

    const uint8_t* kb = a.kc.base + (KV == kKvNvfp4 ? 0 : hk * a.kc.s_head);
    const uint8_t* vb = a.vc.base + (KV == kKvNvfp4 ? 0 : hk * a.vc.s_head);
    const int32_t* table = a.table + b * a.ld_table;
    const int ps = a.shape.page_size;

    const int step = kAttnWaves * kAttnTile;
    int t0 = t_begin + w * kAttnTile;
    auto page_of = [&](int t) {   // table entry of token t (-1 past the split's end)
        return t < t_end ? table[(uint32_t)t / (uint32_t)ps] : -1;
    };
    int next_page = lane < kAttnTile ? page_of(t0 + lane) : -1;
    for (; t0 < t_end; t0 += step) {
        // ---- the tile's row offsets, 16 bytes a unit
        uint32_t valid;
        {
            const int t = t0 + lane;
            const int page = next_page;
            const bool ok = lane < kAttnTile && t < t_end && page >= 0 && (int64_t)page < a.shape.pages;
            valid = (uint32_t)__ballot(ok);
            if (lane < kAttnTile) {
                const int tok = (int)((uint32_t)t % (uint32_t)ps);
                if constexpr (KV == kKvNvfp4) {
                    s_off[w][0][lane] = ok ? (uint32_t)((page * a.kc.s_page + hk * a.kc.s_head) >> 4) : 0u;
                    s_off[w][1][lane] = ok ? (uint32_t)((page * a.vc.s_page + hk * a.vc.s_head) >> 4) : 0u;
                    s_off[w][2][lane] = ok ? (uint32_t)tok : 0u;
                } else {
                    s_off[w][0][lane] = ok ? (uint32_t)((page * a.kc.s_page + tok * a.kc.s_token) >> 4) : 0u;
                    s_off[w][1][lane] = ok ? (uint32_t)((page * a.vc.s_page + tok * a.vc.s_token) >> 4) : 0u;
                }
                next_page = page_of(t + step);
            }
            // a wave's LDS accesses complete in order: only the compiler has to keep theirs
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        // ---- loads: keys of tokens c and 16 + c, values of the lane's eight slots
        constexpr int KP = KV == kKv16 ? KSTEPS : KV == kKvE4m3 ? KSTEPS / 2 : (DT == 256 ? 2 : 1);   // 16-byte pieces of a key row
        uint4 kraw[2][KP];
        uint32_t ksc[2][KP];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t off = s_off[w][0][h * 16 + c];
            if constexpr (KV == kKvNvfp4) {
                const uint32_t tok = s_off[w][2][h * 16 + c];
                const uint8_t* blk = kb + (uint64_t)off * 16u;
                const uint8_t* row = blk + (int64_t)tok * (D / 2);
                const uint8_t* srow = blk + (int64_t)ps * (D / 2) + (int64_t)tok * (D / 16);
#pragma unroll
                for (int p = 0; p < KP; ++p) {
                    const int col = DT == 64 ? g * 16 : p * 128 + g * 32;
                    const bool in = FULL || col < D;
                    if constexpr (DT == 64) {
                        const uint2 v = in ? *reinterpret_cast<const uint2*>(row + col / 2) : make_uint2(0u, 0u);
                        kraw[h][p] = make_uint4(v.x, v.y, 0u, 0u);
                        ksc[h][p] = in ? srow[col / 16] : 0u;
                    } else {
                        kraw[h][p] = in ? *reinterpret_cast<const uint4*>(row + col / 2) : make_uint4(0u, 0u, 0u, 0u);
                        ksc[h][p] = in ? *reinterpret_cast<const uint16_t*>(srow + col / 16) : 0u;
                    }
                }
            } else {
                const uint8_t* row = kb + (uint64_t)off * 16u;
#pragma unroll
                for (int p = 0; p < KP; ++p) {
                    const int col = KV == kKv16 ? p * 32 + g * 8 : p * 64 + g * 16;
                    const bool in = FULL || col < D;
                    kraw[h][p] = in ? *reinterpret_cast<const uint4*>(row + col * (KV == kKv16 ? 2 : 1))
                                    : make_uint4(0u, 0u, 0u, 0u);
                }
            }
        }
        constexpr int VB = KV == kKv16 ? VD * 2 : KV == kKvE4m3 ? VD : VD / 2;   // bytes of a lane's value columns
        constexpr int VW = VB < 4 ? 1 : VB / 4;                                  // dwords
        uint32_t vraw[8][VW];
        uint32_t vsc[8];
        const bool vin = FULL || c * VD < D;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int slot = (i >> 2) * 16 + g * 4 + (i & 3);
            const uint32_t off = s_off[w][1][slot];
            const uint8_t* row = vb + (uint64_t)off * 16u;
            const uint8_t* srow = nullptr;
            if constexpr (KV == kKvNvfp4) {
                const uint32_t tok = s_off[w][2][slot];
                srow = row + (int64_t)ps * (D / 2) + (int64_t)tok * (D / 16);
                row += (int64_t)tok * (D / 2);
            }
            row += c * VB;
#pragma unroll
            for (int x = 0; x < VW; ++x) vraw[i][x] = 0u;
            vsc[i] = 0u;
            if (vin) {
                if constexpr (VB == 2) vraw[i][0] = *reinterpret_cast<const uint16_t*>(row);
                else if constexpr (VB == 4) vraw[i][0] = *reinterpret_cast<const uint32_t*>(row);
                else if constexpr (VB == 8) {
                    const uint2 v = *reinterpret_cast<const uint2*>(row);
                    vraw[i][0] = v.x;
                    vraw[i][1] = v.y;
                } else {
#pragma unroll
                    for (int x = 0; x < VB / 16; ++x) {
                        const uint4 v = *reinterpret_cast<const uint4*>(row + x * 16);
                        vraw[i][4 * x] = v.x;
                        vraw[i][4 * x + 1] = v.y;
                        vraw[i][4 * x + 2] = v.z;
                        vraw[i][4 * x + 3] = v.w;
                    }
                }
                if constexpr (KV == kKvNvfp4) vsc[i] = srow[c * VD / 16];
            }
        }
        // ---- scores
        f32x4 sc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sc[h] = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (KV == kKv16) {
#pragma unroll
                for (int j = 0; j < KSTEPS; ++j) sc[h] = mma16<F16>(kraw[h][j], qf[j], sc[h]);
            } else if constexpr (KV == kKvE4m3) {
#pragma unroll
                for (int p = 0; p < KP; ++p) {
                    const uint4 v = kraw[h][p];
                    sc[h] = mma16<true>(make_uint4(f16_of_e4m3<false>(v.x), f16_of_e4m3<true>(v.x),
                                                   f16_of_e4m3<false>(v.y), f16_of_e4m3<true>(v.y)), qf[2 * p], sc[h]);
                    sc[h] = mma16<true>(make_uint4(f16_of_e4m3<false>(v.z), f16_of_e4m3<true>(v.z),
                                                   f16_of_e4m3<false>(v.w), f16_of_e4m3<true>(v.w)), qf[2 * p + 1], sc[h]);
                }
            } else {
#pragma unroll
                for (int p = 0; p < KP; ++p) {
                    const uint32_t cw[4] = {kraw[h][p].x, kraw[h][p].y, kraw[h][p].z, kraw[h][p].w};
                    constexpr int W = DT == 64 ? 2 : 4;
#pragma unroll
                    for (int x = 0; x < W; ++x)
                        sc[h] = mma16<true>(f16_of_nvfp4(cw[x], f16_group_scale(ksc[h][p], x >= 2)), qf[p * W + x], sc[h]);
                }
            }
        }
        // ---- weights of the lane's eight tokens
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = sc[i >> 2][i & 3] * qk_log2;
        if (valid != 0xFFFFFFFFu) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool ok = (valid >> ((i >> 2) * 16 + g * 4 + (i & 3))) & 1u;
                x[i] = ok ? x[i] : -INFINITY;
                vsc[i] = ok ? vsc[i] : 0u;
#pragma unroll
                for (int y = 0; y < VW; ++y) vraw[i][y] = ok ? vraw[i][y] : 0u;
            }
        }
        float top = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, x[i]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        if (__any(top > m)) {
            const float mn = fmaxf(m, top);
            const float down = m == mn ? 1.0f : __builtin_amdgcn_exp2f(m - mn);   // m = -inf gives 0
            m = mn;
            l *= down;
#pragma unroll
            for (int e = 0; e < VD; ++e) acc[e] *= down;
        }
        const float ms = m == -INFINITY ? 0.f : m;
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = __builtin_amdgcn_exp2f(x[i] - ms);
            l += p[i];
        }
        const uint4 pf = make_uint4(pack_round2<F16>(p[0], p[1]), pack_round2<F16>(p[2], p[3]),
                                    pack_round2<F16>(p[4], p[5]), pack_round2<F16>(p[6], p[7]));
        // ---- values: 16-bit words of (token pair, column)
        constexpr int HW = VD / 2;   // dwords of a lane's row in 16 bits
        uint32_t vh[8][HW];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (KV == kKv16) {
#pragma unroll
                for (int y = 0; y < HW; ++y) vh[i][y] = vraw[i][y];
            } else if constexpr (KV == kKvE4m3) {
#pragma unroll
                for (int y = 0; y < HW; ++y)
                    vh[i][y] = (y & 1) ? f16_of_e4m3<true>(vraw[i][y >> 1]) : f16_of_e4m3<false>(vraw[i][y >> 1]);
            } else {
                const f16x2v gs = f16_group_scale(vsc[i], false);
                if constexpr (VD == 4) {
                    vh[i][0] = f16_times(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(vraw[i][0], 1.0f, 0)), gs);
                    vh[i][1] = f16_times(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(vraw[i][0], 1.0f, 1)), gs);
                } else {
#pragma unroll
                    for (int y = 0; y < VW; ++y) {
                        const uint4 d = f16_of_nvfp4(vraw[i][y], gs);
                        vh[i][4 * y] = d.x;
                        vh[i][4 * y + 1] = d.y;
                        vh[i][4 * y + 2] = d.z;
                        vh[i][4 * y + 3] = d.w;
                    }
                }
            }
        }
#pragma unroll
        for (int e = 0; e < VD; ++e) {
            const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;
            const int y = e >> 1;
            const uint4 vf = make_uint4(__builtin_amdgcn_perm(vh[1][y], vh[0][y], sel),
                                        __builtin_amdgcn_perm(vh[3][y], vh[2][y], sel),
                                        __builtin_amdgcn_perm(vh[5][y], vh[4][y], sel),
                                        __builtin_amdgcn_perm(vh[7][y], vh[6][y], sel));
            acc[e] = mma16<F16>(vf, pf, acc[e]);
        }
    }

    // ---- join the waves: every lane's sum is of its own tokens, its maximum of all four groups'
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
        s_m[w][c] = m;
        s_l[w][c] = l;
    }
    const int64_t pair = (int64_t)b * gridDim.y + blockIdx.y;
    const int hp = a.G < kAttnHeads ? a.G : kAttnHeads;
    const int64_t part_floats = (int64_t)hp * (D + 2);
    float* part = a.partials + (pair * a.S + s) * part_floats;
    const float vscale = KV != kKv16 && a.vc.scale ? a.vc.scale[hk] : 1.0f;
    auto store_out = [&](int h, int d, float v0, float v1) {
        const uint32_t o = a.f16 ? pack_round2<true>(fp32_value(v0), fp32_value(v1))
                                 : pack_round2<false>(fp32_value(v0), fp32_value(v1));
        *reinterpret_cast<uint32_t*>(a.out + b * a.o_b + (int64_t)(head0 + h) * a.o_h + d) = o;
    };
    auto store_lse = [&](int h, float mm, float ll) {
        if (a.lse) a.lse[(int64_t)b * a.Hq + head0 + h] = ll > 0.f ? (mm + __log2f(ll)) * 0.69314718055994530942f : (ll == 0.f ? -INFINITY : ll);
    };
    for (int pass = 0; pass < PASSES; ++pass) {
        if (pass > 0) __syncthreads();
        if (c < nh) {
#pragma unroll
            for (int rr = 0; rr < RP; ++rr)
#pragma unroll
                for (int e = 0; e < VD; ++e) {
                    float v = acc[e][rr];
                    if (PASSES > 1 && pass == 1) v = acc[e][(RP + rr) & 3];
                    s_o[(w * nh + c) * OS + (g * RP + rr) * VD + e] = v;
                }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < nh * (LD / 2); i += kAttnWaves * 64) {
            const int h = i / (LD / 2), ld = (i - h * (LD / 2)) * 2;
            // local column -> column: (4 g + row) VD + e
            const int d = ((ld / (RP * VD)) * 4 + pass * RP) * VD + ld % (RP * VD);
            if (!FULL && d >= D) continue;
            float mm = s_m[0][h];
#pragma unroll
            for (int x = 1; x < kAttnWaves; ++x) mm = fmaxf(mm, s_m[x][h]);
            float ll = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
            for (int x = 0; x < kAttnWaves; ++x) {
                const float f = s_m[x][h] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(s_m[x][h] - mm);
                ll += f * s_l[x][h];
                o0 += f * s_o[(x * nh + h) * OS + ld];
                o1 += f * s_o[(x * nh + h) * OS + ld + 1];
            }
            if (parts == 1) {
                const float inv = ll == 0.f ? 0.f : vscale / ll;
                store_out(h, d, o0 * inv, o1 * inv);
                if (d == 0) store_lse(h, mm, ll);
            } else {
                // 8-byte agent-scope stores: coherent across the XCDs' L2 caches
                __hip_atomic_store(reinterpret_cast<uint64_t*>(part + h * D + d),
                                   (uint64_t)__float_as_uint(o0) | ((uint64_t)__float_as_uint(o1) << 32),
                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                if (d == 0)
                    __hip_atomic_store(reinterpret_cast<uint64_t*>(part + hp * D + 2 * h),
                                       (uint64_t)__float_as_uint(mm) | ((uint64_t)__float_as_uint(ll) << 32),
                                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
    }
    if (parts == 1) return;
    if (!split_arrive(a.counters, pair, parts, &s_flag)) return;
    // ---- the split that arrived last joins all of them, in their order
    const float* parts0 = a.partials + pair * a.S * part_floats;
    auto load2 = [&](const float* at) {
        return __hip_atomic_load(reinterpret_cast<const uint64_t*>(at), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    const int half = D / 2;
    for (int i = threadIdx.x; i < nh * half; i += kAttnWaves * 64) {
        const int h = i / half, d = (i - h * half) * 2;
        float mm = -INFINITY;
        for (int x = 0; x < parts; ++x)
            mm = fmaxf(mm, __uint_as_float((uint32_t)load2(parts0 + x * part_floats + hp * D + 2 * h)));
        float ll = 0.f, o0 = 0.f, o1 = 0.f;
        for (int x = 0; x < parts; ++x) {
            const uint64_t ml = load2(parts0 + x * part_floats + hp * D + 2 * h);
            const uint64_t o = load2(parts0 + x * part_floats + h * D + d);
            const float mx = __uint_as_float((uint32_t)ml);
            const float f = mx == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mx - mm);
            ll += f * __uint_as_float((uint32_t)(ml >> 32));
            o0 += f * __uint_as_float((uint32_t)o);
            o1 += f * __uint_as_float((uint32_t)(o >> 32));
        }
        const float inv = ll == 0.f ? 0.f : vscale / ll;
        store_out(h, d, o0 * inv, o1 * inv);
        if (d == 0) store_lse(h, mm, ll);
    }
}

}  // namespace nvfp4
