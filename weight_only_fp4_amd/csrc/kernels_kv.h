// Rotary positions with several axes, the paged key-value cache's writes
// (16-bit, E4M3 or NVFP4 rows) and its read back.
#pragma once
#include "decode.h"
#include "quant.h"

namespace nvfp4 {

constexpr int kKv16 = 0, kKvE4m3 = 1, kKvNvfp4 = 2;

// One side (keys or values) of the paged cache on the device.  A (page, head)
// block starts at base + page * s_page + head * s_head; token i of the page
// starts s_token bytes further each (16-bit and E4M3 rows).  An NVFP4 block
// holds the codes of its tokens back to back (D / 2 bytes each) and then
// their group scales (D / 16 bytes each).
struct KvSide {
    uint8_t* base;
    int64_t s_page, s_head, s_token;   // bytes
    const float* scale;                // per head, or NULL (1)
};
struct KvShape {
    int64_t pages;
    int page_size, heads, D;
};

// Row `slot` of the cache is token slot % page_size of page slot / page_size;
// false for a slot outside it.
__device__ __forceinline__ bool kv_locate(const KvShape& s, int32_t slot, int64_t& page, int& tok) {
    if (slot < 0) return false;
    page = (uint32_t)slot / (uint32_t)s.page_size;
    tok = (int)((uint32_t)slot - (uint32_t)page * (uint32_t)s.page_size);
    return page < s.pages;
}

// Codes and group scales of token `tok` in an NVFP4 block, which may pass 2 GB
// (a page of 2^24 tokens of 256 columns): 64-bit offsets.
template <typename B>
__device__ __forceinline__ B* kv_code_row(B* block, const KvShape& s, int tok) {
    return block + (int64_t)tok * (s.D / 2);
}
template <typename B>
__device__ __forceinline__ B* kv_scale_row(B* block, const KvShape& s, int tok) {
    return block + (int64_t)s.page_size * (s.D / 2) + (int64_t)tok * (s.D / 16);
}

// ------------------------------------------------------------------ rotary --

struct RopeArgs {
    const float* inv_freq;       // [R / 2]
    const int32_t* positions;    // [axes][ld_pos]
    const int32_t* pair_axis;    // [R / 2] or NULL (axis 0)
    int64_t ld_pos;
    int axes, R;                 // R = 0: nothing is rotated
};

// sin and cos of a position times a frequency.  The product is taken in fp64
// (31 + 24 bits: its rounding is 2^-53 of the angle), reduced to [-pi/4,
// pi/4] by a two-term multiple of pi/2 (fused, so the first subtraction is
// exact up to one rounding) and evaluated by the Taylor series: the first
// terms left out are below 3e-14 there.  Rounded to fp32 once; an fp32 angle
// would be off by 2^-24 of itself, 0.06 rad at position 10^6.
__device__ __forceinline__ float2 rope_cos_sin(int32_t pos, float freq) {
    const double a = (double)pos * (double)freq;
    const double n = __builtin_rint(a * 0.63661977236758134308);   // 2 / pi
    double r = __builtin_fma(n, -1.57079632679489655800, a);       // pi / 2 rounded to fp64 ...
    r = __builtin_fma(n, -6.12323399573676603587e-17, r);          // ... and what that leaves
    const double z = r * r;
    double s = 1.0 / 6227020800.0;                                 // 1 / 13!
    s = __builtin_fma(s, z, -1.0 / 39916800.0);
    s = __builtin_fma(s, z, 1.0 / 362880.0);
    s = __builtin_fma(s, z, -1.0 / 5040.0);
    s = __builtin_fma(s, z, 1.0 / 120.0);
    s = __builtin_fma(s, z, -1.0 / 6.0);
    s = __builtin_fma(s * z, r, r);
    double c = 1.0 / 479001600.0;                                  // 1 / 12!
    c = __builtin_fma(c, -z, 1.0 / 3628800.0);
    c = __builtin_fma(c, -z, 1.0 / 40320.0);
    c = __builtin_fma(c, -z, 1.0 / 720.0);
    c = __builtin_fma(c, -z, 1.0 / 24.0);
    c = __builtin_fma(c, -z, 0.5);
    c = __builtin_fma(c, -z, 1.0);
    const long long q = (long long)n;
    const double cc = (q & 1) ? s : c, ss = (q & 1) ? c : s;
    return make_float2((float)(((q + 1) & 2) ? -cc : cc), (float)((q & 2) ? -ss : ss));
}

// One pair turned: every product and sum is rounded to fp32 by itself, so the
// result does not depend on what the compiler would fuse.
__device__ __forceinline__ void rope_turn(float& x0, float& x1, float2 cs) {
#pragma clang fp contract(off)
    const float a = x0 * cs.x, b = x1 * cs.y, c = x1 * cs.x, d = x0 * cs.y;
    x0 = a - b;
    x1 = c + d;
}

// ------------------------------------------------------- rotate and append --

struct AppendArgs {
    RopeArgs rope;
    // queries: rotated into q_out (NULL q with Hq = 0)
    const uint16_t* q;
    uint16_t* q_out;
    int64_t q_t, q_h, qo_t, qo_h;        // strides in elements: token, head
    int Hq;
    // keys and values into the cache (Hk = 0: none)
    const uint16_t *k, *v;
    int64_t k_t, k_h, v_t, v_h;
    int Hk;
    const int32_t* slots;
    KvSide kc, vc;
    KvShape shape;
    int64_t T;
    int D;
};

// Stores 16 values of one cache row: with `pair` the 8 + 8 columns c0.. and
// c1.., else the 16 columns c0...  NVFP4 pairs: the two threads of a 16-column
// group (lanes 2i, 2i + 1) exchange their largest values; the even one writes
// the first group's scale, the odd one the second's.
template <int FMT, bool F16>
__device__ __forceinline__ void kv_store16(const KvSide& side, const KvShape& sh, bool there, int64_t page, int tok,
                                           int head, int c0, int c1, bool pair, const float (&lo)[8],
                                           const float (&hi)[8]) {
    uint8_t* block = side.base + page * side.s_page + head * side.s_head;
    if constexpr (FMT == kKv16) {
        if (!there) return;
        uint8_t* row = block + tok * side.s_token;
        *reinterpret_cast<uint4*>(row + c0 * 2) = pack8<F16>(lo);
        *reinterpret_cast<uint4*>(row + c1 * 2) = pack8<F16>(hi);
        return;
    }
    const float r = side.scale ? __fdiv_rn(1.0f, side.scale[head]) : 1.0f;
    if constexpr (FMT == kKvE4m3) {
        if (!there) return;
        uint8_t* row = block + tok * side.s_token;
        *reinterpret_cast<uint2*>(row + c0) = e4m3_pack8(lo, r);
        *reinterpret_cast<uint2*>(row + c1) = e4m3_pack8(hi, r);
        return;
    }
    if constexpr (FMT == kKvNvfp4) {
        uint32_t m0 = 0u, m1 = 0u;   // largest absolute values as bits: a NaN's are above infinity's
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t a = __float_as_uint(lo[e]) & 0x7FFFFFFFu, b = __float_as_uint(hi[e]) & 0x7FFFFFFFu;
            m0 = a > m0 ? a : m0;
            m1 = b > m1 ? b : m1;
        }
        if (pair) {
            const uint32_t o0 = __shfl_xor(m0, 1), o1 = __shfl_xor(m1, 1);
            m0 = o0 > m0 ? o0 : m0;
            m1 = o1 > m1 ? o1 : m1;
        } else {
            m0 = m1 > m0 ? m1 : m0;
            m1 = m0;
        }
        if (!there) return;
        const uint32_t b0 = nvfp4_group_scale(__uint_as_float(m0), r), b1 = nvfp4_group_scale(__uint_as_float(m1), r);
        const float f0 = nvfp4_group_factor(b0, r), f1 = nvfp4_group_factor(b1, r);
        uint8_t* row = kv_code_row(block, sh, tok);
        uint8_t* srow = kv_scale_row(block, sh, tok);
        *reinterpret_cast<uint32_t*>(row + c0 / 2) = nvfp4_codes8(lo, f0);
        *reinterpret_cast<uint32_t*>(row + c1 / 2) = nvfp4_codes8(hi, f1);
        if (!pair || (c0 & 8) == 0) srow[c0 / 16] = (uint8_t)b0;
        if (pair && (c0 & 8) != 0) srow[c1 / 16] = (uint8_t)b1;
    }
}

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 128;   // R <= 256
constexpr int kRopeMaxTokens = 8;    // of a workgroup
// A unit's eight (cos, sin) pairs take 64 bytes of LDS; units start 80 bytes
// apart, which spreads the eight units of a 128-column row over all banks.
constexpr int kRopeUnitWords = 20;

// Workgroup: TB <= kRopeMaxTokens tokens (blockIdx.x) and every gridDim.y-th run of 256 units
// of them.  First the tokens' (cos, sin) pairs go to LDS, one per thread and
// round; then each thread takes 16 values at a time: 8 rotated pairs (halves:
// columns 8 u .. and R / 2 + 8 u ..; neighbours: 16 u ..) or 16 columns that
// pass.  All of a unit's loads come before its stores and no two units share
// a column, so q_out may be q.
// Bound by HBM (the reads and writes of q, k and v): 4096 tokens of 32 + 8
// heads of 128 into an E4M3 cache (92 MB) take 20.7 us, 4.5 TB/s (a large copy
// reaches 4.8), into an NVFP4 cache (89 MB) 20.2; q alone, 5003 tokens of 16
// heads of 80 (26 MB), 7.6 us; 1003 tokens of 24 + 24 heads of 64 (18.5 MB) 7.5,
// where each token is a workgroup and its 288 units a second round of 32; 16
// tokens 3.3 .. 4.4 us, of which the fp64 angles and the loads after the
// barrier are most.  16 values a thread keeps every 16-bit access 16 bytes
// wide and a whole NVFP4 group within two lanes.
template <int FMT, bool F16, bool NEIGHBOURS>
__global__ void __launch_bounds__(kRopeThreads) k_rope_append(AppendArgs a, int TB) {
    __shared__ __attribute__((aligned(16))) float s_cs[kRopeMaxTokens * (kRopeMaxPairs / 8) * kRopeUnitWords];
    const int64_t t0 = (int64_t)blockIdx.x * TB;
    const int nt = a.T - t0 < TB ? (int)(a.T - t0) : TB;
    const int half = a.rope.R >> 1, ru = a.rope.R >> 4, U = a.D >> 4;
    for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
        const int tt = i / half, p = i - tt * half;
        int ax = a.rope.pair_axis ? a.rope.pair_axis[p] : 0;
        ax = ax < 0 ? 0 : (ax >= a.rope.axes ? a.rope.axes - 1 : ax);   // kept in bounds
        const float2 cs = rope_cos_sin(a.rope.positions[(int64_t)ax * a.rope.ld_pos + t0 + tt], a.rope.inv_freq[p]);
        float* to = s_cs + (tt * ru + (p >> 3)) * kRopeUnitWords + (p & 7) * 2;
        to[0] = cs.x;
        to[1] = cs.y;
    }
    __syncthreads();
    const int per_token = (a.Hq + 2 * a.Hk) * U;
    const int total = nt * per_token;
    // every lane of a wave takes part in each round (kv_store16 exchanges values between lanes)
    for (int i0 = blockIdx.y * kRopeThreads; i0 < total; i0 += gridDim.y * kRopeThreads) {
        const int i = i0 + threadIdx.x;
        const bool valid = i < total;
        const int ii = valid ? i : 0;
        const int tt = ii / per_token, j = ii - tt * per_token;
        const int head = j / U, u = j - head * U;
        const int64_t t = t0 + tt;
        const bool is_q = head < a.Hq, is_k = !is_q && head < a.Hq + a.Hk;
        const int hk = is_k ? head - a.Hq : head - a.Hq - a.Hk;
        const uint16_t* src = is_q ? a.q + t * a.q_t + head * a.q_h
                                   : is_k ? a.k + t * a.k_t + hk * a.k_h : a.v + t * a.v_t + hk * a.v_h;
        const bool turn = u < ru && (is_q || is_k);
        const bool pair = turn && !NEIGHBOURS;
        const int c0 = pair ? 8 * u : 16 * u, c1 = pair ? half + 8 * u : 16 * u + 8;
        float lo[8], hi[8];
        unpack8<F16>(*reinterpret_cast<const uint4*>(src + c0), lo);
        unpack8<F16>(*reinterpret_cast<const uint4*>(src + c1), hi);
        if (turn) {
            const float4* cs = reinterpret_cast<const float4*>(s_cs + (tt * ru + u) * kRopeUnitWords);
            float4 w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = cs[e];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 c = make_float2(w[e].x, w[e].y), d = make_float2(w[e].z, w[e].w);
                if constexpr (NEIGHBOURS) {
                    float(&g)[8] = e < 2 ? lo : hi;
                    rope_turn(g[(e & 1) * 4], g[(e & 1) * 4 + 1], c);
                    rope_turn(g[(e & 1) * 4 + 2], g[(e & 1) * 4 + 3], d);
                } else {
                    rope_turn(lo[2 * e], hi[2 * e], c);
                    rope_turn(lo[2 * e + 1], hi[2 * e + 1], d);
                }
            }
        }
        if (is_q) {
            if (valid) {
                uint16_t* dst = a.q_out + t * a.qo_t + head * a.qo_h;
                *reinterpret_cast<uint4*>(dst + c0) = pack8<F16>(lo);
                *reinterpret_cast<uint4*>(dst + c1) = pack8<F16>(hi);
            }
        }
        if (a.Hk > 0) {
            if constexpr (FMT != kKv16) {
                if (turn && !is_q) {   // the rotated keys are rounded to 16 bits before they are quantised
                    unpack8<F16>(pack8<F16>(lo), lo);
                    unpack8<F16>(pack8<F16>(hi), hi);
                }
            }
            int64_t page = 0;
            int tok = 0;
            bool there = valid && !is_q;
            if (there) there = kv_locate(a.shape, a.slots[t], page, tok);
            const int hc = is_q ? 0 : hk;
            if (is_k) kv_store16<FMT, F16>(a.kc, a.shape, there, page, tok, hc, c0, c1, pair, lo, hi);
            else if (!is_q) kv_store16<FMT, F16>(a.vc, a.shape, there, page, tok, hc, c0, c1, pair, lo, hi);
        }
    }
}

// --------------------------------------------------------------- read back --

struct ReadArgs {
    KvSide kc, vc;
    KvShape shape;
    const int32_t* slots;
    uint16_t *k, *v;
    int64_t k_t, k_h, v_t, v_h;   // strides in elements: token, head
    int64_t T;
};

// 16 columns of one cache row as fp32, without the head's scale.
template <int FMT, bool F16>
__device__ __forceinline__ void kv_load16(const KvSide& side, const KvShape& sh, int64_t page, int tok, int head,
                                          int c0, float (&lo)[8], float (&hi)[8]) {
    const uint8_t* block = side.base + page * side.s_page + head * side.s_head;
    if constexpr (FMT == kKv16) {
        const uint4* row = reinterpret_cast<const uint4*>(block + tok * side.s_token + c0 * 2);
        unpack8<F16>(row[0], lo);
        unpack8<F16>(row[1], hi);
    } else if constexpr (FMT == kKvE4m3) {
        const uint4 b = *reinterpret_cast<const uint4*>(block + tok * side.s_token + c0);
        const uint32_t d[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(d[i], 1.0f, false);
            const f32x2 q = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(d[i], 1.0f, true);
            float(&f)[8] = i < 2 ? lo : hi;
            f[(i & 1) * 4] = p.x;
            f[(i & 1) * 4 + 1] = p.y;
            f[(i & 1) * 4 + 2] = q.x;
            f[(i & 1) * 4 + 3] = q.y;
        }
    } else {
        const uint2 b = *reinterpret_cast<const uint2*>(kv_code_row(block, sh, tok) + c0 / 2);
        const float s = e4m3_to_f32(kv_scale_row(block, sh, tok)[c0 / 16]);
#define NVFP4_KV_PAIR(WORD, BYTE, F, I)                                                 \
    {                                                                                   \
        const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(WORD, 1.0f, BYTE);     \
        F[I] = p.x * s;                                                                 \
        F[I + 1] = p.y * s;                                                             \
    }
        NVFP4_KV_PAIR(b.x, 0, lo, 0) NVFP4_KV_PAIR(b.x, 1, lo, 2) NVFP4_KV_PAIR(b.x, 2, lo, 4) NVFP4_KV_PAIR(b.x, 3, lo, 6)
        NVFP4_KV_PAIR(b.y, 0, hi, 0) NVFP4_KV_PAIR(b.y, 1, hi, 2) NVFP4_KV_PAIR(b.y, 2, hi, 4) NVFP4_KV_PAIR(b.y, 3, hi, 6)
#undef NVFP4_KV_PAIR
    }
}

// Thread: 16 columns of one row; RNE16(value * head scale), zeros for a slot
// outside the cache.  Bound by the bytes it moves: 4096 tokens of 8 heads of
// 128 from E4M3 (25 MB, most of it just written) take 7.3 us, from NVFP4 7.7, 16
// tokens 2.9: with so few bytes a thread the divisions of its index count too.
template <int FMT, bool F16>
__global__ void __launch_bounds__(256) k_kv_read(ReadArgs a) {
    const int U = a.shape.D >> 4, per_token = 2 * a.shape.heads * U;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.T * per_token) return;
    const int64_t t = i / per_token;
    const int j = (int)(i - t * per_token), hh = j / U, c0 = (j - hh * U) * 16;
    const bool is_v = hh >= a.shape.heads;
    const int head = is_v ? hh - a.shape.heads : hh;
    const KvSide& side = is_v ? a.vc : a.kc;
    float lo[8] = {}, hi[8] = {};
    int64_t page;
    int tok;
    if (kv_locate(a.shape, a.slots[t], page, tok)) {
        kv_load16<FMT, F16>(side, a.shape, page, tok, head, c0, lo, hi);
        if (FMT != kKv16 && side.scale) {
            const float g = side.scale[head];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                lo[e] *= g;
                hi[e] *= g;
            }
        }
    }
    uint16_t* dst = is_v ? a.v + t * a.v_t + head * a.v_h : a.k + t * a.k_t + head * a.k_h;
    *reinterpret_cast<uint4*>(dst + c0) = pack8<F16>(lo);
    *reinterpret_cast<uint4*>(dst + c0 + 8) = pack8<F16>(hi);
}

}  // namespace nvfp4
