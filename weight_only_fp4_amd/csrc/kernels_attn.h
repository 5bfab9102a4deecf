// Attention of one new token per sequence over the paged key-value cache,
// split over the cache's length and joined.
#pragma once
#include <type_traits>

#include "decode.h"
#include "kernels_gemm.h"
#include "kernels_kv.h"

namespace nvfp4 {

struct AttnArgs {
    // what a workgroup's beginning needs: one cache line
    KvShape shape;
    const int32_t* lengths;      // [B]
    int B;
    int head_tiles;              // ceil(G / 16)
    int width;                   // table entries used of a sequence
    int window;                  // 0: all tokens
    int split;                   // 0: one workgroup per pair
    int grid;                    // workgroups of a split call
    // a segment's
    uint32_t page_magic;         // token / page_size = umulhi(token, magic) >> shift (page_size > 1)
    int page_shift;
    const uint16_t* q;           // [B][Hq][D]
    int64_t q_b, q_h;            // strides in elements
    const int32_t* table;        // [B][ld_table], `width` entries used
    int64_t ld_table;
    KvSide kc, vc;
    int G;                       // query heads per key-value head
    float scale_log2;            // softmax scale * log2(e)
    int f16;                     // q and out are fp16 (else bf16)
    // its end's
    int Hq;
    uint16_t* out;
    int64_t o_b, o_h;
    float* lse;                  // [B][Hq] or NULL
    float* partials;             // [workgroups][2][part_floats]: sums, then (maximum, sum of weights) pairs
    int* counters;               // [workgroups], zero between calls
};

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = kAttnWaves * 64;
constexpr int kAttnTile = 32;                               // tokens a wave takes at a time
constexpr int kAttnUnit = kAttnWaves * kAttnTile;           // tokens a workgroup takes at a time
constexpr int kAttnHeads = 16;                              // query heads of one workgroup
constexpr int kAttnScan = 2048;                             // sequences whose unit counts are kept in LDS
constexpr int kAttnMaxWorkgroups = 512;                     // of a split call
constexpr int kAttnPairSplits = 64;                         // at most this many workgroups per pair on average: the
                                                            // last of them joins what they leave
constexpr unsigned kAttnWhole = 6;                          // pairs of fewer places are not split
constexpr int kAttnJoin = 16;                               // partial results a join fetches at a time
constexpr int kAttnOutCols = 128;                           // columns of the accumulators that go through LDS at a time (at most):
                                                            // 64 at a time take 0.2 us more a segment (D = 128)

// Read-only memory at a uniform address (scalar loads), and rows of the cache.
typedef const __attribute__((address_space(4))) int32_t* AttnTable;
typedef const __attribute__((address_space(4))) float* AttnScales;
typedef const __attribute__((address_space(1))) uint8_t* AttnRow;

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

// Maximum over the four lanes of a query head (lanes 16 apart).
__device__ __forceinline__ float attn_head_max(float v) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Maximum / sum over the wave in registers: lanes 32 and 16 apart change places,
// then the rows of 16 lanes rotate by 8, 4, 2 and 1.
template <typename Op>
__device__ __forceinline__ float attn_wave_reduce(float v, Op op) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
    v = op(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x128, 0xF, 0xF, true)));
    v = op(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x124, 0xF, 0xF, true)));
    v = op(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x122, 0xF, 0xF, true)));
    return op(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x121, 0xF, 0xF, true)));
}

// Sums over the lanes up to each: within rows of 16 by 1, 2, 4 and 8 lanes,
// then rows 0 and 2 onto the next, then the first two rows onto the others.
__device__ __forceinline__ int attn_wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast:15
    return v + __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast:31
}

// Lane i of four gets the j-th's x[i] as x[j]: the square of four lanes and
// four registers, transposed.
__device__ __forceinline__ void attn_quad_transpose(uint32_t& x0, uint32_t& x1, uint32_t& x2, uint32_t& x3, int lane) {
    const bool b0 = lane & 1, b1 = lane & 2;
    auto next = [](uint32_t v) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true); };    // lane ^ 1
    auto other = [](uint32_t v) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true); };   // lane ^ 2
    // every lane takes part in the exchanges: they stand before the selections
    const uint32_t n0 = next(x0), n1 = next(x1), n2 = next(x2), n3 = next(x3);
    const uint32_t y0 = b0 ? n1 : x0, y1 = b0 ? x1 : n0, y2 = b0 ? n3 : x2, y3 = b0 ? x3 : n2;
    const uint32_t o0 = other(y0), o1 = other(y1), o2 = other(y2), o3 = other(y3);
    x0 = b1 ? o2 : y0;
    x2 = b1 ? y2 : o0;
    x1 = b1 ? o3 : y1;
    x3 = b1 ? y3 : o1;
}
template <int J>
__device__ __forceinline__ uint32_t attn_quad_lane(uint32_t v) {   // lane J's of each four
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, J * 0x55, 0xF, 0xF, true);
}

// Streaming loads: the cache's rows are read once.
template <int BYTES>
__device__ __forceinline__ void attn_load(AttnRow p, uint32_t* d) {
    typedef unsigned u32x2v __attribute__((ext_vector_type(2)));
    if constexpr (BYTES == 1) d[0] = __builtin_nontemporal_load(p);
    else if constexpr (BYTES == 2) d[0] = __builtin_nontemporal_load((const __attribute__((address_space(1))) uint16_t*)p);
    else if constexpr (BYTES == 4) d[0] = __builtin_nontemporal_load((const __attribute__((address_space(1))) uint32_t*)p);
    else if constexpr (BYTES == 8) {
        const u32x2v t = __builtin_nontemporal_load((const __attribute__((address_space(1))) u32x2v*)p);
        d[0] = t[0];
        d[1] = t[1];
    } else {
#pragma unroll
        for (int x = 0; x < BYTES / 16; ++x) {
            const u32x4v t = __builtin_nontemporal_load((const __attribute__((address_space(1))) u32x4v*)p + x);
            d[4 * x] = t[0];
            d[4 * x + 1] = t[1];
            d[4 * x + 2] = t[2];
            d[4 * x + 3] = t[3];
        }
    }
}

// A row of the cache as a buffer: the scalar base, 32-bit offsets of the lanes,
// and reads of nothing (zeros come back) where `there` is false.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t attn_buffer(uint64_t base, bool there) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, there ? 1 << 30 : 0, 0x00027000);
}
template <int BYTES>
__device__ __forceinline__ void attn_buffer_load(__amdgpu_buffer_rsrc_t r, uint32_t lane_at, uint32_t at, uint32_t* d) {
    constexpr int NT = 2;   // streaming
    typedef unsigned u32x2v __attribute__((ext_vector_type(2)));
    if constexpr (BYTES == 1) d[0] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, (int)lane_at, (int)at, NT);
    else if constexpr (BYTES == 2) d[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)lane_at, (int)at, NT);
    else if constexpr (BYTES == 4) d[0] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)lane_at, (int)at, NT);
    else if constexpr (BYTES == 8) {
        const u32x2v t = __builtin_amdgcn_raw_buffer_load_b64(r, (int)lane_at, (int)at, NT);
        d[0] = t[0];
        d[1] = t[1];
    } else {
#pragma unroll
        for (int x = 0; x < BYTES / 16; ++x) {
            const u32x4v t = __builtin_amdgcn_raw_buffer_load_b128(r, (int)lane_at + x * 16, (int)at, NT);
            d[4 * x] = t[0];
            d[4 * x + 1] = t[1];
            d[4 * x + 2] = t[2];
            d[4 * x + 3] = t[3];
        }
    }
}

// The work.  A sequence's tokens are cut into units of 128 (kAttnUnit); its
// key-value heads (times tiles of 16 query heads) all have that many.  The
// units of all (sequence, head) pairs stand in one row, sequence by sequence,
// each pair with one more place in front for what a pair costs besides its
// tokens (two with an NVFP4 cache, whose units take less time, and more pairs
// than half the grid, where a workgroup that takes short sequences holds several
// pairs: 64 sequences of up to 8191 tokens, 512 pairs, 42.5 us with one, 40 with
// two or four), and workgroup j of N takes the places
// from floor(j P / N) to floor((j + 1) P / N) of all P, so every compute unit
// gets the same work whatever the lengths are.  N is at most the grid, and a
// multiple of the pairs (equal lengths are then split at equal places): with p
// places a pair on average
//   p < 6      one workgroup a pair: a join costs more than four units do
//              (2 x 300 tokens: 8.3 us, halved 9.4);
//   p <= 17    p workgroups while no compute unit gets a second one, so each
//              works on one unit and the join takes one round trip (1 x 1024
//              tokens: 8.4 us, p / 2 workgroups 10.4, p / 4 12.5);
//   else       p / 2 (1 x 8192 tokens: 14.8 us, p / 4 16.3, p 17.2: the join
//              of more than 16 partial results takes several).
// A stretch is a few segments, each a run of units of one pair; a segment that
// is not the whole pair leaves a partial result, and the workgroup that arrives
// last at a pair adds the partial results in their order (so the result does
// not depend on timing).
//
// A workgroup's waves take the segment's tiles of 32 tokens in turn, each with
// its own running maximum, sum and accumulators: the loop has no barrier.  A
// tile's rows are loaded while the one before is worked on.
//
// A wave's tile:
//   S^T = K Q^T       mfma 16x16x32, rows = tokens, columns = heads: lane (g, c)
//                     (g = lane / 16, c = lane % 16) loads 16-byte pieces of
//                     token c's key row straight into the A operand, and gets
//                     the scores of head c for tokens 4 g .. 4 g + 3;
//   softmax           all of a lane's values belong to head c; the four lanes
//                     of a head exchange maxima only;
//   O^T += V^T P^T    rows = columns of V, columns = heads: the contraction
//                     slots are numbered so that lane (g, c) holds in slots
//                     0..3 / 4..7 the tokens 4 g .. of the tile's two halves,
//                     which are the tokens whose weights it just computed, so
//                     P goes from the scores to the B operand inside the lane.
//                     V's rows are loaded as stored (lane c: columns c VD ..
//                     c VD + VD - 1, VD = DT / 16) and transposed in
//                     registers, one byte permute per two values; MFMA e takes
//                     the columns c VD + e.
//
// Two forms of the addresses:
//   FAST   D is DT and pages are multiples of 16 tokens: a half-tile of 16
//          tokens lies in one page, so its base is a scalar and the lanes'
//          offsets never change (tiles begin at multiples of 32 tokens; a
//          window's first tile masks the tokens before it).  It is read as a
//          buffer whose size is 0 for a half-tile past the segment's end or
//          of a page outside the cache: such loads touch no memory (with page
//          0's rows read in their place, which every wave of the chip did at
//          its end, 128 x 0..2000 tokens took 63 us instead of 59);
//   else   any D and page size: the tile's 32 row offsets pass through LDS
//          (each wave its own, no barrier).
//
// Quantised caches are decoded to fp16, which holds E4M3 and E2M1 x E4M3
// exactly; q is scaled by a power of two per head, its largest column to [2^14,
// 2^15), so that it fits: only columns below 2^-28 of that one (2^-31 with a
// bf16 q) lose bits.
//
// The weights go into the second product as fp16 (bf16 with a bf16 cache);
// the sum of the weights is taken in fp32 before that.  The running maximum m
// is kept 7 below the largest score (in powers of two) where the product is of
// fp16, so the weights are at most 2^7, or 2^8 where a score's last place is
// above 1 and 7 is rounded, and those down to 2^-32 of the largest are not
// rounded to 0: what vanishes adds up to less than a rounding of fp16 for up to
// 2^21 tokens of a wave (2^14 with 1 as the largest weight, where a tile's 31
// tokens of 2^-26 beside one of zero values gave 0).  8 could be rounded to 16,
// at a last place of 16, and overflow.  With a 16-bit
// or E4M3 cache they go as two values, the rounded weight and what the
// rounding took off, with a product each: 16 bits of a weight with bf16, 22
// with fp16 (rounded once they added a sixth to the error of a 16-bit result).
// These kernels wait for memory, so the second product costs them nothing (32
// x 8192 tokens bf16: 174.9 us with and without, in a graph; 131072 E4M3 54.1
// and 54.0; 1000 short sequences, E4M3, 89 and 87.4).  With an NVFP4 cache it
// would (32 x 8192: 61 -> 64 us, 64 ragged ones 38.5 -> 40.8), for bits that a
// value of four has no use for: there a weight is one fp16, off by 2^-11 of
// itself.  The heads' key scale goes into the softmax scale, the value scale
// into the final normalisation.
//
// Tokens past the length or before the window, and tokens of pages whose table
// entry is outside the cache, get the weight 0 and their value rows are
// replaced by zeros, so nothing in them (an infinity, a NaN) reaches the
// result.
//
// What bounds it, with 8 key-value heads of 128: of 16-bit and E4M3 caches the
// HBM reads, 32 x 8192 tokens (bf16, 1.07 GB) in 169 us and one sequence of
// 131072 (E4M3, 268 MB) in 51 (kernel trace), 6.4 and 5.2 TB/s with a plain read
// at 7.1: about 9 us of a call are its beginning (the lengths, the table, the
// first rows, one after another) and its end (the join).  NVFP4 caches take 32 x
// 8192 tokens (302 MB) in 54 us and 64 sequences of up to 8191 (147 MB) in 37.7.
// In a graph with other calls those take 60 and 39, one of 131072 35.7, and with
// the work on the tiles left out 54, 33 and 33.9: most of the distance to the
// read rate is in the loads themselves (few bytes under way: a tile is 4.6 KB,
// in 16 bits 16) and in the beginnings and ends of the segments, of which the
// ragged ones have more; the decoding adds 5 to 18 %.  130 tokens take 6.7 us,
// all latency.
//
// With heads of 64 the registers stay within 168, so that three workgroups fit a
// compute unit: calls of more than 2048 sequences, which are not split, have that
// many (3000 of up to 500 tokens, 8 heads, bf16: 207 us, with two of them 245).
template <int FMT, int DT, bool FAST>
__global__ void __launch_bounds__(kAttnThreads, DT == 64 ? 3 : 0) k_paged_attn(AttnArgs a) {
    constexpr bool F16 = FMT != 0;                   // type of the products: 0 is a bf16 cache
    constexpr int KV = FMT <= 1 ? kKv16 : FMT == 2 ? kKvE4m3 : kKvNvfp4;
    constexpr int KSTEPS = DT / 32;                  // 32-column steps of the first product
    constexpr int VD = DT / 16;                      // value columns of a lane
    constexpr bool FINE = KV != kKvNvfp4;            // weights in two parts
    constexpr float ABOVE = F16 ? 7.0f : 0.0f;       // log2 of the largest weight
    const int D = FAST ? DT : a.shape.D;
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ps = a.shape.page_size;
    const int HT = a.shape.heads * a.head_tiles;

    __shared__ int s_pre[kAttnScan + 1];   // places of the sequences before b, per head
    __shared__ uint32_t s_off[FAST ? 1 : kAttnWaves][3][kAttnTile];
    __shared__ float s_m[kAttnWaves][kAttnHeads], s_l[kAttnWaves][kAttnHeads];
    __shared__ int s_flag;
    // the waves' accumulators on their way out: [waves][nh][OS], a pass at a time
    extern __shared__ float s_o[];
    constexpr int LD = DT < kAttnOutCols ? DT : kAttnOutCols, OS = LD + 4;   // 16-byte aligned rows, spread over the banks
    constexpr int PASSES = DT / LD, RP = 4 / PASSES;                         // accumulator rows of a lane per pass

    // the arguments, to be read from memory again
    typedef const __attribute__((address_space(4))) AttnArgs KernArgs;
    auto kernel_args = [] {
        KernArgs* z = (KernArgs*)__builtin_amdgcn_kernarg_segment_ptr();
        asm volatile("" : "+s"(z));
        return z;
    };

    // tokens [first, len) of sequence b; units are counted from the tile `first` lies in
    AttnTable lengths = (AttnTable)(uint64_t)a.lengths;
    const int most = a.width * ps;   // below 2^30
    auto clamp_range = [&](int n, int& first, int& len) {
        len = n < 0 ? 0 : (n > most ? most : n);
        first = a.window > 0 && len > a.window ? len - a.window : 0;
    };
    auto count_units = [&](int first, int len) {
        const int n = (len - (first & ~(kAttnTile - 1)) + kAttnUnit - 1) / kAttnUnit;
        return n < 1 ? 1 : n;   // an empty sequence's output is written too
    };

    // ---- this workgroup's stretch of places [p_begin, p_end)
    const int front = KV == kKvNvfp4 && a.B * HT > kAttnMaxWorkgroups / 2 ? 2 : 1;   // places in front of a pair's units
    int p_begin, p_end, groups = 1, b = 0, ph0 = 0;
    unsigned places = 1;
    // floor(x / y) of a 41-bit and a 31-bit number, exact in fp64: the quotient is
    // further from the next integer than it is rounded by
    auto quotient = [](int64_t x, unsigned y) { return (int)((double)x / (double)y); };
    int me = (int)blockIdx.x;   // which of the stretches
    if (!a.split) {
        b = (int)(blockIdx.x / (unsigned)HT);
        ph0 = (int)blockIdx.x - b * HT;
        p_begin = 0;
        p_end = 1;
    } else {
        if (a.B == 1) {
            int f, n;
            clamp_range(lengths[0], f, n);
            if (threadIdx.x == 0) {
                s_pre[0] = 0;
                s_pre[1] = front + count_units(f, n);
            }
        } else if (w == 0) {
            int before = 0, ahead = lane < a.B ? a.lengths[lane] : 0;
            for (int b0 = 0; b0 < a.B; b0 += 64) {
                int v = 0;
                if (b0 + lane < a.B) {
                    int f, n;
                    clamp_range(ahead, f, n);
                    v = front + count_units(f, n);
                }
                ahead = b0 + 64 + lane < a.B ? a.lengths[b0 + 64 + lane] : 0;
                v = attn_wave_scan(v);
                if (b0 + lane < a.B) s_pre[b0 + lane + 1] = before + v;
                before += __builtin_amdgcn_readlane(v, 63);
            }
            if (lane == 0) s_pre[0] = 0;
        }
        __syncthreads();
        places = (unsigned)__builtin_amdgcn_readfirstlane(s_pre[a.B]) * (unsigned)HT;   // below 2^31
        const unsigned pairs = (unsigned)(a.B * HT), per = places / pairs;
        unsigned each = per < kAttnWhole ? 1u : per / 2;
        if (per >= kAttnWhole && per <= kAttnJoin + 1 && places <= 256) each = per;
        if (each > kAttnPairSplits) each = kAttnPairSplits;
        groups = (int)(pairs * each);
        groups = groups < a.grid ? groups : a.grid;
        if (me >= groups) return;
        // A full grid is two workgroups a compute unit, of which the second ones
        // start later and find the memory busy: neighbours in the row are one of
        // either (32 x 8192 tokens: 175 us, in the grid's order 181; 8 x 4096
        // NVFP4 16 us instead of 17.5).
        if (groups == kAttnMaxWorkgroups)
            me = me < kAttnMaxWorkgroups / 2 ? 2 * me : 2 * (me - kAttnMaxWorkgroups / 2) + 1;
        p_begin = quotient((int64_t)me * places, groups);
        p_end = quotient((int64_t)(me + 1) * places, groups);
        int lo = 0, hi = a.B;   // the sequence of the first place: the last b with HT * s_pre[b] <= p_begin
        const int at = p_begin / HT;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_pre[mid] <= at) lo = mid;
            else hi = mid;
        }
        b = __builtin_amdgcn_readfirstlane(lo);
    }

    // Of the waves of a SIMD the oldest issues first, so that a younger one's
    // work is largely left for the end, when it has the SIMD to itself and
    // cannot fill it.  Every wave therefore gives up a step of priority with
    // each quarter of its stretch: those behind go first.
    __builtin_amdgcn_s_setprio(3);
    const int quarter = (p_end - p_begin + 3) / 4;
    int prio_place = p_begin + quarter, prio = 3;
    for (int place = p_begin; place < p_end;) {
        // The arguments a segment needs are fetched when it begins: kept, they would
        // have to make way for the loop's scalars, 60 lane writes in front of the
        // first load (130 tokens: 7.5 us, so 7.0).
        const KernArgs* y = kernel_args();
        // ---- the segment: units [unit0, unit1) of pair (b, ph)
        int first, len, ph, units, unit0, unit1;
        int pair_begin = 0;   // the pair's first place
        if (!a.split) {
            ph = ph0;
            clamp_range(lengths[b], first, len);
            units = count_units(first, len);
            unit0 = 0;
            unit1 = units;
            place = p_end;
        } else {
            int next = __builtin_amdgcn_readfirstlane(s_pre[b + 1]);
            while (next * HT <= place) next = __builtin_amdgcn_readfirstlane(s_pre[++b + 1]);
            const int before = __builtin_amdgcn_readfirstlane(s_pre[b]);
            clamp_range(lengths[b], first, len);
            units = next - before - front;
            const int local = place - before * HT;
            ph = (int)((unsigned)local / (unsigned)(units + front));
            pair_begin = before * HT + ph * (units + front);
            const int o0 = place - pair_begin;
            const int o1 = p_end - pair_begin < units + front ? p_end - pair_begin : units + front;
            place = pair_begin + o1;
            unit0 = o0 > front ? o0 - front : 0;
            unit1 = o1 - front;
            if (unit1 <= unit0) continue;   // only places in front: the next workgroup begins the pair
        }
        const int hk = y->head_tiles == 1 ? ph : (int)((unsigned)ph / (unsigned)y->head_tiles), ht = ph - hk * y->head_tiles;
        const int nh = y->G - ht * kAttnHeads < kAttnHeads ? y->G - ht * kAttnHeads : kAttnHeads;
        const int head0 = hk * y->G + ht * kAttnHeads;
        const int base_t = first & ~(kAttnTile - 1);
        const int t_stop = len - base_t < unit1 * kAttnUnit ? len : base_t + unit1 * kAttnUnit;

        // The wave's table entries come first: its rows wait for them.  FAST: of the
        // half-tiles of 32 tiles, else of a tile's tokens.
        int t0 = base_t + unit0 * kAttnUnit + w * kAttnTile;
        auto page_index = [&](int t) { return !FAST && ps == 1 ? t : (int)(__umulhi((uint32_t)t, y->page_magic) >> y->page_shift); };
        int ahead = -1;   // the lane's table entry
        auto lane_token = [&](int t) { return FAST ? t + (lane >> 1) * kAttnUnit + (lane & 1) * 16 : t + lane; };
        auto fetch_entries = [&](int t) {
            const int mine = lane_token(t);
            ahead = -1;
            const KernArgs* y = kernel_args();
            if (mine < t_stop && (FAST || lane < kAttnTile)) ahead = y->table[b * y->ld_table + page_index(mine)];
        };
        fetch_entries(t0);

        // q of head c as the B operand of each 32-column step: the columns of
        // step j are the ones the key pieces deliver
        uint4 qf[KSTEPS];
        float qk_log2 = y->scale_log2;
        auto key_column = [&](int j) {   // first of the 8 columns lane (g, c) holds in step j
            if constexpr (KV == kKv16) return j * 32 + g * 8;
            else if constexpr (KV == kKvE4m3) return (j >> 1) * 64 + g * 16 + (j & 1) * 8;
            else if constexpr (DT == 64) return g * 16 + j * 8;
            else return (j >> 2) * 128 + g * 32 + (j & 3) * 8;
        };
        {
            const uint16_t* qr = y->q + b * y->q_b + (int64_t)(head0 + c) * y->q_h;
#pragma unroll
            for (int j = 0; j < KSTEPS; ++j) qf[j] = make_uint4(0u, 0u, 0u, 0u);
            if (c < nh) {
#pragma unroll
                for (int j = 0; j < KSTEPS; ++j) {
                    const int col = key_column(j);
                    if (FAST || col < D) qf[j] = *reinterpret_cast<const uint4*>(qr + col);
                }
            }
        }

        const uint64_t kb = (uint64_t)y->kc.base + hk * y->kc.s_head, vb = (uint64_t)y->vc.base + hk * y->vc.s_head;
        auto in_cache = [&](int p) { return (uint32_t)p < (uint32_t)a.shape.pages; };

        constexpr int KP = KV == kKv16 ? KSTEPS : KV == kKvE4m3 ? KSTEPS / 2 : (DT == 256 ? 2 : 1);   // pieces of a key row
        constexpr int KB = KV == kKvNvfp4 && DT == 64 ? 8 : 16;                  // bytes of a piece, 64 bytes apart
        constexpr int VB = KV == kKv16 ? VD * 2 : KV == kKvE4m3 ? VD : VD / 2;   // bytes of a lane's value columns
        constexpr int VW = VB < 4 ? 1 : VB / 4;                                  // dwords
        struct Tile {
            uint32_t kraw[2][KP][4], ksc[2][KP], vraw[8][VW], vsc[8];
            uint32_t valid;
        };
        // NVFP4: from a block's start to its scales (below 2^31 where it is FAST)
        const std::conditional_t<FAST, uint32_t, int64_t> scales_at = (std::conditional_t<FAST, uint32_t, int64_t>)ps * (D / 2);
        // FAST: the lane's offsets inside a half-tile
        const uint32_t k_tok = KV == kKvNvfp4 ? (uint32_t)(D / 2) : (uint32_t)y->kc.s_token;
        const uint32_t v_tok = KV == kKvNvfp4 ? (uint32_t)(D / 2) : (uint32_t)y->vc.s_token;
        // WIDE: of an NVFP4 value row a lane loads the quarter c / 4 of token 4 g +
        // c % 4, and four lanes then exchange pieces so that each has its columns
        // of the four tokens: 8 loads a tile instead of 20 with the lane's own
        // columns, which cost more than the exchange (32 x 8192 tokens: 65 -> 60
        // us).  A row of 64 columns has only two bytes a lane to exchange.
        constexpr bool WIDE = FAST && KV == kKvNvfp4 && DT >= 128;
        const uint32_t k_lane = c * k_tok + g * KB;
        const uint32_t v_lane = WIDE ? (g * 4 + (c & 3)) * v_tok + (c >> 2) * VB * 4 : g * 4 * v_tok + c * VB;
        const uint32_t ks_lane = c * (D / 16) + (DT == 64 ? g : g * 2);
        const uint32_t vs_lane = WIDE ? (g * 4 + (c & 3)) * (D / 16) + (c >> 2) * (VD / 4) : g * 4 * (D / 16) + c * VD / 16;
        // WIDE: picks the lane's group scale of a token pair from both tokens' quarters
        const uint32_t vs_at = DT == 256 ? c & 3 : (c >> 1) & 1, vs_pair = 0x0C0C0400u + vs_at * 0x0101u;

        auto token_mask = [&](int t) {   // tokens of the tile at t inside [first, t_stop), one bit each
            const int lo = first > t ? first - t : 0, hi = t_stop - t;
            uint32_t valid = hi >= kAttnTile ? 0xFFFFFFFFu : (hi <= 0 ? 0u : (1u << hi) - 1u);
            if (lo > 0) valid = lo >= kAttnTile ? 0u : valid & (0xFFFFFFFFu << lo);
            return valid;
        };
        // FAST: where the rows of the wave's next 32 tiles are: lane 2 i + h holds
        // the offsets of half-tile h of the i-th (in 16 bytes; `deep`: from its
        // codes to its group scales, NVFP4), so a tile takes a few lane reads
        // instead of two table lookups and their 64-bit products.
        uint32_t at_k = 0, at_v = 0, deep = 0;
        uint64_t odd = 0, out_of_cache = 0;   // half-tiles that are not whole; whose entry is outside the cache
        int turn = 0;                         // lane of the next tile
        auto place_rows = [&](int t) {   // of the 32 tiles from the one at t
            const KernArgs* y = kernel_args();
            const int mine = lane_token(t);
            const bool ok = in_cache(ahead);
            // offsets in 16 bytes fit 32 bits, and so do the strides where there is more than one page
            const uint32_t page = ok ? (uint32_t)ahead : 0u, tok = ok ? (uint32_t)(mine - page_index(mine) * ps) : 0u;
            at_k = page * (uint32_t)(y->kc.s_page >> 4) + tok * (k_tok >> 4);
            at_v = page * (uint32_t)(y->vc.s_page >> 4) + tok * (v_tok >> 4);
            if constexpr (KV == kKvNvfp4) deep = scales_at - tok * (uint32_t)(D / 2 - D / 16);
            out_of_cache = __ballot(!ok);
            odd = __ballot(!ok || mine < first || mine + 16 > t_stop);
            turn = 0;
            // past the segment's end there are none: such tiles are outside the cache
            if (t + 32 * kAttnUnit < t_stop) fetch_entries(t + 32 * kAttnUnit);
            else ahead = -1;
        };
        auto load_tile = [&](Tile& x, int t) {
            if constexpr (FAST) {
                uint32_t valid = 0xFFFFFFFFu;   // tokens of the tile inside [first, t_stop) and the cache, one bit each
                if ((odd >> turn) & 3u) {
                    valid = token_mask(t);
                    if ((out_of_cache >> turn) & 1u) valid &= 0xFFFF0000u;
                    if ((out_of_cache >> turn) & 2u) valid &= 0x0000FFFFu;
                }
                x.valid = valid;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool there = !((out_of_cache >> (turn + h)) & 1u);
                    const auto kr = attn_buffer(kb + ((uint64_t)(uint32_t)__builtin_amdgcn_readlane(at_k, turn + h) << 4), there);
                    const auto vr = attn_buffer(vb + ((uint64_t)(uint32_t)__builtin_amdgcn_readlane(at_v, turn + h) << 4), there);
#pragma unroll
                    for (int p = 0; p < KP; ++p) attn_buffer_load<KB>(kr, k_lane + p * 64, 0u, x.kraw[h][p]);
                    const uint32_t far = KV == kKvNvfp4 ? __builtin_amdgcn_readlane(deep, turn + h) : 0u;
                    if constexpr (KV == kKvNvfp4) {
#pragma unroll
                        for (int p = 0; p < KP; ++p) attn_buffer_load<DT == 64 ? 1 : 2>(kr, ks_lane + p * 8, far, &x.ksc[h][p]);
                    }
                    if constexpr (WIDE) {
                        uint32_t row[4 * VW];
                        attn_buffer_load<VB * 4>(vr, v_lane, 0u, row);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int y = 0; y < VW; ++y) x.vraw[4 * h + i][y] = row[i * VW + y];
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) attn_buffer_load<VB>(vr, v_lane + i * v_tok, 0u, x.vraw[4 * h + i]);
                    }
                    if constexpr (KV == kKvNvfp4) {
                        if constexpr (WIDE) {
                            attn_buffer_load<VD / 4>(vr, vs_lane, far, &x.vsc[4 * h]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) attn_buffer_load<1>(vr, vs_lane + i * (D / 16), far, &x.vsc[4 * h + i]);
                        }
                    }
                }
                turn += 2;
            } else {
                // `ahead`: the table entry of the lane's token (the first 32 lanes)
                const int page = ahead, tok = t + lane - page_index(t + lane) * ps;
                const bool ok = in_cache(page);
                x.valid = token_mask(t) & (uint32_t)__ballot(ok);
                fetch_entries(t + kAttnUnit);
                if (lane < kAttnTile) {
                    // offsets in units of 16 bytes; a masked row is the head's first in its place
                    s_off[w][0][lane] = ok ? (uint32_t)((page * a.kc.s_page + (KV == kKvNvfp4 ? 0 : tok * a.kc.s_token)) >> 4) : 0u;
                    s_off[w][1][lane] = ok ? (uint32_t)((page * a.vc.s_page + (KV == kKvNvfp4 ? 0 : tok * a.vc.s_token)) >> 4) : 0u;
                    s_off[w][2][lane] = ok ? (uint32_t)tok : 0u;
                }
                // a wave's LDS accesses complete in order: only the compiler has to keep theirs
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint64_t row = kb + (uint64_t)s_off[w][0][h * 16 + c] * 16u;
                    const uint32_t tk = s_off[w][2][h * 16 + c];
                    const uint64_t srow = row + scales_at + (uint64_t)tk * (D / 16);
                    if constexpr (KV == kKvNvfp4) row += (uint64_t)tk * (D / 2);
#pragma unroll
                    for (int p = 0; p < KP; ++p) {
                        // first column of the piece: past D the row has none
                        const int col = KV == kKv16 ? p * 32 + g * 8 : KV == kKvE4m3 ? p * 64 + g * 16 : p * 128 + g * KB * 2;
                        x.ksc[h][p] = 0u;
#pragma unroll
                        for (int y = 0; y < 4; ++y) x.kraw[h][p][y] = 0u;
                        if (col < D) {
                            attn_load<KB>((AttnRow)(row + g * KB + p * 64), x.kraw[h][p]);
                            if constexpr (KV == kKvNvfp4) attn_load<DT == 64 ? 1 : 2>((AttnRow)(srow + col / 16), &x.ksc[h][p]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int slot = (i >> 2) * 16 + g * 4 + (i & 3);
                    uint64_t row = vb + (uint64_t)s_off[w][1][slot] * 16u;
                    const uint32_t tk = s_off[w][2][slot];
                    const uint64_t srow = row + scales_at + (uint64_t)tk * (D / 16);
                    if constexpr (KV == kKvNvfp4) row += (uint64_t)tk * (D / 2);
#pragma unroll
                    for (int y = 0; y < VW; ++y) x.vraw[i][y] = 0u;
                    x.vsc[i] = 0u;
                    if (c * VD < D) {
                        attn_load<VB>((AttnRow)(row + c * VB), x.vraw[i]);
                        if constexpr (KV == kKvNvfp4) attn_load<1>((AttnRow)(srow + c * VD / 16), &x.vsc[i]);
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
        };

        f32x4 acc[VD];
#pragma unroll
        for (int e = 0; e < VD; ++e) acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
        // columns without a head have q = 0 and, by this maximum, the weights 0 (with a
        // copy of the first head in them 64 ragged NVFP4 sequences took 41 us instead
        // of 39.7: it seems the power of the products, not their number)
        float m = c < nh ? -INFINITY : INFINITY, l = 0.f;

        auto work_tile = [&](Tile& x) {
            // ---- scores
            f32x4 sc[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                sc[h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int p = 0; p < KP; ++p) {
                    const uint32_t(&kw)[4] = x.kraw[h][p];
                    if constexpr (KV == kKv16) {
                        sc[h] = mma16<F16>(make_uint4(kw[0], kw[1], kw[2], kw[3]), qf[p], sc[h]);
                    } else if constexpr (KV == kKvE4m3) {
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            sc[h] = mma16<true>(make_uint4(f16_of_e4m3<false>(kw[2 * y]), f16_of_e4m3<true>(kw[2 * y]),
                                                           f16_of_e4m3<false>(kw[2 * y + 1]), f16_of_e4m3<true>(kw[2 * y + 1])),
                                                qf[2 * p + y], sc[h]);
                    } else {
                        constexpr int W = KB / 4;
#pragma unroll
                        for (int y = 0; y < W; ++y)
                            sc[h] = mma16<true>(f16_of_nvfp4(kw[y], f16_group_scale(x.ksc[h][p], y >= 2)), qf[p * W + y], sc[h]);
                    }
                }
            }
            // ---- weights of the lane's eight tokens (scaled first: a fused s qk - m
            // would not be 0 at the maximum of very large scores)
            float s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = sc[i >> 2][i & 3] * qk_log2;
            if (x.valid != 0xFFFFFFFFu) {
                // a branch: as selects the masks cost every tile 50 operations, and worked
                // out ahead their bits cost every workgroup's beginning
                int gm = g;
                asm volatile("" : "+v"(gm));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool ok = (x.valid >> ((i >> 2) * 16 + gm * 4 + (i & 3))) & 1u;
                    s[i] = ok ? s[i] : -INFINITY;
                    // the value row loaded into x.vraw[i]
                    const bool row_ok = WIDE ? (x.valid >> ((i >> 2) * 16 + gm * 4 + (c & 3))) & 1u : ok;
                    if constexpr (KV == kKvNvfp4) {
                        if (!WIDE || (i & 3) == 0) x.vsc[i] = row_ok ? x.vsc[i] : 0u;
                    }
#pragma unroll
                    for (int y = 0; y < VW; ++y) x.vraw[i][y] = row_ok ? x.vraw[i][y] : 0u;
                }
            }
            float top = s[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, s[i]);
            top = attn_head_max(top) - ABOVE;
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
                p[i] = __builtin_amdgcn_exp2f(s[i] - ms);
                l += p[i];
            }
            const uint4 pf = make_uint4(pack_round2<F16>(p[0], p[1]), pack_round2<F16>(p[2], p[3]),
                                        pack_round2<F16>(p[4], p[5]), pack_round2<F16>(p[6], p[7]));
            uint4 pl = pf;   // FINE: what that rounding took off them
            if constexpr (FINE) {
                const uint32_t d[4] = {pf.x, pf.y, pf.z, pf.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] -= act_to_f32<F16>((i & 1) ? d[i >> 1] >> 16 : d[i >> 1] & 0xFFFFu);
                pl = make_uint4(pack_round2<F16>(p[0], p[1]), pack_round2<F16>(p[2], p[3]),
                                pack_round2<F16>(p[4], p[5]), pack_round2<F16>(p[6], p[7]));
            }
            uint32_t vs[4];   // NVFP4: group scales of the token pairs
            if constexpr (KV == kKvNvfp4) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (WIDE) {
#pragma unroll
                        for (int y = 0; y < VW; ++y)
                            attn_quad_transpose(x.vraw[4 * h][y], x.vraw[4 * h + 1][y], x.vraw[4 * h + 2][y], x.vraw[4 * h + 3][y], lane);
                        const uint32_t q = x.vsc[4 * h];
                        vs[2 * h] = __builtin_amdgcn_perm(attn_quad_lane<1>(q), attn_quad_lane<0>(q), vs_pair);
                        vs[2 * h + 1] = __builtin_amdgcn_perm(attn_quad_lane<3>(q), attn_quad_lane<2>(q), vs_pair);
                    } else {
                        vs[2 * h] = x.vsc[4 * h] | (x.vsc[4 * h + 1] << 8);
                        vs[2 * h + 1] = x.vsc[4 * h + 2] | (x.vsc[4 * h + 3] << 8);
                    }
                }
            }
            // ---- values, transposed: a dword holds one column of a token pair
#pragma unroll
            for (int e0 = 0; e0 < VD; e0 += 8) {
                constexpr int EN = VD < 8 ? VD : 8;
                uint32_t vt[4][EN];   // [token pair][column e0 + ..]
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (KV == kKvNvfp4) {
                        // the pair's codes of a column side by side in a byte, then
                        // both values and both scales at once
                        const uint32_t ca = x.vraw[2 * i][e0 / 8], cb = x.vraw[2 * i + 1][e0 / 8];
                        const uint32_t even = (ca & 0x0F0F0F0Fu) | ((cb << 4) & 0xF0F0F0F0u);
                        const uint32_t odd = ((ca >> 4) & 0x0F0F0F0Fu) | (cb & 0xF0F0F0F0u);
                        const f16x2v gs = __builtin_bit_cast(f16x2v, f16_of_e4m3<false>(vs[i]));
                        const uint4 ve = f16_of_nvfp4(even, gs), vo = f16_of_nvfp4(odd, gs);
                        const uint32_t d[8] = {ve.x, vo.x, ve.y, vo.y, ve.z, vo.z, ve.w, vo.w};
#pragma unroll
                        for (int e = 0; e < EN; ++e) vt[i][e] = d[e];
                    } else {
#pragma unroll
                        for (int y = 0; y < EN / 2; ++y) {
                            uint32_t p0, p1;   // columns (2 y, 2 y + 1) of either token
                            if constexpr (KV == kKv16) {
                                p0 = x.vraw[2 * i][e0 / 2 + y];
                                p1 = x.vraw[2 * i + 1][e0 / 2 + y];
                            } else {
                                const uint32_t w0 = x.vraw[2 * i][e0 / 4 + y / 2], w1 = x.vraw[2 * i + 1][e0 / 4 + y / 2];
                                p0 = (y & 1) ? f16_of_e4m3<true>(w0) : f16_of_e4m3<false>(w0);
                                p1 = (y & 1) ? f16_of_e4m3<true>(w1) : f16_of_e4m3<false>(w1);
                            }
                            vt[i][2 * y] = __builtin_amdgcn_perm(p1, p0, 0x05040100u);
                            vt[i][2 * y + 1] = __builtin_amdgcn_perm(p1, p0, 0x07060302u);
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < EN; ++e) {
                    const uint4 vf = make_uint4(vt[0][e], vt[1][e], vt[2][e], vt[3][e]);
                    acc[e0 + e] = mma16<F16>(vf, pf, acc[e0 + e]);
                    if constexpr (FINE) acc[e0 + e] = mma16<F16>(vf, pl, acc[e0 + e]);
                }
            }
        };

        auto step_down = [&](int t) {   // before the tile at t
            if (pair_begin + (t - base_t) / kAttnUnit < prio_place) return;
            prio_place += quarter;
            if (--prio == 2) __builtin_amdgcn_s_setprio(2);
            else if (prio == 1) __builtin_amdgcn_s_setprio(1);
            else __builtin_amdgcn_s_setprio(0);
        };

        // ---- the tiles.  Loads run one tile ahead where the registers hold
        // two tiles (with the accumulators and q within 200 of 256; the scales
        // and transposes, not counted here, take NVFP4 at D = 256 to 262).  Two
        // ahead are slower: 131072 tokens (E4M3) 63 us instead of 56.
        constexpr bool AHEAD = FAST && 2 * (KP * 8 + VW * 8) + VD * 4 + KSTEPS * 4 <= 200;
        if (t0 < t_stop) {
            if constexpr (FAST) place_rows(t0);
            Tile x0, x1;
            load_tile(x0, t0);
            if constexpr (KV != kKv16) {   // q to fp16, while the first tile is on its way
                uint32_t top = 0u;
                float f[KSTEPS][8];
#pragma unroll
                for (int j = 0; j < KSTEPS; ++j) {
                    if (y->f16) unpack8<true>(qf[j], f[j]);
                    else unpack8<false>(qf[j], f[j]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t v = __float_as_uint(f[j][e]) & 0x7FFFFFFFu;
                        top = v > top ? v : top;
                    }
                }
                uint32_t o = __shfl_xor(top, 16);
                top = o > top ? o : top;
                o = __shfl_xor(top, 32);
                top = o > top ? o : top;
                // the largest to [2^14, 2^15): 2^14 more than [1, 2) for the columns below it
                int ex = (int)(top >> 23);
                ex = ex < 15 ? 15 : (ex > 253 ? 253 : ex);
                const float down = __uint_as_float((uint32_t)(268 - ex) << 23);   // 2^(141 - ex)
#pragma unroll
                for (int j = 0; j < KSTEPS; ++j) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[j][e] *= down;
                    qf[j] = pack8<true>(f[j]);
                }
                qk_log2 *= __uint_as_float((uint32_t)(ex - 14) << 23);
                if (y->kc.scale) qk_log2 *= ((AttnScales)(uint64_t)y->kc.scale)[hk];
            }
            if constexpr (AHEAD) {
                for (;;) {
                    step_down(t0);
                    load_tile(x1, t0 + kAttnUnit);
                    work_tile(x0);
                    t0 += kAttnUnit;
                    if (t0 >= t_stop) break;
                    if (turn == 64) place_rows(t0 + kAttnUnit);
                    load_tile(x0, t0 + kAttnUnit);
                    work_tile(x1);
                    t0 += kAttnUnit;
                    if (t0 >= t_stop) break;
                }
            } else {
                for (;;) {
                    step_down(t0);
                    work_tile(x0);
                    t0 += kAttnUnit;
                    if (t0 >= t_stop) break;
                    if (FAST && turn == 64) place_rows(t0);
                    load_tile(x0, t0);
                }
            }
        }

        // ---- join the waves: every lane's sum is of its own tokens, its
        // maximum of all four groups'.  The arguments this part needs are
        // fetched again, so that the loop does not have to keep them.
        const KernArgs* z = kernel_args();
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (g == 0) {
            s_m[w][c] = m;
            s_l[w][c] = l;
        }
        const int hp = z->G < kAttnHeads ? z->G : kAttnHeads;
        const int part_floats = hp * (D + 2);
        const bool whole = unit0 == 0 && unit1 == units;
        // a workgroup's partial result is its second one if the pair's first place lies inside its stretch
        float* part = z->partials + (int64_t)(me * 2 + (pair_begin > p_begin ? 1 : 0)) * part_floats;
        const float vscale = KV != kKv16 && z->vc.scale ? ((AttnScales)(uint64_t)z->vc.scale)[hk] : 1.0f;
        uint16_t* out = z->out + b * z->o_b + (int64_t)head0 * z->o_h;
        float* lse = z->lse ? z->lse + (int64_t)b * z->Hq + head0 : nullptr;
        const int64_t o_h = z->o_h;
        const bool out_f16 = z->f16 != 0;
        auto store_out = [&](int h, int d, float v0, float v1) {
            const uint32_t o = out_f16 ? pack_round2<true>(fp32_value(v0), fp32_value(v1))
                                       : pack_round2<false>(fp32_value(v0), fp32_value(v1));
            *reinterpret_cast<uint32_t*>(out + h * o_h + d) = o;
        };
        auto store_lse = [&](int h, float mm, float ll) {
            if (lse) lse[h] = ll > 0.f ? (mm + __log2f(ll)) * 0.69314718055994530942f : (ll == 0.f ? -INFINITY : ll);
        };
#pragma unroll
        for (int pass = 0; pass < PASSES; ++pass) {
            if (pass > 0) __syncthreads();
            if (c < nh) {
#pragma unroll
                for (int rr = 0; rr < RP; ++rr)
#pragma unroll
                    for (int e = 0; e < VD; ++e) s_o[(w * nh + c) * OS + (g * RP + rr) * VD + e] = acc[e][pass * RP + rr];
            }
            __syncthreads();
            for (int i = threadIdx.x; i < nh * (LD / 2); i += kAttnThreads) {
                const int h = i / (LD / 2), ld = (i - h * (LD / 2)) * 2;
                // local column -> column: (4 g + row) VD + e
                const int d = ((ld / (RP * VD)) * 4 + pass * RP) * VD + ld % (RP * VD);
                if (!FAST && d >= D) continue;
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
                if (whole) {
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
        if (whole) {
            __syncthreads();   // LDS is free for the next segment
            continue;
        }
        // The workgroups of the pair: the one holding its first unit (of which
        // this can be the only pair that goes on past its stretch: the counter
        // is that workgroup's) to the one holding its last.
        // Workgroup j holds place p if it is the last with floor(j P / N) <= p.
        const int j0 = quotient((int64_t)groups * (pair_begin + front + 1) - 1, places);
        const int j1 = quotient((int64_t)groups * (pair_begin + units + front) - 1, places);
        const int parts = j1 - j0 + 1;
        if (!split_arrive(z->counters, j0, parts, &s_flag)) continue;
        // ---- the workgroup that arrived last joins all of them, in their
        // order: the sum of (factor x partial sums), the factor of a (partial
        // result, head) being exp2(its maximum - the largest) over the sum of
        // weights.
        // workgroup j0's is its first partial result or its second, the others' are their first
        const int second = quotient((int64_t)j0 * places, groups) < pair_begin ? part_floats : 0;
        const float* parts0 = z->partials + (int64_t)j0 * 2 * part_floats;
        auto load2 = [&](const float* from) {
            return __hip_atomic_load(reinterpret_cast<const uint64_t*>(from), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        };
        const int half = D / 2;
        uint64_t v[kAttnJoin];
        auto fetch = [&](const float* from, int x0) {   // partial results x0 .. (the last one again past the end)
            from += (int64_t)x0 * 2 * part_floats + (x0 == 0 ? second : 0);
#pragma unroll
            for (int x = 0; x < kAttnJoin; ++x) {
                v[x] = load2(from);
                from += x0 + x + 1 < parts ? 2 * part_floats - (x0 + x == 0 ? second : 0) : 0;
            }
        };
        if (parts <= kAttnJoin) {
            // few: each thread fetches its head's (maximum, sum) pairs with its
            // columns and works the factors out itself, one round trip in all
            for (int i = threadIdx.x; i < nh * half; i += kAttnThreads) {
                const int h = i / half, d = (i - h * half) * 2;
                uint64_t ml[kAttnJoin];
                fetch(parts0 + hp * D + 2 * h, 0);
#pragma unroll
                for (int x = 0; x < kAttnJoin; ++x) ml[x] = v[x];
                fetch(parts0 + h * D + d, 0);
                float mm = __uint_as_float((uint32_t)ml[0]);
#pragma unroll
                for (int x = 1; x < kAttnJoin; ++x) mm = fmaxf(mm, __uint_as_float((uint32_t)ml[x]));
                float ll = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
                for (int x = 0; x < kAttnJoin; ++x) {
                    const float mx = __uint_as_float((uint32_t)ml[x]);
                    const float f = x >= parts || mx == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mx - mm);
                    if (x < parts) {
                        ll = __builtin_fmaf(f, __uint_as_float((uint32_t)(ml[x] >> 32)), ll);
                        o0 = __builtin_fmaf(f, __uint_as_float((uint32_t)v[x]), o0);
                        o1 = __builtin_fmaf(f, __uint_as_float((uint32_t)(v[x] >> 32)), o1);
                    }
                }
                const float inv = ll == 0.f ? 0.f : vscale / ll;
                store_out(h, d, o0 * inv, o1 * inv);
                if (d == 0) store_lse(h, mm, ll);
            }
            __syncthreads();
            continue;
        }
        // many: the factors go through LDS, a wave per head and a lane per
        // partial result, while each thread's first loads are under way
        float* s_f = s_o;   // [parts][nh]
        int i = threadIdx.x;
        auto columns = [&](int i) { return parts0 + (i < nh * half ? (i / half) * D + (i % half) * 2 : 0); };
        fetch(columns(i), 0);
        for (int h = w; h < nh; h += kAttnWaves) {
            constexpr int LANE_PARTS = kAttnMaxWorkgroups / 64;
            float mx[LANE_PARTS], lx[LANE_PARTS];
            float mm = -INFINITY;
#pragma unroll
            for (int y = 0; y < LANE_PARTS; ++y) {
                mx[y] = -INFINITY;
                lx[y] = 0.f;
                const int x = lane + 64 * y;
                if (x < parts) {
                    const uint64_t ml = load2(parts0 + (int64_t)x * 2 * part_floats + (x == 0 ? second : 0) + hp * D + 2 * h);
                    mx[y] = __uint_as_float((uint32_t)ml);
                    lx[y] = __uint_as_float((uint32_t)(ml >> 32));
                }
            }
#pragma unroll
            for (int y = 0; y < LANE_PARTS; ++y) mm = fmaxf(mm, mx[y]);
            mm = attn_wave_reduce(mm, [](float p, float q) { return fmaxf(p, q); });
            float ll = 0.f;
#pragma unroll
            for (int y = 0; y < LANE_PARTS; ++y) {
                mx[y] = mx[y] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mx[y] - mm);
                ll += mx[y] * lx[y];
            }
            ll = attn_wave_reduce(ll, [](float p, float q) { return p + q; });
            const float inv = ll == 0.f ? 0.f : vscale / ll;
#pragma unroll
            for (int y = 0; y < LANE_PARTS; ++y)
                if (lane + 64 * y < parts) s_f[(lane + 64 * y) * nh + h] = mx[y] * inv;
            if (lane == 0) store_lse(h, mm, ll);
        }
        __syncthreads();
        for (;;) {
            float o0 = 0.f, o1 = 0.f;
            const int h = i / half;
            for (int x0 = 0;;) {
#pragma unroll
                for (int x = 0; x < kAttnJoin; ++x) {
                    if (x0 + x >= parts) break;
                    const float f = s_f[(x0 + x) * nh + (h < nh ? h : 0)];
                    o0 = __builtin_fmaf(f, __uint_as_float((uint32_t)v[x]), o0);
                    o1 = __builtin_fmaf(f, __uint_as_float((uint32_t)(v[x] >> 32)), o1);
                }
                x0 += kAttnJoin;
                if (x0 >= parts) break;
                fetch(columns(i), x0);
            }
            if (i < nh * half) store_out(h, (i - h * half) * 2, o0, o1);
            i += kAttnThreads;
            if (i - (int)threadIdx.x >= nh * half) break;
            fetch(columns(i), 0);
        }
        __syncthreads();
    }
}

}  // namespace nvfp4
