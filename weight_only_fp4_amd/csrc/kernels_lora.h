// Low-rank adapters of many requests beside a shared projection (nvfp4_lora_add):
//
//   out[t] = RNE16(y[t] + s_a (x[t] A_a^T) B_a^T),  a = adapter[t]
//
// in two launches: k_lora_down makes h = x A_a^T (fp32, [K slice][row][rank]),
// k_lora_up adds s_a h B_a^T to y.
//
// What bounds it: the adapters' and rows' bytes.  r is small, so the matrix
// instructions wait for loads everywhere (2 r flops a value of x read), and an
// adapter should be read once.  A workgroup therefore makes the list of an
// adapter's rows itself and takes them 16 at a time with the adapter's
// fragments in registers; there is no launch that sorts.  With up to kLoraLists
// rows (a decoding batch: adapters in any order) a workgroup belongs to an
// adapter and looks through all rows; with more (prompts, whose tokens share
// their adapter) it belongs to 64 neighbouring rows and takes the adapters that
// occur among them one after another.
//
// Measured in a graph over sets of inputs beyond the last cache, the two kernels'
// own times behind: 16 tokens of 32 adapters, 4096 x 4096, rank 16 8.5 us (4.0 +
// 5.3); 133 tokens of 12, 4096 x 14336, rank 64 20.5 (7.3 + 13.7; 37 MB, 1.8
// TB/s); 4099 rows of 6 prompts, 5120 x 5120, rank 32 49 (20.3, 2.1 TB/s, + 29.8,
// 2.8 TB/s).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decode.h"

namespace nvfp4 {

constexpr int kLoraRows = 16;        // rows of a product
constexpr int kLoraTile = 64;        // neighbouring rows of a workgroup
// Rows up to which a workgroup belongs to an adapter.  T and L alone do not say
// how the rows are spread (that is on the device), and each form loses where the
// other wins.  Lists against tiles, us, 4096 x 4096, rank 16: 256 rows of one of 40
// adapters 29, 14; of 32 in any order 13, 26; 300 of 32 in any order 14, 26; of 3
// prompts 13, 14; 512 of 8 in any order 22, 13; 1000 of 16 30, 27; 1000 of 4
// prompts 29, 16; 361 rows of one of 40, 2421 columns, 64, 20.  Lists end where
// their worst case has grown to four times the other's and tiles' stays at twice:
// rows of one adapter have a workgroup for all of them in lists, rows in any order
// a turn for each adapter in tiles.
constexpr int kLoraLists = 256;
constexpr int kLoraThreads = 256;
constexpr int kLoraWaves = kLoraThreads / 64;
constexpr int kLoraMaxRank = 128;
constexpr int kLoraCols = 32;        // output columns a wave of k_lora_up takes at a time

template <int N>
struct LoraTiles {
    static constexpr int value = N;
};

struct LoraArgs {
    const uint16_t* x;
    const uint16_t* a;
    const uint16_t* b;
    const uint16_t* y;
    uint16_t* out;
    const int32_t* adapter;
    const float* scale;    // or NULL: 1
    float* h;              // [slices][T][rank] workspace
    int64_t ld_x, ld_y, ld_o;
    int64_t a_l, a_r, b_l, b_n;   // strides of adapters and rows, in values
    int T, K, N, R, L;
    int slices, slice;     // K slices and the values of one (a multiple of 8)
    int cols;              // output columns of a wave, a multiple of kLoraCols
    int places;            // workgroups by adapter: min(L, T); 0: by neighbouring rows
};

// f(adapter, count) for each of a workgroup's adapters, with the adapter's
// rows in list[0 .. count) in order; every wave makes the same list, and f may
// hold barriers.  `place`: the adapter (L <= T), the row that must be its
// adapter's first (L > T), or the tile of neighbouring rows, whose adapters go
// to `turns` workgroups in turn.  none(mask, row) for rows that have no adapter:
// lanes of the mask hold one, and all places (or turn 0) together have them all.
template <typename F, typename N>
__device__ __forceinline__ void lora_rows(const LoraArgs& a, int place, int turn, int turns, int32_t* list, F&& f, N&& none) {
    const int lane = threadIdx.x & 63;
    const uint64_t before = (1ull << lane) - 1;
    if (a.places == 0) {
        const int t = place * kLoraTile + lane;
        int id = t < a.T ? a.adapter[t] : -1;
        id = id >= 0 && id < a.L ? id : -1;
        if (turn == 0) none(__ballot(t < a.T && id < 0), t);
        int nth = 0;
        for (uint64_t left = __ballot(id >= 0); left; ++nth) {
            const int adapter = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
            const uint64_t its = __ballot(id == adapter);
            left &= ~its;
            if (nth % turns != turn) continue;
            if (id == adapter) list[__popcll(its & before)] = t;
            f(adapter, __popcll(its));
        }
        return;
    }
    int adapter = a.L > a.T ? a.adapter[place] : place;
    if (adapter < 0 || adapter >= a.L) adapter = -1;   // (with no adapters at all there is one place, for their rows)
    int count = 0, others = 0;
    bool first = true;
    for (int t0 = 0; t0 < a.T; t0 += 64) {
        const int t = t0 + lane, id = t < a.T ? a.adapter[t] : 0;
        const uint64_t its = __ballot(t < a.T && id == adapter && adapter >= 0);
        if (a.L > a.T && its && count == 0) first = t0 + __builtin_ctzll(its) == place;
        if ((its >> lane) & 1ull) list[count + __popcll(its & before)] = t;
        count += __popcll(its);
        // rows without an adapter go to the places in turn
        const bool has_none = t < a.T && (id < 0 || id >= a.L);
        const uint64_t nones = __ballot(has_none);
        if (nones && turn == 0) none(__ballot(has_none && (others + __popcll(nones & before)) % a.places == place), t);
        others += __popcll(nones);
    }
    if (count > 0 && first) f(adapter, count);
}

// A wave's part of the products of 16 M rows (xr: this lane's, r = lane & 15)
// with an adapter's RT rank tiles, over chunks [c0, c1) of 128 values from k0.
// Lane l of a step of 32 has the eight values from 8 (l >> 4) on, of x and of A
// alike; pieces past k1 read the slice's first values, and count as zeros on
// both sides.
template <int RT, int M, bool F16>
__device__ __forceinline__ void lora_chunks(const uint16_t* const (&xr)[M], const uint16_t* const (&ar)[RT], int k0, int k1, int c0,
                                            int c1, f32x4 (&acc)[M][RT]) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int c = c0; c < c1; ++c) {
        uint4 xv[M][4], av[RT][4];
        bool in[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int k = k0 + c * 128 + 32 * t + 8 * g;
            in[t] = k < k1;
            const int at = in[t] ? k : k0;
#pragma unroll
            for (int m = 0; m < M; ++m) xv[m][t] = *reinterpret_cast<const uint4*>(xr[m] + at);
#pragma unroll
            for (int j = 0; j < RT; ++j) av[j][t] = *reinterpret_cast<const uint4*>(ar[j] + at);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const uint4 x = in[t] ? av[j][t] : zero;
#pragma unroll
                for (int m = 0; m < M; ++m) acc[m][j] = mma16<F16>(in[t] ? xv[m][t] : zero, x, acc[m][j]);
            }
        }
    }
}

// RT rank tiles of 16, MT tiles of 16 rows at a time (or one, where a list has
// no more).  Grid: (K slices, places or tiles, shares of a list or turns).  Each
// wave takes a share of the slice's chunks; the waves' sums meet in LDS.
template <int RT, int MT, bool F16>
__global__ void __launch_bounds__(kLoraThreads) k_lora_down(LoraArgs a) {
    __shared__ float red[kLoraWaves][MT * kLoraRows * RT * 16];
    __shared__ int32_t list[kLoraLists];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, r = lane & 15;
    const int k0 = blockIdx.x * a.slice, k1 = k0 + a.slice < a.K ? k0 + a.slice : a.K;
    const int chunks = (k1 - k0 + 127) / 128;
    const int c0 = chunks * w / kLoraWaves, c1 = chunks * (w + 1) / kLoraWaves;
    auto rows = [&](int adapter, int count) {
        const uint16_t* ar[RT];
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            const int row = 16 * j + r;
            ar[j] = a.a + (int64_t)adapter * a.a_l + (int64_t)(row < a.R ? row : 0) * a.a_r;
        }
        auto take = [&](auto tiles, int s0) {
            constexpr int M = decltype(tiles)::value;
            f32x4 acc[M][RT];
            const uint16_t* xr[M];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int at = s0 + kLoraRows * m + r;
                xr[m] = a.x + (int64_t)list[at < count ? at : s0] * a.ld_x;
            }
            lora_chunks<RT, M, F16>(xr, ar, k0, k1, c0, c1, acc);
            // lane: rows 4 g + i, rank 16 j + r
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int j = 0; j < RT; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) red[w][(kLoraRows * m + 4 * g + i) * (RT * 16) + 16 * j + r] = acc[m][j][i];
            __syncthreads();
            for (int i = threadIdx.x; i < M * kLoraRows * RT * 16; i += kLoraThreads) {
                const int row = s0 + i / (RT * 16), rank = i % (RT * 16);
                if (row < count && rank < a.R) {
                    float sum = 0.f;
#pragma unroll
                    for (int ww = 0; ww < kLoraWaves; ++ww) sum += red[ww][i];
                    a.h[((int64_t)blockIdx.x * a.T + list[row]) * a.R + rank] = sum;
                }
            }
            __syncthreads();
        };
        const int share = a.places ? blockIdx.z : 0, shares = a.places ? gridDim.z : 1;
        for (int s0 = share * MT * kLoraRows; s0 < count; s0 += shares * MT * kLoraRows) {
            if (count - s0 <= kLoraRows) take(LoraTiles<1>{}, s0);
            else take(LoraTiles<MT>{}, s0);
        }
    };
    lora_rows(a, blockIdx.y, blockIdx.z, gridDim.z, list, rows, [](uint64_t, int) {});
}

// Sixteen bits of the rows' h (fp32) in two parts, the rounded values and what
// the rounding took off, so that h counts with 16 (bf16) or 22 (fp16) bits.  In
// fp16 a row is first scaled by a power of two that brings its largest value
// to [2^13, 2^14): the range of x A_a^T is not that of fp16.
template <bool F16>
__device__ __forceinline__ void lora_split(const float (&v)[8], float up, uint4& hi, uint4& lo) {
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float v0 = v[2 * e] * up, v1 = v[2 * e + 1] * up;
        ph[e] = pack_round2<F16>(v0, v1);
        // an infinity (or NaN) leaves nothing over
        const float d0 = v0 - act_to_f32<F16>(ph[e] & 0xFFFFu), d1 = v1 - act_to_f32<F16>(ph[e] >> 16);
        pl[e] = pack_round2<F16>(fabsf(d0) < __builtin_inff() ? d0 : 0.f, fabsf(d1) < __builtin_inff() ? d1 : 0.f);
    }
    hi = make_uint4(ph[0], ph[1], ph[2], ph[3]);
    lo = make_uint4(pl[0], pl[1], pl[2], pl[3]);
}

// Eight values of a row of y or out, whose rows begin anywhere: one access of 16
// bytes, which global memory takes at any address (8296 rows of 1031 columns: 27
// us, by two bytes 52; aligned rows as before).
struct __attribute__((packed, aligned(2))) LoraPiece {
    uint32_t w[4];
};
__device__ __forceinline__ uint4 lora_load(const uint16_t* p) {
    const LoraPiece v = *reinterpret_cast<const LoraPiece*>(p);
    return make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}
__device__ __forceinline__ void lora_store(uint16_t* p, uint4 v) {
    *reinterpret_cast<LoraPiece*>(p) = LoraPiece{{v.x, v.y, v.z, v.w}};
}

// KT steps of 32 ranks.  Grid: (column blocks, places or tiles, shares of a list
// or turns).  64 rows of a list at a time: their h is added up over the K slices
// and split, into LDS in the order of the matrix instruction's operand; then a
// wave goes through its columns, 32 at a time, with B's fragments for them in
// registers and the rows' y on their way.  The products are taken with B's rows
// first, in an order that leaves lane l with row l & 15's eight consecutive
// columns 8 (l >> 4) .. + 7.
template <int KT, bool F16>
__global__ void __launch_bounds__(kLoraThreads) k_lora_up(LoraArgs a) {
    constexpr int kTiles = kLoraTile / kLoraRows;
    __shared__ uint4 s_h[kTiles][KT][2][64];
    __shared__ float s_down[kTiles][kLoraRows];
    __shared__ float s_sum[kLoraTile][32 * KT + 4];   // four more: rows begin in other banks
    __shared__ uint32_t s_most[kLoraTile];
    __shared__ int32_t s_none[kLoraWaves][64];
    __shared__ int32_t list[kLoraLists];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, r = lane & 15;
    const int n_first = (blockIdx.x * kLoraWaves + w) * a.cols, n_end = n_first + a.cols < a.N ? n_first + a.cols : a.N;
    if (threadIdx.x < kLoraTile) s_most[threadIdx.x] = 0;
    __syncthreads();
    auto rows = [&](int adapter, int count) {
        const uint16_t* bl = a.b + (int64_t)adapter * a.b_l;
        const float scale = a.scale ? a.scale[adapter] : 1.f;
        const int share = a.places ? blockIdx.z : 0, shares = a.places ? gridDim.z : 1;
        for (int s0 = share * kLoraTile; s0 < count; s0 += shares * kLoraTile) {
            const int tiles = count - s0 >= kLoraTile ? kTiles : (count - s0 + kLoraRows - 1) / kLoraRows;
            int row[kTiles];   // this lane's of each tile; those past the list: its first, not stored
#pragma unroll
            for (int m = 0; m < kTiles; ++m) row[m] = list[s0 + kLoraRows * m + r < count ? s0 + kLoraRows * m + r : s0];
            // B's fragments and y for the columns from n0 on, asked for one step ahead of their use
            uint4 bv[2][KT], yv[kTiles];
            auto ask = [&](int n0) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int col = n0 + 8 * (r >> 2) + 4 * j + (r & 3);
                    const uint16_t* br = bl + (int64_t)(col < a.N ? col : 0) * a.b_n;
#pragma unroll
                    for (int s = 0; s < KT; ++s) {
                        const int rank = 32 * s + 8 * g;
                        bv[j][s] = *reinterpret_cast<const uint4*>(br + (rank < a.R ? rank : 0));
                    }
                }
                if (a.N >= 8) {   // a piece that is not whole: the row's first, not used
                    const int from = n0 + 8 * g + 8 <= a.N ? n0 + 8 * g : 0;
#pragma unroll
                    for (int m = 0; m < kTiles; ++m)
                        if (m < tiles) yv[m] = lora_load(a.y + (int64_t)row[m] * a.ld_y + from);
                }
            };
            ask(n_first);
            // the rows' h: the slices' sums, four ranks a thread and step
            const int many = count - s0 < kLoraTile ? count - s0 : kLoraTile, quads = a.R / 4;
            for (int i = threadIdx.x; i < many * quads; i += kLoraThreads) {
                const int at = i / quads, rank = 4 * (i - at * quads);
                const float* p = a.h + (int64_t)list[s0 + at] * a.R + rank;
                float4 v = *reinterpret_cast<const float4*>(p);
#pragma unroll 4
                for (int sl = 1; sl < a.slices; ++sl) {
                    const float4 o = *reinterpret_cast<const float4*>(p + (int64_t)sl * a.T * a.R);
                    v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                }
                *reinterpret_cast<float4*>(&s_sum[at][rank]) = v;
                // absolute values order as their bits do
                if (F16)
                    atomicMax(&s_most[at], __float_as_uint(fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)))));
            }
            __syncthreads();
            for (int u = w; u < tiles * KT; u += kLoraWaves) {   // (tile of 16 rows, step of 32 ranks)
                const int m = u / KT, s = u % KT, at = kLoraRows * m + r, rank = 32 * s + 8 * g;
                float hv[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) hv[e] = at < many && rank < a.R ? s_sum[at][rank + e] : 0.f;
                float up = 1.f;
                if (F16) {
                    const float most = __uint_as_float(s_most[at]);
                    int e = at < many && most > 0.f && most < __builtin_inff() ? 13 - ilogbf(most) : 0;
                    e = e > 126 ? 126 : e < -126 ? -126 : e;
                    up = ldexpf(1.f, e);
                    if (s == 0 && g == 0) s_down[m][r] = scale * ldexpf(1.f, -e);
                } else if (s == 0 && g == 0) {
                    s_down[m][r] = scale;
                }
                lora_split<F16>(hv, up, s_h[m][s][0][lane], s_h[m][s][1][lane]);
            }
            __syncthreads();
            if (F16 && threadIdx.x < kLoraTile) s_most[threadIdx.x] = 0;
            for (int n0 = n_first; n0 < n_end; n0 += kLoraCols) {
                const int n = n0 + 8 * g;
                const bool whole = n + 8 <= a.N;
                uint4 b0[2][KT], y0[kTiles];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int s = 0; s < KT; ++s) b0[j][s] = 32 * s + 8 * g < a.R ? bv[j][s] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int m = 0; m < kTiles; ++m) y0[m] = yv[m];
                if (n0 + kLoraCols < n_end) ask(n0 + kLoraCols);
#pragma unroll
                for (int m = 0; m < kTiles; ++m) {
                    if (m >= tiles) break;
                    f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                    for (int s = 0; s < KT; ++s)
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
                            const uint4 hv = s_h[m][s][part][lane];
                            acc[0] = mma16<F16>(b0[0][s], hv, acc[0]);
                            acc[1] = mma16<F16>(b0[1][s], hv, acc[1]);
                        }
                    if (s0 + kLoraRows * m + r >= count) continue;
                    const float down = s_down[m][r];
                    uint16_t* orow = a.out + (int64_t)row[m] * a.ld_o;
                    auto sum = [&](uint32_t y16, int e) {
                        return fp32_value(act_to_f32<F16>(y16) + down * acc[e >> 2][e & 3]);
                    };
                    if (whole) {
                        const uint32_t in[4] = {y0[m].x, y0[m].y, y0[m].z, y0[m].w};
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = pack_round2<F16>(sum(in[e] & 0xFFFFu, 2 * e), sum(in[e] >> 16, 2 * e + 1));
                        lora_store(orow + n, make_uint4(o[0], o[1], o[2], o[3]));
                    } else {
                        // all of y first: out may be its memory, so that loads would stay behind stores
                        const uint16_t* yr = a.y + (int64_t)row[m] * a.ld_y;
                        uint32_t in[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) in[e] = n + e < a.N ? yr[n + e] : 0u;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (n + e < a.N) orow[n + e] = (uint16_t)round_out<F16>(sum(in[e], e));
                    }
                }
            }
            __syncthreads();   // s_h and the list are read
        }
    };
    // rows without an adapter: 16 at a time, four lanes each with eight columns
    auto none = [&](uint64_t mask, int t) {
        if (a.out == a.y || mask == 0) return;
        if ((mask >> lane) & 1ull) s_none[w][__popcll(mask & ((1ull << lane) - 1))] = t;
        const int count = __popcll(mask);
        for (int i = lane >> 2; i < count; i += 16) {
            const int64_t row = s_none[w][i];
            for (int n = n_first + 8 * (lane & 3); n < n_end; n += kLoraCols) {
                const uint16_t* yr = a.y + row * a.ld_y + n;
                uint16_t* orow = a.out + row * a.ld_o + n;
                if (n + 8 <= a.N) {
                    lora_store(orow, lora_load(yr));
                } else {
                    for (int e = 0; e < 8; ++e)
                        if (n + e < a.N) orow[e] = yr[e];
                }
            }
        }
    };
    lora_rows(a, blockIdx.y, blockIdx.z, gridDim.z, list, rows, none);
}

}  // namespace nvfp4
