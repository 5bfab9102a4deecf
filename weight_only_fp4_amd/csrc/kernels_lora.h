// Low-rank adapters of many requests beside a shared projection (nvfp4_lora_add):
//
//   out[t] = RNE16(y[t] + s_a (x[t] A_a^T) B_a^T),  a = adapter[t]
//
// in two launches: k_lora_down makes h = x A_a^T (fp32, [K slice][row][rank]),
// k_lora_up adds s_a h B_a^T to y.
//
// Rows are taken 16 at a time in the order they come, and a tile's rows are
// multiplied by each of the adapters that occur among them, one after another
// or a workgroup each; an MFMA's row results do not depend on its other rows,
// so rows of other adapters are computed and not stored.  A prompt's tokens
// share their adapter (one or two a tile), and in a decoding batch the tiles
// are few, so that re-reading an adapter for another tile is an L2 hit; sorting
// the rows first would cost a launch more than the second product takes.
//
// What bounds it: the adapters' and rows' bytes.  r is small, so the matrix
// instructions wait for loads everywhere: 2 r flops a value of x read.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decode.h"

namespace nvfp4 {

constexpr int kLoraRows = 16;        // rows of a tile
constexpr int kLoraThreads = 256;
constexpr int kLoraWaves = kLoraThreads / 64;
constexpr int kLoraMaxRank = 128;
constexpr int kLoraCols = 64;        // output columns a wave and step of k_lora_up

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
    int vec;               // rows of y and out are 16-byte aligned
};

// The tile's rows (lane l: row l & 15) and what they belong to; none: -1.
struct LoraTile {
    int t0, rows, mine;
    uint32_t left;   // rows whose adapter is still to come
    __device__ __forceinline__ LoraTile(const LoraArgs& a, int tile) {
        const int lane = threadIdx.x & 63;
        t0 = tile * kLoraRows;
        rows = a.T - t0 < kLoraRows ? a.T - t0 : kLoraRows;
        const int r = lane & 15;
        const int id = r < rows ? a.adapter[t0 + r] : -1;
        mine = id >= 0 && id < a.L ? id : -1;
        left = (uint32_t)(__ballot(mine >= 0) & 0xFFFFu);
    }
    // The next adapter among the rows, and its rows; false when there is none.
    __device__ __forceinline__ bool next(int& adapter, uint32_t& its) {
        if (!left) return false;
        adapter = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
        its = (uint32_t)(__ballot(mine == adapter) & 0xFFFFu);
        left &= ~its;
        return true;
    }
};

// RT rank tiles of 16.  Grid: (K slices, row tiles, 1 or the places of a
// tile's adapters).  A wave takes a quarter of the slice's 128-value chunks;
// the four waves' sums meet in LDS.  Lane l of a chunk holds 32 consecutive
// values of row l & 15 from 32 (l >> 4) on, of x and of A alike.
template <int RT, bool F16>
__global__ void __launch_bounds__(kLoraThreads) k_lora_down(LoraArgs a) {
    __shared__ float red[kLoraWaves][RT * 16 * kLoraRows];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, r = lane & 15;
    LoraTile tile(a, blockIdx.y);
    const int k0 = blockIdx.x * a.slice, k1 = k0 + a.slice < a.K ? k0 + a.slice : a.K;
    const int chunks = (k1 - k0 + 127) / 128;
    const int c0 = chunks * w / kLoraWaves, c1 = chunks * (w + 1) / kLoraWaves;
    const uint16_t* xr = a.x + (int64_t)(tile.t0 + (r < tile.rows ? r : 0)) * a.ld_x;
    int adapter;
    uint32_t its;
    for (int place = 0; tile.next(adapter, its); ++place) {
        if (gridDim.z > 1 && place != (int)blockIdx.z) continue;
        f32x4 acc[RT];
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        const uint16_t* ar[RT];
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            const int row = 16 * j + r;
            ar[j] = a.a + (int64_t)adapter * a.a_l + (int64_t)(row < a.R ? row : 0) * a.a_r;
        }
        for (int c = c0; c < c1; ++c) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                // pieces past the slice read its first values, and count as zeros on both sides
                const int k = k0 + c * 128 + 32 * g + 8 * t;
                const bool in = k < k1;
                const int at = in ? k : k0;
                uint4 xv = *reinterpret_cast<const uint4*>(xr + at);
                if (!in) xv = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int j = 0; j < RT; ++j) {
                    uint4 av = *reinterpret_cast<const uint4*>(ar[j] + at);
                    if (!in) av = make_uint4(0u, 0u, 0u, 0u);
                    acc[j] = mma16<F16>(xv, av, acc[j]);
                }
            }
        }
        // lane: rows 4 g + i, rank 16 j + r
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[w][(4 * g + i) * (RT * 16) + 16 * j + r] = acc[j][i];
        __syncthreads();
        for (int i = threadIdx.x; i < kLoraRows * RT * 16; i += kLoraThreads) {
            const int row = i / (RT * 16), rank = i % (RT * 16);
            if (((its >> row) & 1u) && rank < a.R) {
                float sum = 0.f;
#pragma unroll
                for (int ww = 0; ww < kLoraWaves; ++ww) sum += red[ww][i];
                a.h[((int64_t)blockIdx.x * a.T + tile.t0 + row) * a.R + rank] = sum;
            }
        }
        __syncthreads();
    }
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

// KT steps of 32 ranks.  Grid: (column blocks, row tiles, 1 or the places of a
// tile's adapters); place 0 also hands on the rows without an adapter.  The
// products are taken with B's rows first, in an order that leaves lane l with
// row l & 15's eight consecutive columns 8 (l >> 4) .. + 7 of every 32.
template <int KT, bool F16>
__global__ void __launch_bounds__(kLoraThreads) k_lora_up(LoraArgs a) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, r = lane & 15;
    LoraTile tile(a, blockIdx.y);
    const int n0 = (blockIdx.x * kLoraWaves + w) * kLoraCols;
    const int t = tile.t0 + (r < tile.rows ? r : 0);
    const uint16_t* yr = a.y + (int64_t)t * a.ld_y;
    uint16_t* orow = a.out + (int64_t)t * a.ld_o;
    const bool copies = a.out != a.y && blockIdx.z == 0 && r < tile.rows && tile.mine < 0;
    auto columns = [&](int n, auto&& delta) {   // out = y + delta(e) for columns n .. n + 7
        if (a.vec && n + 8 <= a.N) {
            const uint4 v = *reinterpret_cast<const uint4*>(yr + n);
            const uint32_t in[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = pack_round2<F16>(fp32_value(act_to_f32<F16>(in[e] & 0xFFFFu) + delta(2 * e)),
                                        fp32_value(act_to_f32<F16>(in[e] >> 16) + delta(2 * e + 1)));
            *reinterpret_cast<uint4*>(orow + n) = make_uint4(o[0], o[1], o[2], o[3]);
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (n + e < a.N) orow[n + e] = (uint16_t)round_out<F16>(fp32_value(act_to_f32<F16>(yr[n + e]) + delta(e)));
    };
    if (copies)
        for (int s = 0; s < kLoraCols; s += 32)
            for (int e = 0; e < 8; ++e)
                if (n0 + s + 8 * g + e < a.N) orow[n0 + s + 8 * g + e] = yr[n0 + s + 8 * g + e];
    int adapter;
    uint32_t its;
    for (int place = 0; tile.next(adapter, its); ++place) {
        if (gridDim.z > 1 && place != (int)blockIdx.z) continue;
        const bool mine = (its >> r) & 1u;
        // this lane's values of h: rank 32 s + 8 g .. + 7 of row r (rows of other adapters as zeros)
        float hv[KT][8];
        float most = 0.f;
#pragma unroll
        for (int s = 0; s < KT; ++s) {
#pragma unroll
            for (int e = 0; e < 8; ++e) hv[s][e] = 0.f;
            const int rank = 32 * s + 8 * g;
            if (mine && rank < a.R)
                for (int sl = 0; sl < a.slices; ++sl) {
                    const float4* p = reinterpret_cast<const float4*>(a.h + ((int64_t)sl * a.T + t) * a.R + rank);
                    const float4 p0 = p[0], p1 = p[1];
                    hv[s][0] += p0.x, hv[s][1] += p0.y, hv[s][2] += p0.z, hv[s][3] += p0.w;
                    hv[s][4] += p1.x, hv[s][5] += p1.y, hv[s][6] += p1.z, hv[s][7] += p1.w;
                }
#pragma unroll
            for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(hv[s][e]));
        }
        float up = 1.f, down = a.scale ? a.scale[adapter] : 1.f;
        if (F16) {
            most = fmaxf(most, __shfl_xor(most, 16));
            most = fmaxf(most, __shfl_xor(most, 32));
            int e = most > 0.f && most < __builtin_inff() ? 13 - ilogbf(most) : 0;
            e = e > 126 ? 126 : e < -126 ? -126 : e;
            up = ldexpf(1.f, e);
            down = down * ldexpf(1.f, -e);
        }
        uint4 hi[KT], lo[KT];
#pragma unroll
        for (int s = 0; s < KT; ++s) lora_split<F16>(hv[s], up, hi[s], lo[s]);
        const uint16_t* bl = a.b + (int64_t)adapter * a.b_l;
#pragma unroll
        for (int s0 = 0; s0 < kLoraCols; s0 += 32) {
            f32x4 acc[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
                const int n = n0 + s0 + 8 * (r >> 2) + 4 * j + (r & 3);
                const uint16_t* br = bl + (int64_t)(n < a.N ? n : 0) * a.b_n;
#pragma unroll
                for (int s = 0; s < KT; ++s) {
                    const int rank = 32 * s + 8 * g;
                    uint4 bv = *reinterpret_cast<const uint4*>(br + (rank < a.R ? rank : 0));
                    if (rank >= a.R) bv = make_uint4(0u, 0u, 0u, 0u);
                    acc[j] = mma16<F16>(bv, hi[s], acc[j]);
                    acc[j] = mma16<F16>(bv, lo[s], acc[j]);
                }
            }
            if (mine) columns(n0 + s0 + 8 * g, [&](int e) { return down * acc[e >> 2][e & 3]; });
        }
    }
}

}  // namespace nvfp4
