// Root-mean-square norm of rows, with the residual's addition before it and
// an output in 16 or 8 bits.
#pragma once
#include "decode.h"
#include "quant.h"

namespace nvfp4 {

// Row t of N values:
//   h = RNE16(x + r)  (h = x without a residual; h is stored when asked for),
//   y = h * rsqrt(mean(h^2) + eps) * w                    (fp32),
//   out = RNE16(y), or with F8 out = e4m3(y * (1 / s)), s = max(max |y| / 448, 2^-126).
// The mean is taken over h as it is stored, so the fused call gives what an
// addition in 16 bits followed by a norm gives.  Sums are fp32 in a fixed
// order (lanes, then waves), so results are reproducible.
struct NormArgs {
    const uint16_t *x, *r, *w;
    uint16_t* h;
    void* y;
    float* scales;
    int64_t ld_x, ld_r, ld_h, ld_y;
    int64_t T;
    int N;
    float eps;
};

constexpr int kNormMaxWaves = 16;

// Sum and maximum over aligned groups of L lanes (every lane gets it).
template <int L = 64>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int d = L / 2; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
template <int L = 64>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
    for (int d = L / 2; d >= 1; d >>= 1) {
        const uint32_t o = __shfl_xor(v, d);
        v = o > v ? o : v;
    }
    return v;
}

// A 16-byte piece, streamed past the caches (PAST) or not.
template <bool PAST>
__device__ __forceinline__ uint4 norm_load(const uint16_t* p) {
    if constexpr (PAST) return load_stream_u4(reinterpret_cast<const uint8_t*>(p));
    else return *reinterpret_cast<const uint4*>(p);
}
// h of a 16-byte piece (x plus the residual's, rounded) as fp32; stored if asked for.
template <bool F16>
__device__ __forceinline__ void norm_sum8(const NormArgs& a, int64_t t, int p, uint4 xv, uint4 rv, float (&f)[8]) {
    unpack8<F16>(xv, f);
    if (a.r) {
        float rf[8];
        unpack8<F16>(rv, rf);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += rf[e];
        const uint4 h = pack8<F16>(f);
        if (a.h) *reinterpret_cast<uint4*>(a.h + t * a.ld_h + p * 8) = h;
        unpack8<F16>(h, f);
    }
}

// Rows of at most 8 L values: L lanes a row, no workgroup-wide step.
template <bool F16, bool F8, int L>
__global__ void __launch_bounds__(256) k_rms_norm_short(NormArgs a) {
    const int p = threadIdx.x & (L - 1);
    const int64_t row = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    const bool in = row < a.T && p < (a.N >> 3);
    const int64_t t = row < a.T ? row : 0;
    float f[8] = {};
    uint4 wv = make_uint4(0u, 0u, 0u, 0u);
    if (in) {
        wv = *reinterpret_cast<const uint4*>(a.w + p * 8);
        uint4 rv = wv;
        if (a.r) rv = *reinterpret_cast<const uint4*>(a.r + t * a.ld_r + p * 8);
        norm_sum8<F16>(a, t, p, *reinterpret_cast<const uint4*>(a.x + t * a.ld_x + p * 8), rv, f);
    }
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(f[e], f[e], sum);
    sum = lanes_sum<L>(sum);
    const float inv = rsqrtf(sum / (float)a.N + a.eps);
    float wf[8];
    unpack8<F16>(wv, wf);
    uint32_t top = 0u;   // largest |y| as bits: a NaN's are above infinity's, so it is kept
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        f[e] = f[e] * inv * wf[e];
        const uint32_t u = __float_as_uint(f[e]) & 0x7FFFFFFFu;
        top = in && u > top ? u : top;
    }
    if constexpr (!F8) {
        if (in) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + t * a.ld_y + p * 8) = pack8<F16>(f);
    } else {
        const float scale = norm_row_scale(__uint_as_float(lanes_max<L>(top)));
        if (in) {
            if (p == 0) a.scales[t] = scale;
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + t * a.ld_y + p * 8) = e4m3_pack8(f, __fdiv_rn(1.0f, scale));
        }
    }
}

// One workgroup per row, the row held in registers (V 16-byte pieces a
// thread): one pass over HBM, which bounds it from some hundred rows on: 8192
// rows of 5120 with a residual (336 MB) take 55 us, 6.1 TB/s, and 777 rows to
// E4M3 (28 MB) 8.7 (calls in a graph).  One row of 4096 takes the kernel 2.0 us,
// a call of it in a graph 3.2: a load, the sum over the waves and a store one
// after another.  N, the leading
// dimensions and the pointers keep 16-byte alignment (checked on the host).
template <bool F16, bool F8, int V, bool PAST>
__global__ void __launch_bounds__(64 * kNormMaxWaves) k_rms_norm(NormArgs a) {
    __shared__ float s_sum[kNormMaxWaves];
    __shared__ uint32_t s_max[kNormMaxWaves];
    const int tid = threadIdx.x, threads = blockDim.x, waves = threads >> 6;
    const int64_t t = blockIdx.x;
    const int pieces = a.N >> 3;
    float f[V][8];
    float sum = 0.f;
    uint4 xv[V], rv[V], wv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int p = tid + i * threads;
        if (p < pieces) {
            xv[i] = norm_load<PAST>(a.x + t * a.ld_x + p * 8);
            if (a.r) rv[i] = norm_load<PAST>(a.r + t * a.ld_r + p * 8);
            wv[i] = *reinterpret_cast<const uint4*>(a.w + p * 8);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int p = tid + i * threads;
        if (p < pieces) {
            norm_sum8<F16>(a, t, p, xv[i], rv[i], f[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(f[i][e], f[i][e], sum);
        }
    }
    sum = lanes_sum(sum);
    if (waves > 1) {
        if ((tid & 63) == 0) s_sum[tid >> 6] = sum;
        __syncthreads();
        sum = 0.f;
        for (int i = 0; i < waves; ++i) sum += s_sum[i];
    }
    const float inv = rsqrtf(sum / (float)a.N + a.eps);
    uint32_t top = 0u;   // largest |y| as bits: a NaN's are above infinity's, so it is kept
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int p = tid + i * threads;
        if (p < pieces) {
            float wf[8];
            unpack8<F16>(wv[i], wf);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[i][e] = f[i][e] * inv * wf[e];
                if constexpr (F8) {
                    const uint32_t u = __float_as_uint(f[i][e]) & 0x7FFFFFFFu;
                    top = u > top ? u : top;
                }
            }
            if constexpr (!F8) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + t * a.ld_y + p * 8) = pack8<F16>(f[i]);
        }
    }
    if constexpr (F8) {
        top = lanes_max(top);
        if (waves > 1) {
            if ((tid & 63) == 0) s_max[tid >> 6] = top;
            __syncthreads();
            for (int i = 0; i < waves; ++i) top = s_max[i] > top ? s_max[i] : top;
        }
        const float scale = norm_row_scale(__uint_as_float(top));
        const float back = __fdiv_rn(1.0f, scale);
        if (tid == 0) a.scales[t] = scale;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int p = tid + i * threads;
            if (p < pieces)
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + t * a.ld_y + p * 8) = e4m3_pack8(f[i], back);
        }
    }
}

// Any row length up to 2^31 - 256 (the 32-bit counters then end below 2^31),
// stride and alignment: one workgroup of 256 threads per row, single values,
// the row read again for each of the two or three passes.  With h the later
// passes read h back (each thread its own values), so h may be the residual's
// or x's own memory; y is written in the last pass only.
template <bool F16, bool F8>
__global__ void __launch_bounds__(256) k_rms_norm_any(NormArgs a) {
    __shared__ float s_sum[4];
    __shared__ uint32_t s_max[4];
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x;
    const uint16_t* x = a.x + t * a.ld_x;
    const uint16_t* r = a.r ? a.r + t * a.ld_r : nullptr;
    uint16_t* h = a.h ? a.h + t * a.ld_h : nullptr;
    const bool again = r != nullptr && h != nullptr;
    float sum = 0.f;
    for (int i = tid; i < a.N; i += 256) {
        uint32_t v = x[i];
        if (r) v = round_out<F16>(act_to_f32<F16>(v) + act_to_f32<F16>(r[i]));
        if (again) h[i] = (uint16_t)v;
        const float f = act_to_f32<F16>(v);
        sum = __builtin_fmaf(f, f, sum);
    }
    sum = lanes_sum(sum);
    if ((tid & 63) == 0) s_sum[tid >> 6] = sum;
    __syncthreads();
    sum = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
    const float inv = rsqrtf(sum / (float)a.N + a.eps);
    auto value = [&](int i) {
        uint32_t v = again ? h[i] : x[i];
        if (r && !again) v = round_out<F16>(act_to_f32<F16>(v) + act_to_f32<F16>(r[i]));
        return act_to_f32<F16>(v) * inv * act_to_f32<F16>(a.w[i]);
    };
    if constexpr (!F8) {
        uint16_t* y = static_cast<uint16_t*>(a.y) + t * a.ld_y;
        for (int i = tid; i < a.N; i += 256) y[i] = (uint16_t)round_out<F16>(fp32_value(value(i)));
    } else {
        uint32_t top = 0u;
        for (int i = tid; i < a.N; i += 256) {
            const uint32_t u = __float_as_uint(value(i)) & 0x7FFFFFFFu;
            top = u > top ? u : top;
        }
        top = lanes_max(top);
        if ((tid & 63) == 0) s_max[tid >> 6] = top;
        __syncthreads();
        for (int i = 0; i < 4; ++i) top = s_max[i] > top ? s_max[i] : top;
        const float scale = norm_row_scale(__uint_as_float(top));
        const float back = __fdiv_rn(1.0f, scale);
        if (tid == 0) a.scales[t] = scale;
        uint8_t* y = static_cast<uint8_t*>(a.y) + t * a.ld_y;
        for (int i = tid; i < a.N; i += 256) y[i] = (uint8_t)e4m3_byte(value(i) * back);
    }
}

}  // namespace nvfp4
