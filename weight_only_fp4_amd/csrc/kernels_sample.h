// The next token of each row from its logits (nvfp4_sample): temperature,
// top-k, top-p, min-p and a draw by a given random number.
//
// With l the row's logits (NaN as -infinity) and m their maximum, the weights
// are whole numbers
//   q_i = rint(2^s exp((l_i - m) / t)),  s = min(52, 62 - ceil(log2 V)),
// the exponential in fp64, so that every sum of them is exact and no order of
// atomics or lanes can change a result (a weight's rounding is 2^-46 of the
// largest with 131072 logits, far below what a 32-bit random number can tell
// apart).  Tokens are ordered by (l descending, index ascending); each filter
// keeps a prefix of that order, so what is kept is a threshold (key, index):
//   top-k: the first k;
//   top-p: those with the sum of the weights before them < p * (sum of what top-k left);
//   min-p: those with exp(..) >= min_p.
// The token is the first of the kept ones, in the vocabulary's order, whose
// cumulative weight exceeds u * (the kept ones' sum).
//
// k_sample_row: a workgroup a row, which reads the row again for every step: a
// radix descent of 8 bits a round finds each threshold, counting elements
// (top-k) or adding weights (top-p) in LDS.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decode.h"

namespace nvfp4 {

constexpr int kSampleThreads = 1024;
constexpr int kSampleWaves = kSampleThreads / 64;
constexpr int kSampleCopies = 16;      // of the 256 digits' counters: lanes of a wave mostly hit few digits
constexpr int kSampleMaxBlocks = 4096; // steps of kSampleThreads pieces a row may have

struct SampleArgs {
    const void* logits;
    int64_t ld;
    const float* u;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* tokens;
    float* logprobs;
    int B, V;
    int shift;   // s
};

enum { kLogitBf16 = 0, kLogitF16 = 1, kLogitF32 = 2 };

template <int DT>
struct Logit {
    static constexpr int kSize = DT == kLogitF32 ? 4 : 2;
    static constexpr int kPiece = 16 / kSize;   // logits of a 16-byte piece
    static __device__ __forceinline__ float value(uint32_t bits) {
        const float f = DT == kLogitF32 ? __uint_as_float(bits) : act_to_f32<DT == kLogitF16>(bits);
        return f != f ? -__builtin_inff() : f;
    }
};

// Ordered key of a value: a > b exactly when key(a) > key(b); both zeros have one key.
__device__ __forceinline__ uint32_t sample_key(float f) {
    const uint32_t b = __float_as_uint(f == 0.f ? 0.f : f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float sample_value(uint32_t key) {
    return __uint_as_float((key >> 31) ? key & 0x7FFFFFFFu : ~key);
}
constexpr uint32_t kSampleNone = 0x007FFFFFu;   // the key of -infinity

// A row as 16-byte pieces on its own alignment: logit i of the row is place i +
// skew of pieces that start 16-byte aligned, and places outside [skew, skew + V)
// are not read.  f(index, value) for each logit of the piece.
template <int DT>
struct SampleRow {
    const uint8_t* base;   // the first piece, aligned down
    int skew, V, pieces;
    __device__ __forceinline__ SampleRow(const SampleArgs& a, int b) {
        const uint8_t* p = static_cast<const uint8_t*>(a.logits) + (int64_t)b * a.ld * Logit<DT>::kSize;
        const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15);
        base = p - off;
        skew = off / Logit<DT>::kSize;
        V = a.V;
        pieces = (skew + V + Logit<DT>::kPiece - 1) / Logit<DT>::kPiece;
    }
    template <typename F>
    __device__ __forceinline__ void piece(int c, F&& f) const {
        constexpr int P = Logit<DT>::kPiece;
        const int i0 = c * P - skew;
        const uint8_t* p = base + (int64_t)c * 16;
        if (i0 >= 0 && i0 + P <= V) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const uint32_t bits = DT == kLogitF32 ? w[e & 3] : (e & 1) ? w[(e >> 1) & 3] >> 16 : w[(e >> 1) & 3] & 0xFFFFu;
                f(i0 + e, Logit<DT>::value(bits));
            }
            return;
        }
        for (int e = 0; e < P; ++e) {
            if (i0 + e < 0 || i0 + e >= V) continue;
            const uint32_t bits = DT == kLogitF32 ? reinterpret_cast<const uint32_t*>(p)[e] : reinterpret_cast<const uint16_t*>(p)[e];
            f(i0 + e, Logit<DT>::value(bits));
        }
    }
};

__device__ __forceinline__ uint64_t shfl_xor_u64(uint64_t v, int m) {
    const uint32_t lo = __shfl_xor((uint32_t)v, m), hi = __shfl_xor((uint32_t)(v >> 32), m);
    return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t shfl_up_u64(uint64_t v, int d) {
    const uint32_t lo = __shfl_up((uint32_t)v, d), hi = __shfl_up((uint32_t)(v >> 32), d);
    return (uint64_t)hi << 32 | lo;
}

// What a row's filters and draw go by.
struct SampleWeights {
    double top, per;    // m, 1 / t
    double unit;        // 2^s
    double min_p;
    // exp((l - m) / t): 1 for the maximum (an infinite one takes all), 0 for -infinity
    __device__ __forceinline__ double weight(float l) const {
        if ((double)l == top) return 1.0;
        if (l == -__builtin_inff() || top == __builtin_inf()) return 0.0;
        return exp(((double)l - top) * per);
    }
    __device__ __forceinline__ uint64_t units(double w) const { return (uint64_t)rint(w * unit); }
};

// Inclusive scan over the workgroup (threads in order); total in all.
template <typename T>
__device__ __forceinline__ T sample_scan(T v, uint64_t* sums, T& total) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    uint64_t x = (uint64_t)v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t o = shfl_up_u64(x, d);
        if (lane >= d) x += o;
    }
    __syncthreads();   // sums of the scan before have been read
    if (lane == 63) sums[w] = x;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kSampleWaves; ++i) {
        before += i < w ? sums[i] : 0;
        all += sums[i];
    }
    total = (T)all;
    return (T)(before + x);
}

// Everything up to and including (key, index) in the row's order.
struct SampleCut {
    uint32_t key;
    int index;
    __device__ __forceinline__ bool holds(uint32_t k, int i) const { return k > key || (k == key && i <= index); }
};

struct SampleShared {
    uint64_t digits[256 * kSampleCopies];   // counters or weights of the digits; of the row's steps in the draw
    uint64_t sums[kSampleWaves];
    uint64_t best;
    uint64_t above;    // of the digits above the chosen one
    uint64_t all;
    int digit;
    int found;
};

// The element of the cut's elements that the row's order reaches at `target`:
// the first with the sum of (count or weight) up to and including itself >=
// target (1 <= target <= the sum over all).  COUNT: elements count 1 each.
// Equal keys go by index.
template <int DT, bool COUNT>
__device__ SampleCut sample_descend(const SampleRow<DT>& row, const SampleWeights& sw, SampleCut cut, uint64_t target,
                                    SampleShared& sh) {
    const int tid = threadIdx.x;
    uint32_t prefix = 0;
    uint64_t above = 0;   // of keys above the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256 * kSampleCopies; i += kSampleThreads) sh.digits[i] = 0;
        __syncthreads();
        for (int c = tid; c < row.pieces; c += kSampleThreads)
            row.piece(c, [&](int i, float l) {
                const uint32_t k = sample_key(l);
                if (shift < 24 && (k >> (shift + 8)) != (prefix >> (shift + 8))) return;
                if (!cut.holds(k, i)) return;
                const uint64_t n = COUNT ? 1 : sw.units(sw.weight(l));
                if (n) atomicAdd((unsigned long long*)&sh.digits[((k >> shift) & 255u) * kSampleCopies + (tid & (kSampleCopies - 1))],
                                 (unsigned long long)n);
            });
        __syncthreads();
        // thread d < 256: digit 255 - d, in descending order
        uint64_t mine = 0;
        if (tid < 256)
            for (int i = 0; i < kSampleCopies; ++i) mine += sh.digits[(255 - tid) * kSampleCopies + i];
        uint64_t total;
        const uint64_t upto = above + sample_scan<uint64_t>(mine, sh.sums, total);
        if (tid < 256 && upto - mine < target && target <= upto) {
            sh.digit = 255 - tid;
            sh.above = upto - mine;
        }
        __syncthreads();
        prefix |= (uint32_t)sh.digit << shift;
        above = sh.above;
        __syncthreads();
    }
    // of the elements with that key, the first ceil((target - above) / each) by index
    const uint64_t each = COUNT ? 1 : sw.units(sw.weight(sample_value(prefix)));
    const uint64_t want = (target - above + each - 1) / each;
    uint64_t before = 0;
    for (int c0 = 0; c0 < row.pieces; c0 += kSampleThreads) {
        uint64_t n = 0;
        if (c0 + tid < row.pieces)
            row.piece(c0 + tid, [&](int i, float l) { n += sample_key(l) == prefix && cut.holds(prefix, i); });
        uint64_t total;
        const uint64_t upto = before + sample_scan<uint64_t>(n, sh.sums, total);
        if (upto >= want && upto - n < want) {
            uint64_t left = want - (upto - n);
            row.piece(c0 + tid, [&](int i, float l) {
                if (sample_key(l) == prefix && cut.holds(prefix, i) && --left == 0) sh.found = i;
            });
        }
        before += total;
        if (before >= want) break;   // total is the same in every thread
    }
    __syncthreads();
    const SampleCut got = {prefix, sh.found};
    __syncthreads();
    return got;
}

template <int DT>
__global__ void __launch_bounds__(kSampleThreads) k_sample_row(SampleArgs a) {
    __shared__ SampleShared sh;
    const int tid = threadIdx.x, b = blockIdx.x;
    const SampleRow<DT> row(a, b);
    if (tid == 0) {
        sh.best = 0;
        sh.all = 0;
    }
    __syncthreads();
    // the largest logit, of equal ones the lowest index
    uint64_t best = 0;
    for (int c = tid; c < row.pieces; c += kSampleThreads)
        row.piece(c, [&](int i, float l) {
            const uint64_t x = (uint64_t)sample_key(l) << 32 | (uint32_t)~i;
            best = x > best ? x : best;
        });
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint64_t o = shfl_xor_u64(best, m);
        best = o > best ? o : best;
    }
    if ((tid & 63) == 0) atomicMax((unsigned long long*)&sh.best, (unsigned long long)best);
    __syncthreads();
    best = sh.best;
    const uint32_t top = (uint32_t)(best >> 32);
    const float t = a.temperature ? a.temperature[b] : 1.f;
    if (top == kSampleNone || !(t > 0.f)) {   // nothing to choose from, or the largest is asked for
        if (tid == 0) {
            a.tokens[b] = top == kSampleNone ? -1 : (int)~(uint32_t)best;
            if (a.logprobs) a.logprobs[b] = top == kSampleNone ? -__builtin_inff() : 0.f;
        }
        return;
    }
    SampleWeights sw;
    sw.top = (double)sample_value(top);
    sw.per = 1.0 / (double)t;
    sw.unit = ldexp(1.0, a.shift);
    sw.min_p = a.min_p ? (double)a.min_p[b] : 0.0;
    SampleCut cut = {0u, a.V};
    const int k = a.top_k ? a.top_k[b] : 0;
    if (k > 0 && k < a.V) cut = sample_descend<DT, true>(row, sw, cut, (uint64_t)k, sh);
    const float p = a.top_p ? a.top_p[b] : 1.f;
    if (p < 1.f) {
        uint64_t sum = 0;
        for (int c = tid; c < row.pieces; c += kSampleThreads)
            row.piece(c, [&](int i, float l) {
                if (cut.holds(sample_key(l), i)) sum += sw.units(sw.weight(l));
            });
        uint64_t total;
        sample_scan<uint64_t>(sum, sh.sums, total);
        // kept: what comes before is < p * total; at least the first
        double target = (double)p * (double)total;
        target = target < 1.0 ? 1.0 : ceil(target);
        const uint64_t whole = target < (double)total ? (uint64_t)target : total;
        cut = sample_descend<DT, false>(row, sw, cut, whole, sh);
    }
    // the kept weight, by steps of the row
    const int steps = (row.pieces + kSampleThreads - 1) / kSampleThreads;
    auto kept = [&](int i, float l) -> uint64_t {
        if (!cut.holds(sample_key(l), i)) return 0;
        const double w = sw.weight(l);
        return !(w < sw.min_p) || w == 1.0 ? sw.units(w) : 0;   // the largest stay whatever min_p is
    };
    for (int i = tid; i < steps; i += kSampleThreads) sh.digits[i] = 0;
    __syncthreads();
    for (int s = 0; s < steps; ++s) {
        uint64_t n = 0;
        const int c = s * kSampleThreads + tid;
        if (c < row.pieces) row.piece(c, [&](int i, float l) { n += kept(i, l); });
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) n += shfl_xor_u64(n, m);
        if ((tid & 63) == 0 && n) atomicAdd((unsigned long long*)&sh.digits[s], (unsigned long long)n);
    }
    __syncthreads();
    // the step, the piece and the element where the cumulative weight passes u * total
    uint64_t total = 0;
    for (int s = 0; s < steps; ++s) total += sh.digits[s];
    const float u = a.u[b];
    double at = u > 0.f ? floor((double)u * (double)total) : 0.0;   // NaN: 0
    uint64_t aim = at < (double)total ? (uint64_t)at : total - 1;   // the first cumulative sum > aim
    if (aim >= total) aim = total - 1;
    int s = 0;
    uint64_t before = 0;
    while (before + sh.digits[s] <= aim) before += sh.digits[s++];
    const int c = s * kSampleThreads + tid;
    uint64_t n = 0;
    if (c < row.pieces) row.piece(c, [&](int i, float l) { n += kept(i, l); });
    uint64_t step;
    const uint64_t upto = before + sample_scan<uint64_t>(n, sh.sums, step);
    if (upto > aim && upto - n <= aim) {
        uint64_t run = upto - n;
        bool done = false;
        row.piece(c, [&](int i, float l) {
            const uint64_t q = kept(i, l);
            run += q;
            if (!done && run > aim) {
                done = true;
                a.tokens[b] = i;
                if (a.logprobs) a.logprobs[b] = (float)(((double)l == sw.top ? 0.0 : ((double)l - sw.top) * sw.per) + log(sw.unit / (double)total));
            }
        });
    }
}

}  // namespace nvfp4
