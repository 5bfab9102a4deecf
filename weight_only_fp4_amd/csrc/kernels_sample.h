// The next token of each row from its logits (nvfp4_sample): temperature,
// top-k, top-p, min-p and a draw by a given random number.
//
// With l the row's logits (NaN as -infinity) and m their maximum, the weights
// are whole numbers
//   q_i = rint(2^s exp((l_i - m) / t)),  s = min(45, 62 - ceil(log2 V)),
// the exponential in fp64, so that sums of them are exact and no order of
// atomics or lanes can change a result (a weight's rounding is 2^-46 of the
// largest, far below what a 32-bit random number can tell apart).  Tokens are
// ordered by (l descending, index ascending); each filter keeps a prefix of
// that order, so what is kept is a threshold (key, index):
//   top-k: the first k;
//   top-p: those with the sum of the weights before them < p * (sum of what top-k left);
//   min-p: those with exp(..) >= min_p, the largest always.
// The token is the first of the kept ones, in the vocabulary's order, whose
// cumulative weight exceeds u * (the kept ones' sum).
//
// Two launches.  k_sample_scan cuts the rows into slices and puts each slice's
// logits into bins of 1/16 in (m - l) / t, on a grid that all slices of a row
// share (floor(16 l / t)); 512 bins reach down to weights that round to 0.
// k_sample_pick, a workgroup a row, joins the slices' bins, which leaves one bin
// to look into, and draws:
//   rows with top-k, or with min-p and without top-p: the slices count their
//     bins and list what lies above their own k-th logit (or min_p of their own
//     maximum), a superset of what is kept; the lists' elements above the row's
//     bin are sorted and everything is done on them;
//   other rows: the slices add the weights of their bins; top-p's threshold is
//     in the bin where the row's sum passes p of the total, whose elements are
//     collected from the row and sorted; the draw picks a slice by its kept sum
//     and goes through that slice alone.
// Where a list is longer than its room (flat rows, many equal logits) the row
// takes sample_slow, which reads the row again for every step: a radix descent
// of 8 bits a round finds each threshold.
//
// What bounds it is no rate of the memory (64 x 131072 bf16 logits are 2.4 us)
// but the slices' fp64 exponentials (64 x 131072: 8 of 19 us, behind which the
// additions in LDS hide) and a chain of some twenty barriers a row.  Measured in a
// graph, scan + pick: 1 x 131072, top-k 50 20.3 us (7.2 + 13.4); 23 x 32003 fp32,
// min-p 23.5 (6.3 + 16.6); 64 x 131072, top-p 59.8 (19.4 + 41.6).  One workgroup a
// row in one launch took 250, 31, 370; rows that take sample_slow 210 to 430.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decode.h"

namespace nvfp4 {

constexpr int kSampleThreads = 1024;
constexpr int kSampleWaves = kSampleThreads / 64;
constexpr int kSampleCopies = 16;      // of the 256 digits' counters: lanes of a wave mostly hit few digits
constexpr int kSampleScanThreads = 512;
constexpr int kSampleBins = 512;
constexpr float kSamplePerUnit = 16.f; // bins a unit of (m - l) / t
constexpr int kSampleListed = 2048;    // elements a slice lists
constexpr int kSampleList = 4096;      // elements k_sample_pick sorts
constexpr int kSampleNarrow = 256;     // above which it narrows them down first
constexpr int kSampleMaxSlices = 64;
constexpr int kSampleHeld = 2;         // pieces that a thread of k_sample_scan holds

// What k_sample_scan leaves of a slice.
struct SampleSlice {
    float largest;                     // its largest logit (-infinity: none)
    float bin;                         // whose grid bin
    int32_t first;                     // rows that ask for the largest: its lowest index
    int32_t listed;                    // elements of the list (more than kSampleListed: it is cut off)
    uint64_t bins[kSampleBins];        // from that bin downwards: counts, or weights relative to the slice's largest
    uint64_t list[kSampleListed];      // (key << 32 | ~index)
};

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
    SampleSlice* slices;   // [B][S] workspace
    int S, slice;          // slices of a row, 16-byte pieces of one
    int slice_shift;       // 2^slice_shift: a slice's largest weight in its own sums
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
    int full0, full1;      // pieces that lie wholly in the row
    __device__ __forceinline__ SampleRow(const SampleArgs& a, int b) {
        const uint8_t* p = static_cast<const uint8_t*>(a.logits) + (int64_t)b * a.ld * Logit<DT>::kSize;
        const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15);
        base = p - off;
        skew = off / Logit<DT>::kSize;
        V = a.V;
        pieces = (skew + V + Logit<DT>::kPiece - 1) / Logit<DT>::kPiece;
        full0 = skew > 0 ? 1 : 0;
        full1 = (skew + V) / Logit<DT>::kPiece;
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

// Pieces c, c + step, .. below `end` as they lie in memory; places outside the
// row are NaN, which counts for nothing anywhere, as a logit that is NaN does.
// The loads are unconditional (from a whole piece of the row) and all in flight
// before the few that are cut by the row's ends are put right.
template <int DT, int N>
__device__ __forceinline__ void sample_load(const SampleRow<DT>& row, int c, int step, int end, uint4 (&v)[N]) {
    constexpr int P = Logit<DT>::kPiece;
    const bool any = row.full1 > row.full0;   // the same in all threads
    if (any) {
#pragma unroll
        for (int h = 0; h < N; ++h) {
            int at = c + h * step;
            at = at < row.full0 ? row.full0 : at >= row.full1 ? row.full1 - 1 : at;
            v[h] = *reinterpret_cast<const uint4*>(row.base + (int64_t)at * 16);
        }
    }
#pragma unroll
    for (int h = 0; h < N; ++h) {
        const int at = c + h * step;
        if (at >= row.full0 && at < row.full1 && at < end) continue;
        uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};
        if (at < end) {
            const uint8_t* p = row.base + (int64_t)at * 16;
            const int i0 = at * P - row.skew;
#pragma unroll
            for (int e = 0; e < P; ++e) {
                if (i0 + e < 0 || i0 + e >= row.V) continue;
                if (DT == kLogitF32) w[e & 3] = reinterpret_cast<const uint32_t*>(p)[e];
                else {
                    const uint32_t x = reinterpret_cast<const uint16_t*>(p)[e];
                    w[(e >> 1) & 3] = (e & 1) ? (w[(e >> 1) & 3] & 0xFFFFu) | x << 16 : (w[(e >> 1) & 3] & 0xFFFF0000u) | x;
                }
            }
        }
        v[h] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
// f(place e, value) of a loaded piece's logits (NaN among them).
template <int DT, typename F>
__device__ __forceinline__ void sample_values(const uint4& v, F&& f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < Logit<DT>::kPiece; ++e) {
        if (DT == kLogitF32) f(e, __uint_as_float(w[e & 3]));
        else f(e, act_to_f32<DT == kLogitF16>((e & 1) ? w[(e >> 1) & 3] >> 16 : w[(e >> 1) & 3] & 0xFFFFu));
    }
}

// The same of one 32-bit word of a piece, e of its first logit in the piece: the
// loops over words stay loops, because code that runs a few times only costs
// its fetch (eight logits unrolled in each pass: 64 x 131072 top-p 66 us, one
// user's 131072 logits without a filter 30; so 60 and 24).
template <int DT, typename F>
__device__ __forceinline__ void sample_word(uint32_t w, int e, F&& f) {
    if (DT == kLogitF32) f(e, __uint_as_float(w));
    else {
        f(e, act_to_f32<DT == kLogitF16>(w & 0xFFFFu));
        f(e + 1, act_to_f32<DT == kLogitF16>(w >> 16));
    }
}

__device__ __forceinline__ uint64_t shfl_xor_u64(uint64_t v, int m) {
    const uint32_t lo = __shfl_xor((uint32_t)v, m), hi = __shfl_xor((uint32_t)(v >> 32), m);
    return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t shfl_up_u64(uint64_t v, int d) {
    const uint32_t lo = __shfl_up((uint32_t)v, d), hi = __shfl_up((uint32_t)(v >> 32), d);
    return (uint64_t)hi << 32 | lo;
}

// 2^(x + shift) for x <= 0 in fp64: 2^n times the series of e^(f ln 2) up to its
// 11th power with n = rint(x), |f| <= 1/2 (the rest is below 2^-47).
__device__ __forceinline__ double sample_exp2(double x, int shift) {
    const double n = rint(x), f = x - n;
    double p = 4.4455382718708114976e-10;   // ln(2)^k / k!, k = 11 .. 1
    p = fma(p, f, 7.0549116208011233299e-09);
    p = fma(p, f, 1.0178086009239699728e-07);
    p = fma(p, f, 1.3215486790144309488e-06);
    p = fma(p, f, 1.5252733804059840280e-05);
    p = fma(p, f, 1.5403530393381609954e-04);
    p = fma(p, f, 1.3333558146428443423e-03);
    p = fma(p, f, 9.6181291076284771619e-03);
    p = fma(p, f, 5.5504108664821579953e-02);
    p = fma(p, f, 2.4022650695910071233e-01);
    p = fma(p, f, 6.9314718055994530942e-01);
    p = fma(p, f, 1.0);
    return ldexp(p, (int)n + shift);
}

// What weights go by: exp((l - m) / t) in units of 2^-shift.
struct SampleWeights {
    double top, per;    // m, log2(e) / t
    int shift;
    __device__ __forceinline__ SampleWeights(float largest, float t, int shift)
        : top((double)largest), per(1.44269504088896340736 / (double)t), shift(shift) {}
    // 2^up times the weight: 2^up for the maximum (an infinite one takes all), 0 for -infinity
    __device__ __forceinline__ double weight(float l, int up = 0) const {
        if ((double)l == top) return ldexp(1.0, up);
        const double x = ((double)l - top) * per;
        return x > -64.0 ? sample_exp2(x, up) : 0.0;   // also for NaN: an infinity's difference times 0
    }
    // rint(2^shift weight), shift < 52: what the addition of 2^52 leaves
    static __device__ __forceinline__ uint64_t rounded(double w) {
        return __double_as_longlong(w + 4503599627370496.0) - 0x4330000000000000ll;
    }
    __device__ __forceinline__ uint64_t units(float l) const { return rounded(weight(l, shift)); }
    __device__ __forceinline__ double unit() const { return ldexp(1.0, shift); }
    __device__ __forceinline__ float logprob(float l, double total) const {
        return (float)(((double)l == top ? 0.0 : ((double)l - top) * per * 0.693147180559945309417) - log(total));
    }
};

// Inclusive scan over the workgroup (threads in order); total in all.
template <typename T>
__device__ __forceinline__ T sample_scan(T v, uint64_t* sums, T& total) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    uint64_t x = (uint64_t)v;
#pragma unroll 1
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
    uint64_t digits[256 * kSampleCopies];   // counters or weights of the digits; of the row's steps in the draw; a list
    uint64_t second[kSampleList];
    uint64_t sums[kSampleWaves];
    uint64_t above;    // of the digits above the chosen one
    double fsums[kSampleWaves];
    double factor[kSampleMaxSlices];        // of the slices' sums: exp((their largest - m) / t)
    uint64_t kept[kSampleMaxSlices];        // the slices' kept units
    float largest[kSampleMaxSlices];
    float top;
    int below[kSampleMaxSlices];            // bins between the row's largest and theirs
    int digit;
    int found;
    int count;
    uint32_t low, high;
};
static_assert(kSampleScanThreads >= kSampleBins, "a bin a thread");
static_assert(256 * kSampleCopies == kSampleList, "the digits' room holds a list");

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
                const uint64_t n = COUNT ? 1 : sw.units(l);
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
    const uint64_t each = COUNT ? 1 : sw.units(sample_value(prefix));
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

// A row's settings, and which way it takes.
struct SampleSettings {
    float t, p, u;
    int k;            // 0: off
    double min_p;
    bool filters;     // min-p is on
    bool listing;     // lists, not sums
    __device__ __forceinline__ SampleSettings(const SampleArgs& a, int b) {
        t = a.temperature ? a.temperature[b] : 1.f;
        p = a.top_p ? a.top_p[b] : 1.f;
        u = a.u[b];
        k = a.top_k ? a.top_k[b] : 0;
        if (k < 0 || k >= a.V) k = 0;
        const float mp = a.min_p ? a.min_p[b] : 0.f;
        min_p = (double)mp;
        filters = mp > 0.f;   // not NaN
        listing = k > 0 || (filters && !(p < 1.f));
    }
    __device__ __forceinline__ bool keeps(double w) const { return !filters || w >= min_p || w == 1.0; }
    // The element where a cumulative sum first exceeds u * total (whole units, total >= 1).
    __device__ __forceinline__ uint64_t aim(uint64_t total) const {
        const double at = u > 0.f ? floor((double)u * (double)total) : 0.0;   // NaN: 0
        const uint64_t x = at < (double)total ? (uint64_t)at : total - 1;
        return x < total ? x : total - 1;
    }
};

// One row by one workgroup, everything from the row itself.  Out of line: few
// rows come here, and the others' registers and instruction fetches stay free
// of it.
template <int DT>
__device__ __noinline__ void sample_slow(SampleArgs a, int b, float largest, SampleShared& sh) {
    const int tid = threadIdx.x;
    const SampleRow<DT> row(a, b);
    const SampleSettings set(a, b);
    const SampleWeights sw(largest, set.t, a.shift);
    const float p = set.p;
    const int k = set.k;
    SampleCut cut = {0u, a.V};
    if (k > 0) cut = sample_descend<DT, true>(row, sw, cut, (uint64_t)k, sh);
    if (p < 1.f) {
        uint64_t sum = 0;
        for (int c = tid; c < row.pieces; c += kSampleThreads)
            row.piece(c, [&](int i, float l) {
                if (cut.holds(sample_key(l), i)) sum += sw.units(l);
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
        return set.keeps(sw.weight(l)) ? sw.units(l) : 0;
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
    const uint64_t aim = set.aim(total);   // the first cumulative sum > aim
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
                if (a.logprobs) a.logprobs[b] = sw.logprob(l, (double)total / sw.unit());
            }
        });
    }
}

// --------------------------------------------------------- slices and bins --

// Grid bin of a logit, as fp32: rises with it, equal for equal ones, NaN for NaN.
__device__ __forceinline__ float sample_grid(float t) { return fminf(kSamplePerUnit / t, 1e30f); }
__device__ __forceinline__ float sample_bin(float l, float grid) { return floorf(l * grid); }
// Whether the bins near the largest logit's are exact (products to a quarter of
// a bin) and finite; rows where they are not take sample_slow.
__device__ __forceinline__ bool sample_grid_holds(float largest, float grid) { return fabsf(largest) * grid < 4194304.f; }
// The same of a slice's largest, which may lie up to the bins' whole reach
// further from zero than that of a row that holds: every slice such a row counts
// has to have added its weights.  (Products are then off by a quarter of a bin
// at most, as sample_min_p_bins allows; a bin is one for all slices either way.)
__device__ __forceinline__ bool sample_grid_reaches(float largest, float grid) {
    return fabsf(largest) * grid < 4194304.f + 2 * kSampleBins;
}
// Bins below the largest that min-p may keep: one more for the grid's place, one for its rounding.
__device__ __forceinline__ int sample_min_p_bins(const SampleSettings& set) {
    if (!set.filters) return kSampleBins - 1;
    const double z = -log(set.min_p) * (double)kSamplePerUnit;
    return z < (double)(kSampleBins - 3) ? (z > 0.0 ? (int)z + 2 : 2) : kSampleBins - 1;
}
// Of a row that lists: top-p's total has the elements that min-p drops later.
__device__ __forceinline__ int sample_listed_bins(const SampleSettings& set) {
    return set.p < 1.f ? kSampleBins - 1 : sample_min_p_bins(set);
}

// Grid: (slices, rows).  A thread's pieces are kSampleScanThreads apart; a slice
// of up to 1024 is read once and stays in LDS.
template <int DT>
__global__ void __launch_bounds__(kSampleScanThreads) k_sample_scan(SampleArgs a) {
    constexpr int P = Logit<DT>::kPiece;
    __shared__ uint64_t s_bins[kSampleBins];
    __shared__ float s_largest[kSampleScanThreads / 64];
    __shared__ uint32_t s_wave[kSampleScanThreads / 64];
    __shared__ int s_listed, s_limit, s_first;
    const int tid = threadIdx.x, lane = tid & 63, s = blockIdx.x, b = blockIdx.y;
    const SampleRow<DT> row(a, b);
    const int c0 = s * a.slice, c1 = c0 + a.slice < row.pieces ? c0 + a.slice : row.pieces;
    constexpr int kAtOnce = kSampleHeld * kSampleScanThreads;
    __shared__ uint32_t s_held[kSampleHeld * 4][kSampleScanThreads];   // word by word; a thread reads what it wrote itself
    auto load = [&](int c) {
        uint4 v[kSampleHeld];
        sample_load<DT, kSampleHeld>(row, c + tid, kSampleScanThreads, c1, v);
#pragma unroll
        for (int h = 0; h < kSampleHeld; ++h) {
            s_held[4 * h][tid] = v[h].x;
            s_held[4 * h + 1][tid] = v[h].y;
            s_held[4 * h + 2][tid] = v[h].z;
            s_held[4 * h + 3][tid] = v[h].w;
        }
    };
    load(c0);
    const SampleSettings set(a, b);
    SampleSlice& out = a.slices[(int64_t)b * a.S + s];
    // f(index, value) of all the slice's logits
    auto all = [&](auto&& f) {
        for (int c = c0; c < c1; c += kAtOnce) {
            if (a.slice > kAtOnce) load(c);
#pragma unroll 1
            for (int j = 0; j < 4 * kSampleHeld; ++j)
                sample_word<DT>(s_held[j][tid], (c + tid + (j >> 2) * kSampleScanThreads) * P - row.skew + (j & 3) * (P / 4), f);
        }
    };
    for (int i = tid; i < kSampleBins; i += kSampleScanThreads) s_bins[i] = 0;
    if (tid == 0) {
        s_listed = 0;
        s_limit = kSampleBins - 1;
        s_first = 0x7FFFFFFF;
    }
    float largest = -__builtin_inff();
    all([&](int, float l) { largest = fmaxf(largest, l); });
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) largest = fmaxf(largest, __shfl_xor(largest, m));
    if (lane == 0) s_largest[tid >> 6] = largest;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSampleScanThreads / 64; ++w) largest = fmaxf(largest, s_largest[w]);
    const float grid = sample_grid(set.t), top = sample_bin(largest, grid);
    const bool none = largest == -__builtin_inff();
    if (!none && !(set.t > 0.f)) {   // the row asks for its largest
        int first = 0x7FFFFFFF;
        all([&](int i, float l) { first = l == largest && i < first ? i : first; });
        atomicMin(&s_first, first);
        __syncthreads();
    }
    if (tid == 0) {
        out.largest = largest;
        out.bin = top;
        out.first = s_first;
        out.listed = 0;
    }
    if (none || !(set.t > 0.f)) return;   // k_sample_pick does not read the rest
    if (set.listing) {
        all([&](int, float l) {
            const float d = top - sample_bin(l, grid);
            if (d < (float)kSampleBins) atomicAdd(reinterpret_cast<uint32_t*>(&s_bins[(int)d]), 1u);
        });
    } else if (sample_grid_reaches(largest, grid)) {   // the largest is finite: its weight comes out as 1 by itself
        const SampleWeights sw(largest, set.t, a.slice_shift);
        all([&](int, float l) {
            const float d = top - sample_bin(l, grid);
            if (d < (float)kSampleBins) {
                const uint64_t n = SampleWeights::rounded(sample_exp2(((double)l - sw.top) * sw.per, sw.shift));
                atomicAdd((unsigned long long*)&s_bins[(int)d], (unsigned long long)n);
            }
        });
    }
    __syncthreads();
    for (int i = tid; i < kSampleBins; i += kSampleScanThreads) out.bins[i] = s_bins[i];
    if (!set.listing) return;
    // down to the bin of the slice's own k-th
    int limit = sample_listed_bins(set);
    if (set.k > 0) {
        // a bin a thread, of the first kSampleBins
        const uint32_t n = tid < kSampleBins ? (uint32_t)s_bins[tid] : 0u, want = (uint32_t)set.k;
        uint32_t upto = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
        if (lane == 63) s_wave[tid >> 6] = upto;
        __syncthreads();
        for (int w = 0; w < (tid >> 6); ++w) upto += s_wave[w];
        if (tid < kSampleBins && upto >= want && upto - n < want) s_limit = tid;
        __syncthreads();
        limit = limit < s_limit ? limit : s_limit;
    }
    const float most = (float)limit;
    all([&](int i, float l) {
        if (top - sample_bin(l, grid) <= most) {
            const int at = atomicAdd(&s_listed, 1);
            if (at < kSampleListed) out.list[at] = (uint64_t)sample_key(l) << 32 | (uint32_t)~i;
        }
    });
    __syncthreads();
    if (tid == 0) out.listed = s_listed;
}

// Bitonic sort of list[0 .. n), n a power of two from 64 on, descending: the
// steps across up to 64 elements between a wave's lanes, the others in LDS.
__device__ __forceinline__ void sample_sort(uint64_t* list, int n) {
    // steps min(k / 2, 32) .. 1 of the merges k0 .. k1
    auto near = [&](int k0, int k1) {
        for (int i = threadIdx.x; i < n; i += kSampleThreads) {
            uint64_t x = list[i];
            for (int k = k0; k <= k1; k <<= 1)
                for (int j = k / 2 < 32 ? k / 2 : 32; j > 0; j >>= 1) {
                    const uint64_t y = shfl_xor_u64(x, j);
                    const bool larger = ((i & j) == 0) == ((i & k) == 0);
                    x = (x > y) == larger ? x : y;
                }
            list[i] = x;
        }
        __syncthreads();
    };
    __syncthreads();
    near(2, 64);
    for (int k = 128; k <= n; k <<= 1) {
        for (int j = k >> 1; j >= 64; j >>= 1) {
            for (int i = threadIdx.x; i < n / 2; i += kSampleThreads) {
                const int lo = ((i & ~(j - 1)) << 1) | (i & (j - 1)), hi = lo | j;
                const uint64_t x = list[lo], y = list[hi];
                if (((lo & k) == 0) == (x < y)) list[lo] = y, list[hi] = x;
            }
            __syncthreads();
        }
        near(k, k);
    }
}

// Inclusive scan of doubles over the workgroup, in a fixed order.
__device__ __forceinline__ double sample_scan_f64(double v, double* sums, double& total) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll 1
    for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    __syncthreads();
    if (lane == 63) sums[w] = v;
    __syncthreads();
    double before = 0.0;
    total = 0.0;
#pragma unroll
    for (int i = 0; i < kSampleWaves; ++i) {
        before += i < w ? sums[i] : 0.0;
        total += sums[i];
    }
    return before + v;
}

// The list's length as a power of two, its rest filled with zeros (no element is 0).
__device__ __forceinline__ int sample_fill(uint64_t* list, int n) {
    int size = 64;
    while (size < n) size <<= 1;
    for (int i = n + threadIdx.x; i < size; i += kSampleThreads) list[i] = 0;
    return size;
}

// Bin d of the row from the slices': f(slice, content), twenty loads in flight.
template <typename F>
__device__ __forceinline__ void sample_join(const SampleSlice* slices, int S, const SampleShared& sh, int d, F&& f) {
    for (int s0 = 0; s0 < S; s0 += 20) {
        uint64_t v[20];
#pragma unroll
        for (int i = 0; i < 20; ++i) {
            const int s = s0 + i < S ? s0 + i : S - 1, at = d - sh.below[s];
            v[i] = slices[s].bins[at > 0 ? at : 0];
        }
#pragma unroll
        for (int i = 0; i < 20; ++i)
            if (s0 + i < S && d >= sh.below[s0 + i]) f(s0 + i, v[i]);
    }
}

// Rows whose slices made lists; false: a list was too long.
template <int DT>
__device__ __forceinline__ bool sample_listed(const SampleArgs& a, int b, const SampleSettings& set, float largest, float top,
                                              SampleShared& sh) {
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const SampleSlice* slices = a.slices + (int64_t)b * a.S;
    const SampleWeights sw(largest, set.t, a.shift);
    const float grid = sample_grid(set.t);
    uint64_t* list = sh.digits;
    int limit = sample_listed_bins(set);
    if (tid == 0) {
        sh.count = 0;
        sh.digit = kSampleBins - 1;
    }
    if (set.k > 0) {   // the bin of the row's k-th
        uint64_t n = 0;
        if (tid < kSampleBins) sample_join(slices, a.S, sh, tid, [&](int, uint64_t v) { n += v; });
        uint64_t total;
        const uint64_t upto = sample_scan<uint64_t>(n, sh.sums, total), want = (uint64_t)set.k;
        if (tid < kSampleBins && upto >= want && upto - n < want) sh.digit = tid;
    }
    __syncthreads();
    limit = limit < sh.digit ? limit : sh.digit;
    const float most = (float)limit;
    for (int s = w; s < a.S; s += kSampleWaves) {
        if (sh.below[s] >= kSampleBins) continue;   // wholly below the bins, or nothing in it
        const int n = slices[s].listed;
        if (n > kSampleListed && lane == 0) atomicAdd(&sh.count, kSampleList + 1);
        for (int i = lane; i < n && i < kSampleListed; i += 64) {
            const uint64_t x = slices[s].list[i];
            if (!(top - sample_bin(sample_value((uint32_t)(x >> 32)), grid) <= most)) continue;
            const int at = atomicAdd(&sh.count, 1);
            if (at < kSampleList) list[at] = x;
        }
    }
    __syncthreads();
    const int n = sh.count;
    __syncthreads();
    if (n > kSampleList) return false;
    const int size = sample_fill(list, n);
    sample_sort(list, size);
    // a thread's elements are neighbours: i0 .. i1 (the loops stay loops: most
    // lists give a thread one, and code that runs once costs its fetch)
    const int each = (size + kSampleThreads - 1) / kSampleThreads;
    const int left = set.k > 0 && set.k < n ? set.k : n;   // after top-k
    auto units = [&](uint64_t key) { return sw.units(sample_value((uint32_t)key)); };
    int i0 = tid * each, i1 = i0 + each < left ? i0 + each : left;
    uint64_t sum = 0, total;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) sum += units(list[i] >> 32);
    uint64_t run = sample_scan<uint64_t>(sum, sh.sums, total) - sum;
    const double target = (double)set.p * (double)total;
    uint64_t kept = 0, all;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const float l = sample_value((uint32_t)(list[i] >> 32));
        if (i == 0 || ((!(set.p < 1.f) || (double)run < target) && set.keeps(sw.weight(l)))) ++kept;
        run += units(list[i] >> 32);
    }
    sample_scan<uint64_t>(kept, sh.sums, all);   // what is kept is a prefix: its length
    const int m = (int)all;
    // the kept ones by index (ascending: the complement descends), with their keys
    uint64_t* by_index = sh.second;
    for (int i = tid; i < m; i += kSampleThreads) by_index[i] = list[i] << 32 | list[i] >> 32;   // (~index, key)
    sample_sort(by_index, sample_fill(by_index, m));
    sum = 0;
    i1 = i0 + each < m ? i0 + each : m;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) sum += units(by_index[i]);
    const uint64_t end = sample_scan<uint64_t>(sum, sh.sums, total);
    run = end - sum;
    const uint64_t aim = set.aim(total);
    if (end > aim && run <= aim) {
        int i = i0;
#pragma unroll 1
        while ((run += units(by_index[i])) <= aim) ++i;
        a.tokens[b] = (int)~(uint32_t)(by_index[i] >> 32);
        if (a.logprobs) a.logprobs[b] = sw.logprob(sample_value((uint32_t)by_index[i]), (double)total / sw.unit());
    }
    return true;
}

// The least fp32 value whose bin is at least `bin`: bins rise with values, so
// a binary search of the keys, next to the quotient if it is there.
__device__ __forceinline__ float sample_bin_begin(float bin, float grid) {
    uint32_t lo = kSampleNone, hi = 0xFF800000u;   // the keys of the infinities
    const uint32_t near = sample_key(bin / grid);
    if (near > lo + 4 && near < hi - 4 && sample_bin(sample_value(near - 4), grid) < bin &&
        sample_bin(sample_value(near + 4), grid) >= bin) {
        lo = near - 3;
        hi = near + 4;
    }
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (sample_bin(sample_value(mid), grid) >= bin) hi = mid;
        else lo = mid + 1;
    }
    return sample_value(lo);
}

// Rows whose slices added weights; false: the bin was too full.  A slice's
// weights are whole numbers relative to its own largest, 2^slice_shift, which
// the row counts times its factor.
template <int DT>
__device__ __forceinline__ bool sample_summed(const SampleArgs& a, int b, const SampleSettings& set, float largest, float top,
                                              SampleShared& sh) {
    constexpr int P = Logit<DT>::kPiece;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const SampleSlice* slices = a.slices + (int64_t)b * a.S;
    const SampleRow<DT> row(a, b);
    const SampleWeights sw(largest, set.t, a.shift);
    const float grid = sample_grid(set.t);
    const double unit = ldexp(1.0, -a.slice_shift);
    uint64_t* list = sh.digits;
    // a slice's units of l, as its bins have them
    auto units_in = [&](int s, float l) {
        return SampleWeights::rounded(sample_exp2(((double)l - (double)sh.largest[s]) * sw.per, a.slice_shift));
    };
    const int per_slice = a.slice * P;
    auto slice_of = [&](uint64_t x) { return ((int)~(uint32_t)x + row.skew) / per_slice; };
    if (tid == 0) {
        sh.count = 0;
        sh.digit = kSampleBins - 1;
        sh.found = 0;
    }
    if (tid < kSampleMaxSlices) sh.kept[tid] = 0;
    double n = 0.0, total;
    if (tid < kSampleBins) sample_join(slices, a.S, sh, tid, [&](int s, uint64_t v) { n += (double)v * unit * sh.factor[s]; });
    const double upto = sample_scan_f64(n, sh.fsums, total);
    // bins above `lo` are kept, those below `hi` dropped; what is between is looked at
    int lo = kSampleBins, hi = kSampleBins;
    const double target = (double)set.p * total;
    if (set.p < 1.f) {
        // the first bin whose end reaches the target: the scan's sums rise with the bins
        int first = tid < kSampleBins && upto >= target ? tid : kSampleBins - 1;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int o = __shfl_xor(first, m);
            first = o < first ? o : first;
        }
        if (lane == 0) atomicMin(&sh.digit, first);
        __syncthreads();
        lo = hi = sh.digit;
    }
    if (set.filters) {
        const int bins = sample_min_p_bins(set);
        hi = hi < bins ? hi : bins;
        lo = lo < bins - 3 ? lo : (bins > 3 ? bins - 3 : 0);
    }
    __syncthreads();
    double above = 0.0;
    if (lo < kSampleBins) {
        if (tid == lo) sh.fsums[0] = upto - n;
        // the values between: whole pieces are tested by two comparisons a logit, four loads in flight
        const float from = sample_bin_begin(top - (float)hi, grid), to = sample_bin_begin(top - (float)lo + 1.f, grid);
        for (int c = tid; c < row.pieces; c += 4 * kSampleThreads) {
            uint4 v[4];
            sample_load<DT, 4>(row, c, kSampleThreads, row.pieces, v);
            uint32_t hits = 0;   // bit h P + e: place e of piece h
#pragma unroll
            for (int h = 0; h < 4; ++h)
                sample_values<DT>(v[h], [&](int e, float l) { hits |= (l >= from && l < to ? 1u : 0u) << (h * P + e); });
            if (hits == 0) continue;
            int at = atomicAdd(&sh.count, __popc(hits));
            do {   // their places: few, so that the values are read again below
                const int bit = __builtin_ctz(hits);
                hits &= hits - 1;
                if (at < kSampleList) list[at] = (uint32_t)((c + bit / P * kSampleThreads) * P + bit % P);
                ++at;
            } while (hits);
        }
        __syncthreads();
        above = sh.fsums[0];
    }
    int count = sh.count;
    if (count > kSampleList) return false;
    for (int i = tid; i < count; i += kSampleThreads) {   // place -> (key, index)
        const int place = (int)list[i];
        const uint8_t* p = row.base + (int64_t)place * Logit<DT>::kSize;
        const uint32_t bits = DT == kLogitF32 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
        list[i] = (uint64_t)sample_key(Logit<DT>::value(bits)) << 32 | (uint32_t)~(place - row.skew);
    }
    __syncthreads();
    SampleCut cut = {0u, -1};   // the list's last kept element, if any
    if (lo < kSampleBins) {
        // in units of the row: what is missing to the target above the list
        double rest = set.p < 1.f ? (target - above) * sw.unit() : 9e18;
        // A long list is first cut down to the part, of 1024 of its keys' range,
        // in which its sum reaches the target: those above are kept.
        if (!set.filters && count > kSampleNarrow) {
            uint32_t low = ~0u, high = 0;
            for (int i = tid; i < count; i += kSampleThreads) {
                const uint32_t k = (uint32_t)(list[i] >> 32);
                low = k < low ? k : low;
                high = k > high ? k : high;
            }
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const uint32_t x = __shfl_xor(low, m), y = __shfl_xor(high, m);
                low = x < low ? x : low;
                high = y > high ? y : high;
            }
            if (tid == 0) {
                sh.low = ~0u;
                sh.high = 0;
                sh.count = 0;
            }
            uint64_t* parts = sh.second;
            parts[tid] = 0;
            __syncthreads();
            if (lane == 0) {
                atomicMin(&sh.low, low);
                atomicMax(&sh.high, high);
            }
            __syncthreads();
            low = sh.low;
            high = sh.high;
            const int shift = 32 - __clz((int)((high - low) >> 10));   // the range is below 2^(10 + shift)
            auto part = [&](uint64_t x) { return (int)((high - (uint32_t)(x >> 32)) >> shift); };
            if (tid == 0) sh.digit = part((uint64_t)low << 32);
#pragma unroll 1
            for (int i = tid; i < count; i += kSampleThreads)
                atomicAdd((unsigned long long*)&parts[part(list[i])],
                          (unsigned long long)sw.units(sample_value((uint32_t)(list[i] >> 32))));
            __syncthreads();
            uint64_t all;
            const uint64_t q = parts[tid], end = sample_scan<uint64_t>(q, sh.sums, all);
            int first = (double)end >= rest ? tid : kSampleThreads;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const int o = __shfl_xor(first, m);
                first = o < first ? o : first;
            }
            if (lane == 0) atomicMin(&sh.digit, first);
            __syncthreads();
            const int chosen = sh.digit;
            if (tid == chosen) sh.above = end - q;
            __syncthreads();
            rest -= (double)sh.above;
#pragma unroll 1
            for (int i = tid; i < count; i += kSampleThreads) {
                const uint64_t x = list[i];
                const int at = part(x);
                if (at == chosen) {
                    sh.second[atomicAdd(&sh.count, 1)] = x;
                } else if (at < chosen) {
                    const int of = slice_of(x);
                    atomicAdd((unsigned long long*)&sh.kept[of],
                              (unsigned long long)units_in(of, sample_value((uint32_t)(x >> 32))));
                }
            }
            if (chosen > 0) cut = SampleCut{high - ((uint32_t)chosen << shift) + 1u, a.V};
            __syncthreads();
            count = sh.count;
            list = sh.second;
        }
        const int size = sample_fill(list, count);
        sample_sort(list, size);
        const int each = (size + kSampleThreads - 1) / kSampleThreads;
        const int i0 = tid * each, i1 = i0 + each < count ? i0 + each : count;
        uint64_t sum = 0, all;
#pragma unroll 1
        for (int i = i0; i < i1; ++i) sum += sw.units(sample_value((uint32_t)(list[i] >> 32)));
        uint64_t run = sample_scan<uint64_t>(sum, sh.sums, all) - sum;
        int kept = 0;
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
            const float l = sample_value((uint32_t)(list[i] >> 32));
            // the first of all always
            if ((lo == 0 && l == largest && i == 0) || ((double)run < rest && set.keeps(sw.weight(l)))) {
                kept = i + 1;
                const int of = slice_of(list[i]);
                atomicAdd((unsigned long long*)&sh.kept[of], (unsigned long long)units_in(of, l));   // whole: in any order
            }
            run += sw.units(l);
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int o = __shfl_xor(kept, m);
            kept = o > kept ? o : kept;
        }
        if (lane == 0) atomicMax(&sh.found, kept);
        __syncthreads();
        kept = sh.found;
        if (kept > 0) cut = SampleCut{(uint32_t)(list[kept - 1] >> 32), (int)~(uint32_t)list[kept - 1]};
    }
    // kept: what is in a bin above lo, and what the cut holds
    auto keeps = [&](int i, float l) {
        const float d = top - sample_bin(l, grid);
        return d < (float)lo || (d < (float)kSampleBins && cut.index >= 0 && cut.holds(sample_key(l), i));
    };
    // the slices' kept sums: their bins above lo, and what they have in the list
    for (int s = w; s < a.S; s += kSampleWaves) {
        const int end = lo - sh.below[s];   // of its own bins
        uint64_t v[kSampleBins / 64], x = 0;
#pragma unroll
        for (int i = 0; i < kSampleBins / 64; ++i) v[i] = slices[s].bins[64 * i + lane];
#pragma unroll
        for (int i = 0; i < kSampleBins / 64; ++i) x += 64 * i + lane < end ? v[i] : 0;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) x += shfl_xor_u64(x, m);
        if (lane == 0) sh.kept[s] += x;
    }
    __syncthreads();
    double kept_total = 0.0;
    for (int s = 0; s < a.S; ++s) kept_total += (double)sh.kept[s] * unit * sh.factor[s];
    const double aim = set.u > 0.f ? (set.u < 1.f ? (double)set.u : 1.0) * kept_total : 0.0;
    // the slice; past the last one by u >= 1 or a rounding: the last with anything in it
    int s = -1, some = 0;
    double before = 0.0, run = 0.0;
    for (int i = 0; i < a.S; ++i) {
        const double x = (double)sh.kept[i] * unit * sh.factor[i];
        if (x > 0.0) some = i;
        if (s < 0 && run + x > aim) {
            s = i;
            before = run;
        }
        run += x;
    }
    const bool past = s < 0;
    if (past) s = some;
    // the first whose cumulative sum exceeds aim, in the slice's whole units; its last if the roundings leave none
    const uint64_t in_slice = sh.kept[s];
    double x = past ? 9e18 : (aim - before) / (unit * sh.factor[s]);
    x = x > 0.0 ? floor(x) : 0.0;
    uint64_t want = x < (double)in_slice ? (uint64_t)x : in_slice - 1;
    want = want < in_slice ? want : in_slice - 1;
    const int c0 = s * a.slice, c1 = c0 + a.slice < row.pieces ? c0 + a.slice : row.pieces;
    uint64_t upto_here = 0;
    for (int c = c0; c < c1; c += kSampleThreads) {
        uint4 loaded[1];
        sample_load<DT, 1>(row, c + tid, 0, c1, loaded);
        uint32_t* words = reinterpret_cast<uint32_t*>(sh.second);   // word by word; a thread reads what it wrote itself
        words[tid] = loaded[0].x;
        words[kSampleThreads + tid] = loaded[0].y;
        words[2 * kSampleThreads + tid] = loaded[0].z;
        words[3 * kSampleThreads + tid] = loaded[0].w;
        const int i0 = (c + tid) * P - row.skew;
        uint64_t mine = 0, step;
#pragma unroll 1
        for (int j = 0; j < 4; ++j)
            sample_word<DT>(words[j * kSampleThreads + tid], i0 + j * (P / 4), [&](int i, float l) {
                if (keeps(i, l)) mine += units_in(s, l);
            });
        const uint64_t end = upto_here + sample_scan<uint64_t>(mine, sh.sums, step);
        if (end > want && end - mine <= want) {
            uint64_t at = end - mine;
            bool done = false;
#pragma unroll 1
            for (int j = 0; j < 4; ++j)
                sample_word<DT>(words[j * kSampleThreads + tid], i0 + j * (P / 4), [&](int i, float l) {
                    if (done || !keeps(i, l)) return;
                    at += units_in(s, l);
                    if (at > want) {
                        done = true;
                        a.tokens[b] = i;
                        if (a.logprobs) a.logprobs[b] = sw.logprob(l, kept_total);
                    }
                });
        }
        upto_here += step;
        if (upto_here > want) break;   // the same in every thread
    }
    return true;
}

// Grid: rows.
template <int DT>
__global__ void __launch_bounds__(kSampleThreads) k_sample_pick(SampleArgs a) {
    __shared__ SampleShared sh;
    const int tid = threadIdx.x, b = blockIdx.x;
    const SampleSettings set(a, b);
    const SampleSlice* slices = a.slices + (int64_t)b * a.S;
    float mine = -__builtin_inff(), bin = 0.f;
    if (tid < 64) {   // S <= 64
        int first = 0x7FFFFFFF;
        if (tid < a.S) {
            mine = slices[tid].largest;
            bin = slices[tid].bin;
            first = slices[tid].first;
        }
        float largest = mine;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) largest = fmaxf(largest, __shfl_xor(largest, m));
        first = mine == largest ? first : 0x7FFFFFFF;   // read where the row asks for its largest
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int o = __shfl_xor(first, m);
            first = o < first ? o : first;
        }
        if (tid == 0) {
            sh.top = largest;
            sh.found = first;
        }
    }
    __syncthreads();
    const float largest = sh.top;
    if (largest == -__builtin_inff() || !(set.t > 0.f)) {   // nothing to choose from, or the largest is asked for
        if (tid == 0) {
            a.tokens[b] = largest == -__builtin_inff() ? -1 : sh.found;
            if (a.logprobs) a.logprobs[b] = largest == -__builtin_inff() ? largest : 0.f;
        }
        return;
    }
    const float grid = sample_grid(set.t), top = sample_bin(largest, grid);
    const SampleWeights sw(largest, set.t, a.shift);
    if (tid < a.S) {
        const float below = top - bin;   // NaN and infinity: nothing in it
        const bool near = mine > -__builtin_inff() && below < (float)kSampleBins;
        sh.largest[tid] = mine;
        sh.below[tid] = near ? (int)below : kSampleBins;
        sh.factor[tid] = near ? sw.weight(mine) : 0.0;
    }
    __syncthreads();
    bool done = false;
    if (sample_grid_holds(largest, grid))
        done = set.listing ? sample_listed<DT>(a, b, set, largest, top, sh) : sample_summed<DT>(a, b, set, largest, top, sh);
    if (done) return;
    __syncthreads();
    sample_slow<DT>(a, b, largest, sh);
}

}  // namespace nvfp4
