// C ABI of the attention half of a decoder layer (include/nvfp4_w4a16.h):
// argument checks, kernel choice and launches.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/nvfp4_w4a16.h"
#include "attn_plan.h"
#include "kernels_kv.h"
#include "kernels_norm.h"
#include "plan.h"

using namespace nvfp4;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kBig = (int64_t)1 << 40;   // strides and row counts stay below: products fit 64 bits

// A launch holds fewer than 2^32 threads.
nvfp4_status check_launch(const char* fn, int64_t workgroups, int64_t threads) {
    if (workgroups * threads >= (int64_t)1 << 32)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: %lld rows of work are too many for one call", fn, (long long)workgroups);
    return NVFP4_OK;
}

// ---------------------------------------------------------------- the norm --

template <bool F16, bool F8>
void launch_norm(const NormArgs& a, bool vec, hipStream_t st) {
    const dim3 grid((unsigned)a.T);
    if (!vec) {
        hipLaunchKernelGGL((k_rms_norm_any<F16, F8>), grid, dim3(256), 0, st, a);
        return;
    }
    // Rows of up to 256 values (heads): 16 or 32 lanes a row, several rows a
    // workgroup (60000 x 128: 18.3 us with a wave each, 11.6 so; from 512 values
    // on a wave each is faster, 20000 x 512 13.1 us against 14.2).  Figures here
    // are of calls in a graph.
    const int pieces = a.N / 8;
    if (pieces <= 16) {
        hipLaunchKernelGGL((k_rms_norm_short<F16, F8, 16>), dim3((unsigned)((a.T + 15) / 16)), dim3(256), 0, st, a);
        return;
    }
    if (pieces <= 32) {
        hipLaunchKernelGGL((k_rms_norm_short<F16, F8, 32>), dim3((unsigned)((a.T + 7) / 8)), dim3(256), 0, st, a);
        return;
    }
    // Longer ones: a workgroup a row, one piece a thread while the rows leave
    // compute units free (a row's latency counts: 1 x 4096 3.2 us against 3.5
    // with two pieces, 64 x 2048 2.9 and 3.1), two from there on (half the waves
    // to start for the same loads in flight: 777 x 5120 to 8 bits 9.5 -> 8.7 us,
    // 8192 x 5120 62 -> 50), four where a row needs them.  Calls that move more
    // than the 256 MB Infinity Cache holds read past it (8192 x 5120, 16 bits:
    // 60 -> 55 us; 2048 x 4096, whose 67 MB it does hold, would take 14.5 for 11.4).
    const int V = pieces > 2048 ? 4 : (pieces > 1024 || a.T >= 256 ? 2 : 1);
    const int threads = ((pieces + V - 1) / V + 63) / 64 * 64;
    const bool past = a.T * a.N * (2 + (a.r ? 2 : 0) + (a.h ? 2 : 0) + (F8 ? 1 : 2)) > (int64_t)256 << 20;
    if (V == 1) hipLaunchKernelGGL((k_rms_norm<F16, F8, 1, false>), grid, dim3(threads), 0, st, a);
    else if (V == 2 && past) hipLaunchKernelGGL((k_rms_norm<F16, F8, 2, true>), grid, dim3(threads), 0, st, a);
    else if (V == 2) hipLaunchKernelGGL((k_rms_norm<F16, F8, 2, false>), grid, dim3(threads), 0, st, a);
    else if (past) hipLaunchKernelGGL((k_rms_norm<F16, F8, 4, true>), grid, dim3(threads), 0, st, a);
    else hipLaunchKernelGGL((k_rms_norm<F16, F8, 4, false>), grid, dim3(threads), 0, st, a);
}

constexpr int64_t kNormVecMax = 1024 * 8 * 4;

// ------------------------------------------------------------ cache checks --

struct CacheView {
    KvSide k, v;
    KvShape shape;
    int format;
};

nvfp4_status check_side(const char* fn, const char* name, const nvfp4_kv_cache& c, const void* base,
                        const int64_t (&st)[3], int64_t block) {
    if (!base) return fail(NVFP4_ERR_INVALID_ARG, "%s: cache %s is NULL", fn, name);
    for (int i = 0; i < 3; ++i) {
        if (i == 2 && c.format == NVFP4_KV_NVFP4) continue;
        if (st[i] < 0 || st[i] >= kBig)
            return fail(NVFP4_ERR_INVALID_ARG, "%s: cache %s stride %d = %lld is out of range", fn, name, i,
                        (long long)st[i]);
        if (st[i] % 16 != 0)
            return fail(NVFP4_ERR_ALIGNMENT, "%s: cache %s stride %d = %lld is not a multiple of 16 bytes", fn, name, i,
                        (long long)st[i]);
    }
    if (!aligned(base, 16)) return fail(NVFP4_ERR_ALIGNMENT, "%s: cache %s must be 16-byte aligned", fn, name);
    // offsets are kept in 32 bits of 16-byte units
    const __int128 span = (__int128)(c.pages - 1) * st[0] + (__int128)(c.heads - 1) * st[1] +
                          (c.format == NVFP4_KV_NVFP4 ? block : (__int128)(c.page_size - 1) * st[2]);
    if (span >= ((__int128)1 << 36))
        return fail(NVFP4_ERR_INVALID_ARG, "%s: cache %s spans 64 GB or more", fn, name);
    return NVFP4_OK;
}

nvfp4_status check_cache(const char* fn, const nvfp4_kv_cache* c, CacheView& out) {
    if (!c) return fail(NVFP4_ERR_INVALID_ARG, "%s: cache is NULL", fn);
    if (c->format < NVFP4_KV_16BIT || c->format > NVFP4_KV_NVFP4)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: unknown cache format %d", fn, (int)c->format);
    const int unit = c->format == NVFP4_KV_NVFP4 ? 32 : 16;
    if (c->head_dim < unit || c->head_dim > 256 || c->head_dim % unit != 0)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: head_dim = %d must be a multiple of %d up to 256", fn, (int)c->head_dim, unit);
    if (c->heads < 1 || c->heads > 65535)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: cache heads = %d must be in [1, 65535]", fn, (int)c->heads);
    if (c->page_size < 1 || c->pages < 1 || c->pages > ((int64_t)1 << 31) / c->page_size - 1)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: pages = %lld of page_size = %d: at least one page and fewer than 2^31 tokens",
                    fn, (long long)c->pages, (int)c->page_size);
    const int64_t block = (int64_t)c->page_size * c->head_dim / 16 * 9;
    if (c->format == NVFP4_KV_NVFP4 && block % 16 != 0)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: page_size = %d: an NVFP4 block of page_size * 9 * head_dim / 16 = %lld bytes "
                    "must be a multiple of 16", fn, (int)c->page_size, (long long)block);
    if (c->format == NVFP4_KV_16BIT && (c->k_scale || c->v_scale))
        return fail(NVFP4_ERR_INVALID_ARG, "%s: a 16-bit cache takes no scales", fn);
    if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: cache scales must be 4-byte aligned", fn);
    nvfp4_status st = check_side(fn, "k", *c, c->k, c->k_stride, block);
    if (st == NVFP4_OK) st = check_side(fn, "v", *c, c->v, c->v_stride, block);
    if (st != NVFP4_OK) return st;
    out.k = KvSide{static_cast<uint8_t*>(c->k), c->k_stride[0], c->k_stride[1], c->k_stride[2], c->k_scale};
    out.v = KvSide{static_cast<uint8_t*>(c->v), c->v_stride[0], c->v_stride[1], c->v_stride[2], c->v_scale};
    out.shape = KvShape{c->pages, c->page_size, c->heads, c->head_dim};
    out.format = c->format;
    return NVFP4_OK;
}

// A [T][H][D] array of 16-bit rows.
nvfp4_status check_rows(const char* fn, const char* name, const void* p, int64_t st_t, int64_t st_h) {
    if (!p) return fail(NVFP4_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    if (st_t < 0 || st_h < 0 || st_t >= kBig || st_h >= kBig)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: %s strides %lld, %lld are out of range", fn, name, (long long)st_t, (long long)st_h);
    if (!aligned(p, 16) || st_t % 8 != 0 || st_h % 8 != 0)
        return fail(NVFP4_ERR_ALIGNMENT, "%s: %s rows must be 16-byte aligned (strides %lld, %lld)", fn, name,
                    (long long)st_t, (long long)st_h);
    return NVFP4_OK;
}

nvfp4_status check_rope(const char* fn, const nvfp4_rope* r, int64_t D, int unit, int64_t T, RopeArgs& out) {
    if (!r->inv_freq || (!r->positions && T > 0)) return fail(NVFP4_ERR_INVALID_ARG, "%s: rope inv_freq or positions is NULL", fn);
    if (r->rotary < unit || r->rotary % unit != 0 || r->rotary > D || r->rotary > 2 * kRopeMaxPairs)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: rotary = %d must be a multiple of %d up to min(head_dim = %lld, %d)", fn,
                    (int)r->rotary, unit, (long long)D, 2 * kRopeMaxPairs);
    if (r->axes < 1 || r->axes > 16 || (r->axes > 1 && !r->pair_axis))
        return fail(NVFP4_ERR_INVALID_ARG, "%s: %d axes: 1 to 16, and more than one need pair_axis", fn, (int)r->axes);
    if (r->ld_pos < T || r->ld_pos >= kBig) return fail(NVFP4_ERR_INVALID_ARG, "%s: ld_pos = %lld < T = %lld", fn, (long long)r->ld_pos, (long long)T);
    if (!aligned(r->inv_freq, 4) || !aligned(r->positions, 4) || !aligned(r->pair_axis, 4))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: rope arrays must be 4-byte aligned", fn);
    out = RopeArgs{r->inv_freq, r->positions, r->pair_axis, r->ld_pos, r->axes, r->rotary};
    return NVFP4_OK;
}

// ---------------------------------------------------------- rotate, append --

template <int FMT, bool F16, bool NB>
void launch_append_as(const AppendArgs& a, int TB, dim3 grid, hipStream_t st) {
    hipLaunchKernelGGL((k_rope_append<FMT, F16, NB>), grid, dim3(kRopeThreads), 0, st, a, TB);
}
template <int FMT>
void launch_append_fmt(const AppendArgs& a, int TB, dim3 grid, bool f16, bool nb, hipStream_t st) {
    if (f16) nb ? launch_append_as<FMT, true, true>(a, TB, grid, st) : launch_append_as<FMT, true, false>(a, TB, grid, st);
    else nb ? launch_append_as<FMT, false, true>(a, TB, grid, st) : launch_append_as<FMT, false, false>(a, TB, grid, st);
}

void launch_append(const AppendArgs& a, int format, bool f16, bool nb, hipStream_t st) {
    // A workgroup takes 256 units at a time.  With many tokens it gets the
    // fewest of them (up to eight) whose units fill its rounds to 90 %, or the
    // best filling there is (5003 tokens of 16 heads of 80: three, 240 units);
    // with fewer than two workgroups per compute unit each token gets its own,
    // and its units are spread over workgroups, a round each.
    const int64_t units = (int64_t)(a.Hq + 2 * a.Hk) * (a.D / 16);
    int TB = 1;
    if (a.T >= 1024) {
        double best = 0.;
        for (int n = 1; n <= kRopeMaxTokens && a.T / n >= 512 && best < 0.9; ++n) {
            const double fill = (double)(n * units) / (double)((n * units + kRopeThreads - 1) / kRopeThreads * kRopeThreads);
            if (fill > best) {
                best = fill;
                TB = n;
            }
        }
    }
    const int64_t rounds = (TB * units + kRopeThreads - 1) / kRopeThreads;
    int64_t gy = a.T >= 1024 ? 1 : (512 + a.T - 1) / a.T;
    if (gy > rounds) gy = rounds;
    const dim3 grid((unsigned)((a.T + TB - 1) / TB), (unsigned)gy);
    if (format == kKv16) launch_append_fmt<kKv16>(a, TB, grid, f16, nb, st);
    else if (format == kKvE4m3) launch_append_fmt<kKvE4m3>(a, TB, grid, f16, nb, st);
    else launch_append_fmt<kKvNvfp4>(a, TB, grid, f16, nb, st);
}

template <int FMT>
void launch_read(const ReadArgs& a, bool f16, dim3 grid, hipStream_t st) {
    if (f16) hipLaunchKernelGGL((k_kv_read<FMT, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_kv_read<FMT, false>), grid, dim3(256), 0, st, a);
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_rms_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_r, const void* weight,
                            float eps, void* y, int64_t ld_y, float* scales, void* h, int64_t ld_h, int64_t T,
                            int64_t N, int f16, void* stream) {
    const char* fn = "nvfp4_rms_norm";
    const int64_t lim = (int64_t)1 << 31;
    // the column counters are 32 bits wide and go on 256 past the last column
    if (T < 0 || T >= lim || N < 1 || N > lim - 256)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: T = %lld, N = %lld", fn, (long long)T, (long long)N);
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(NVFP4_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
    if (h && !residual) return fail(NVFP4_ERR_INVALID_ARG, "%s: h is only written with a residual", fn);
    if (ld_x < N || ld_y < N || (residual && ld_r < N) || (h && ld_h < N) || ld_x >= kBig || ld_y >= kBig ||
        (residual && ld_r >= kBig) || (h && ld_h >= kBig))
        return fail(NVFP4_ERR_INVALID_ARG, "%s: a leading dimension is below N = %lld or too large", fn, (long long)N);
    if (!weight || (T > 0 && (!x || !y))) return fail(NVFP4_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(weight, 2) || !aligned(h, 2) || (!scales && !aligned(y, 2)) ||
        !aligned(scales, 4))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: misaligned pointer", fn);
    if (T == 0) return ok();
    NormArgs a;
    a.x = static_cast<const uint16_t*>(x);
    a.r = static_cast<const uint16_t*>(residual);
    a.w = static_cast<const uint16_t*>(weight);
    a.h = static_cast<uint16_t*>(h);
    a.y = y;
    a.scales = scales;
    a.ld_x = ld_x;
    a.ld_r = ld_r;
    a.ld_h = ld_h;
    a.ld_y = ld_y;
    a.T = T;
    a.N = (int)N;
    a.eps = eps;
    const bool vec = N % 8 == 0 && N <= kNormVecMax && ld_x % 8 == 0 && ld_y % 8 == 0 && (!residual || ld_r % 8 == 0) &&
                     (!h || ld_h % 8 == 0) && aligned(x, 16) && aligned(residual, 16) && aligned(weight, 16) &&
                     aligned(h, 16) && aligned(y, scales ? 8 : 16);
    hipStream_t st = static_cast<hipStream_t>(stream);
    const nvfp4_status sized = check_launch(fn, T, !vec ? 256 : N <= 128 ? 16 : N <= 256 ? 32 : 1024);
    if (sized != NVFP4_OK) return sized;
    if (f16) scales ? launch_norm<true, true>(a, vec, st) : launch_norm<true, false>(a, vec, st);
    else scales ? launch_norm<false, true>(a, vec, st) : launch_norm<false, false>(a, vec, st);
    return launched(fn);
}

nvfp4_status nvfp4_rope_apply(const nvfp4_rope* rope, const void* x, int64_t x_t, int64_t x_h, void* out, int64_t o_t,
                              int64_t o_h, int64_t T, int64_t H, int64_t D, int f16, void* stream) {
    const char* fn = "nvfp4_rope_apply";
    if (T < 0 || T >= (int64_t)1 << 31 || H < 0 || H > 65535)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: T = %lld, H = %lld", fn, (long long)T, (long long)H);
    if (D < 16 || D > 1024 || D % 16 != 0)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: D = %lld must be a multiple of 16 up to 1024", fn, (long long)D);
    if (!rope) return fail(NVFP4_ERR_INVALID_ARG, "%s: rope is NULL", fn);
    AppendArgs a = {};
    nvfp4_status s = check_rope(fn, rope, D, 16, T, a.rope);
    if (s != NVFP4_OK) return s;
    if (T == 0 || H == 0) return ok();
    s = check_rows(fn, "x", x, x_t, x_h);
    if (s == NVFP4_OK) s = check_rows(fn, "out", out, o_t, o_h);
    if (s != NVFP4_OK) return s;
    a.q = static_cast<const uint16_t*>(x);
    a.q_out = static_cast<uint16_t*>(out);
    a.q_t = x_t;
    a.q_h = x_h;
    a.qo_t = o_t;
    a.qo_h = o_h;
    a.Hq = (int)H;
    a.T = T;
    a.D = (int)D;
    s = check_launch(fn, T, kRopeThreads);
    if (s != NVFP4_OK) return s;
    launch_append(a, kKv16, f16 != 0, rope->neighbours != 0, static_cast<hipStream_t>(stream));
    return launched(fn);
}

nvfp4_status nvfp4_kv_append(const nvfp4_kv_cache* cache, const nvfp4_rope* rope, const void* q, int64_t q_t,
                             int64_t q_h, void* q_out, int64_t qo_t, int64_t qo_h, int64_t Hq, const void* k,
                             int64_t k_t, int64_t k_h, const void* v, int64_t v_t, int64_t v_h, const int32_t* slots,
                             int64_t T, int f16, void* stream) {
    const char* fn = "nvfp4_kv_append";
    CacheView c;
    nvfp4_status s = check_cache(fn, cache, c);
    if (s != NVFP4_OK) return s;
    if (T < 0 || T >= (int64_t)1 << 31 || Hq < 0 || Hq > 65535)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: T = %lld, Hq = %lld", fn, (long long)T, (long long)Hq);
    if (Hq > 0 && !rope) return fail(NVFP4_ERR_INVALID_ARG, "%s: queries are only rotated: they need rope", fn);
    AppendArgs a = {};
    if (rope) s = check_rope(fn, rope, c.shape.D, c.format == kKvNvfp4 ? 32 : 16, T, a.rope);
    if (s != NVFP4_OK) return s;
    if (T == 0) return ok();
    if (Hq > 0) {
        s = check_rows(fn, "q", q, q_t, q_h);
        if (s == NVFP4_OK) s = check_rows(fn, "q_out", q_out, qo_t, qo_h);
    }
    if (s == NVFP4_OK) s = check_rows(fn, "k", k, k_t, k_h);
    if (s == NVFP4_OK) s = check_rows(fn, "v", v, v_t, v_h);
    if (s != NVFP4_OK) return s;
    if (!slots) return fail(NVFP4_ERR_INVALID_ARG, "%s: slots is NULL", fn);
    if (!aligned(slots, 4)) return fail(NVFP4_ERR_ALIGNMENT, "%s: slots must be 4-byte aligned", fn);
    a.q = static_cast<const uint16_t*>(q);
    a.q_out = static_cast<uint16_t*>(q_out);
    a.q_t = q_t;
    a.q_h = q_h;
    a.qo_t = qo_t;
    a.qo_h = qo_h;
    a.Hq = (int)Hq;
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.k_t = k_t;
    a.k_h = k_h;
    a.v_t = v_t;
    a.v_h = v_h;
    a.Hk = c.shape.heads;
    a.slots = slots;
    a.kc = c.k;
    a.vc = c.v;
    a.shape = c.shape;
    a.T = T;
    a.D = c.shape.D;
    s = check_launch(fn, T, kRopeThreads);
    if (s != NVFP4_OK) return s;
    launch_append(a, c.format, f16 != 0, rope && rope->neighbours != 0, static_cast<hipStream_t>(stream));
    return launched(fn);
}

nvfp4_status nvfp4_kv_read(const nvfp4_kv_cache* cache, const int32_t* slots, void* k, int64_t k_t, int64_t k_h,
                           void* v, int64_t v_t, int64_t v_h, int64_t T, int f16, void* stream) {
    const char* fn = "nvfp4_kv_read";
    CacheView c;
    nvfp4_status s = check_cache(fn, cache, c);
    if (s != NVFP4_OK) return s;
    if (T < 0 || T >= (int64_t)1 << 31) return fail(NVFP4_ERR_INVALID_ARG, "%s: T = %lld", fn, (long long)T);
    if (T == 0) return ok();
    s = check_rows(fn, "k", k, k_t, k_h);
    if (s == NVFP4_OK) s = check_rows(fn, "v", v, v_t, v_h);
    if (s != NVFP4_OK) return s;
    if (!slots) return fail(NVFP4_ERR_INVALID_ARG, "%s: slots is NULL", fn);
    if (!aligned(slots, 4)) return fail(NVFP4_ERR_ALIGNMENT, "%s: slots must be 4-byte aligned", fn);
    ReadArgs a;
    a.kc = c.k;
    a.vc = c.v;
    a.shape = c.shape;
    a.slots = slots;
    a.k = static_cast<uint16_t*>(k);
    a.v = static_cast<uint16_t*>(v);
    a.k_t = k_t;
    a.k_h = k_h;
    a.v_t = v_t;
    a.v_h = v_h;
    a.T = T;
    const int64_t threads = T * 2 * c.shape.heads * (c.shape.D / 16);
    const int64_t groups = (threads + 255) / 256;
    s = check_launch(fn, groups, 256);
    if (s != NVFP4_OK) return s;
    const dim3 grid((unsigned)groups);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (c.format == kKv16) launch_read<kKv16>(a, f16 != 0, grid, st);
    else if (c.format == kKvE4m3) launch_read<kKvE4m3>(a, f16 != 0, grid, st);
    else launch_read<kKvNvfp4>(a, f16 != 0, grid, st);
    return launched(fn);
}

}  // extern "C"

namespace {

nvfp4_status check_attn_sizes(const char* fn, int64_t B, int64_t Hq, int64_t heads, int64_t D, int64_t max_tokens) {
    if (B < 0 || B > 65535) return fail(NVFP4_ERR_INVALID_ARG, "%s: B = %lld must be in [0, 65535]", fn, (long long)B);
    if (heads < 1 || Hq < 1 || Hq % heads != 0 || Hq > ((int64_t)1 << 20))
        return fail(NVFP4_ERR_INVALID_ARG, "%s: Hq = %lld must be a positive multiple of the %lld key-value heads", fn,
                    (long long)Hq, (long long)heads);
    if (heads * ((Hq / heads + kAttnHeads - 1) / kAttnHeads) > 65535)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: Hq = %lld over %lld key-value heads is too many heads", fn, (long long)Hq, (long long)heads);
    if (D < 16 || D > 256 || D % 16 != 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: D = %lld must be a multiple of 16 up to 256", fn, (long long)D);
    const nvfp4_status sized = check_launch(fn, B * heads * ((Hq / heads + kAttnHeads - 1) / kAttnHeads), kAttnThreads);
    if (sized != NVFP4_OK) return sized;
    if (max_tokens < 0 || max_tokens >= (int64_t)1 << 30)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: %lld tokens: the table must hold fewer than 2^30", fn, (long long)max_tokens);
    return NVFP4_OK;
}

}  // namespace

extern "C" {

int64_t nvfp4_paged_attention_workspace_bytes(int64_t B, int64_t Hq, int64_t heads, int64_t D, int64_t max_tokens) {
    if (check_attn_sizes("nvfp4_paged_attention_workspace_bytes", B, Hq, heads, D, max_tokens) != NVFP4_OK) return -1;
    return attn_shape(B, heads, Hq / heads, D, max_tokens).total;
}

nvfp4_status nvfp4_paged_attention(const nvfp4_kv_cache* cache, const void* q, int64_t q_b, int64_t q_h,
                                   const int32_t* page_table, int64_t ld_table, int64_t max_pages,
                                   const int32_t* lengths, int64_t B, int64_t Hq, float softmax_scale, int64_t window,
                                   void* out, int64_t o_b, int64_t o_h, float* lse, void* workspace,
                                   int64_t workspace_bytes, int f16, void* stream) {
    const char* fn = "nvfp4_paged_attention";
    CacheView c;
    nvfp4_status s = check_cache(fn, cache, c);
    if (s != NVFP4_OK) return s;
    if (max_pages < 0 || max_pages >= (int64_t)1 << 30 || ld_table < max_pages || ld_table >= kBig)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: max_pages = %lld, ld_table = %lld", fn, (long long)max_pages, (long long)ld_table);
    const int64_t max_tokens = max_pages * c.shape.page_size;
    s = check_attn_sizes(fn, B, Hq, c.shape.heads, c.shape.D, max_tokens);
    if (s != NVFP4_OK) return s;
    if (!std::isfinite(softmax_scale)) return fail(NVFP4_ERR_INVALID_ARG, "%s: softmax_scale must be finite", fn);
    if (window < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: window = %lld is negative", fn, (long long)window);
    if (B == 0) return ok();
    s = check_rows(fn, "q", q, q_b, q_h);
    if (s == NVFP4_OK) s = check_rows(fn, "out", out, o_b, o_h);
    if (s != NVFP4_OK) return s;
    if (!lengths || (!page_table && max_pages > 0)) return fail(NVFP4_ERR_INVALID_ARG, "%s: page_table or lengths is NULL", fn);
    if (!aligned(page_table, 4) || !aligned(lengths, 4) || !aligned(lse, 4))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: page_table, lengths and lse must be 4-byte aligned", fn);
    const int64_t G = Hq / c.shape.heads;
    const AttnShape sh = attn_shape(B, c.shape.heads, G, c.shape.D, max_tokens);
    if (sh.total > 0) {
        if (!workspace || workspace_bytes < sh.total)
            return fail(NVFP4_ERR_BUFFER_TOO_SMALL, "%s: workspace of %lld bytes is below the %lld bytes this call needs", fn,
                        (long long)workspace_bytes, (long long)sh.total);
        if (!aligned(workspace, 256)) return fail(NVFP4_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", fn);
    }
    AttnArgs a;
    a.q = static_cast<const uint16_t*>(q);
    a.q_b = q_b;
    a.q_h = q_h;
    a.kc = c.k;
    a.vc = c.v;
    a.shape = c.shape;
    a.table = page_table;
    a.ld_table = ld_table;
    a.width = (int)max_pages;
    a.lengths = lengths;
    a.G = (int)G;
    a.head_tiles = (int)((G + kAttnHeads - 1) / kAttnHeads);
    a.Hq = (int)Hq;
    a.window = window > max_tokens ? 0 : (int)window;
    a.scale_log2 = softmax_scale * 1.44269504088896340736f;
    a.out = static_cast<uint16_t*>(out);
    a.o_b = o_b;
    a.o_h = o_h;
    a.lse = lse;
    a.f16 = f16 != 0;
    a.split = sh.split;
    a.grid = (int)sh.workgroups;
    a.B = (int)B;
    a.counters = static_cast<int*>(workspace);
    a.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + kAttnCounterBytes);
    hipStream_t st = static_cast<hipStream_t>(stream);
    // umulhi(t, ceil(2^(32 + s) / page_size)) >> s is t / page_size for t < 2^31 with 2^s < page_size <= 2^(s + 1)
    a.page_shift = 0;
    while ((int64_t)2 << a.page_shift < c.shape.page_size) ++a.page_shift;
    a.page_magic = c.shape.page_size == 1 ? 0u
                   : (uint32_t)((((uint64_t)1 << (32 + a.page_shift)) + c.shape.page_size - 1) / (uint64_t)c.shape.page_size);
    // 32-bit offsets: inside a half-tile of 16 tokens below 2^30, of an NVFP4 block's scales below 2^31
    const int64_t far = (int64_t)1 << 26;
    const bool fast = c.shape.page_size % 16 == 0 &&
                      (c.format == kKvNvfp4 ? c.shape.page_size < 1 << 23 : c.k.s_token < far && c.v.s_token < far);
    if (c.format == kKvE4m3) launch_attn_e4m3(a, fast, sh.workgroups, st);
    else if (c.format == kKvNvfp4) launch_attn_nvfp4(a, fast, sh.workgroups, st);
    else if (f16) launch_attn_f16(a, fast, sh.workgroups, st);
    else launch_attn_bf16(a, fast, sh.workgroups, st);
    return launched(fn);
}

}  // extern "C"
