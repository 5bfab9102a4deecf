// Rounding to the small formats (E4M3, E2M1 with E4M3 group scales) and back,
// shared by the norm's 8-bit output, the key-value cache and its attention.
#pragma once
#include "decode.h"

namespace nvfp4 {

// 16-byte piece of eight 16-bit values <-> eight fp32.
template <bool F16>
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = act_to_f32<F16>(d[i] & 0xFFFFu);
        f[2 * i + 1] = act_to_f32<F16>(d[i] >> 16);
    }
}
// Round to nearest even; each value passes as an fp32 value (decode.h) so
// that no multiply before it is folded into the rounding.
template <bool F16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = pack_round2<F16>(fp32_value(f[2 * i]), fp32_value(f[2 * i + 1]));
    return make_uint4(d[0], d[1], d[2], d[3]);
}

// Saturation to the largest finite E4M3 value; a NaN stays one.
__device__ __forceinline__ float clamp_e4m3(float v) {
    const float c = fminf(fmaxf(v, -448.0f), 448.0f);
    return v != v ? v : c;
}
// Two values -> two E4M3 bytes (first in the low byte), round to nearest
// even.  The hardware conversion is to the OCP format on gfx950.
__device__ __forceinline__ uint32_t e4m3_bytes2(float a, float b) {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(a), clamp_e4m3(b), 0, false) & 0xFFFFu;
}
__device__ __forceinline__ uint32_t e4m3_byte(float a) { return e4m3_bytes2(a, 0.f) & 0xFFu; }
// Eight values times `by` -> eight E4M3 bytes.
__device__ __forceinline__ uint2 e4m3_pack8(const float (&f)[8], float by) {
    uint32_t d[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(f[4 * i] * by), clamp_e4m3(f[4 * i + 1] * by), 0, false);
        p = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(f[4 * i + 2] * by), clamp_e4m3(f[4 * i + 3] * by), p, true);
        d[i] = (uint32_t)p;
    }
    return make_uint2(d[0], d[1]);
}

// Scale of a row whose largest absolute value is `top`: top / 448, at least
// the smallest normal fp32 (a row of zeros then has finite codes and scale);
// NaN stays NaN.
__device__ __forceinline__ float norm_row_scale(float top) {
    const float s = __fdiv_rn(top, 448.0f);
    return s != s ? s : fmaxf(s, 0x1p-126f);
}

// The E4M3 scale byte of a 16-value NVFP4 group: e4m3(top * r * (1/6)), r the
// reciprocal of the head's scale, so that the largest code is 6 or near it.
// Saturates at 448; a NaN gives the NaN byte, which makes the group read back
// as NaN (E2M1 has none).
__device__ __forceinline__ uint32_t nvfp4_group_scale(float top, float r) {
    return e4m3_byte(fp32_value(top * r) * (1.0f / 6.0f));
}
// What a group's values are multiplied by before they are rounded to E2M1:
// r / scale, 0 for a zero (or NaN) scale.
__device__ __forceinline__ float nvfp4_group_factor(uint32_t scale_byte, float r) {
    const float s = e4m3_to_f32(scale_byte);
    return s > 0.f ? __fdiv_rn(r, s) : 0.f;
}
// Eight values times `by` -> eight E2M1 codes, lowest column in the lowest
// nibble; round to nearest, ties to even, saturating at 6 (a value with by =
// 0 gives code 0, also where it is an infinity or a NaN).
__device__ __forceinline__ uint32_t nvfp4_codes8(const float (&f)[8], float by) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float p = f[i] * by;
        v[i] = by == 0.f ? 0.f : fminf(fmaxf(p, -6.0f), 6.0f);
    }
    uint32_t d = 0u;
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[0], v[1], 1.0f, 0);
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[2], v[3], 1.0f, 1);
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[4], v[5], 1.0f, 2);
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[6], v[7], 1.0f, 3);
    return d;
}

}  // namespace nvfp4
