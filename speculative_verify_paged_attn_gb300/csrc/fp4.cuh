// fp4.cuh -- rows of 4-bit pages: E2M1 codes with one E4M3 scale for each 16
// elements.
//
// A (page, kv head) tile is 16 rows of D / 2 code bytes (two codes a byte, the
// even element in the low half) and behind them 16 rows of D / 16 scale bytes;
// element d of a row stands for e2m1(code) * e4m3(scale[d / 16]) * factor[head].
// The first product has 2 + 4 significant bits and lies in [2^-10, 2688], so
// it is exact in f16 and in bf16.
#pragma once

#include "svpa_device.cuh"

namespace svpa {

// The bytes of one (page, kv head) tile, and of the codes before its scales.
__host__ __device__ constexpr int fp4_tile_bytes(int D) { return 16 * (D / 2 + D / 16); }
__host__ __device__ constexpr int fp4_code_bytes(int D) { return 16 * (D / 2); }

// A head's factor, as it is given (null: 1); outside [2^-60, 2^60], where a
// scale times it could leave the normal range, it is refused.
__device__ __forceinline__ float fp4_factor(const float *factor, int h, int32_t *err) {
    const float f = factor ? __ldg(factor + h) : 1.f;
    if (f >= 0x1p-60f && f <= 0x1p60f) return f;
    raise_error(err, SVPA_DEVERR_BAD_VALUE);
    return 1.f;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The largest magnitude of eight bf16 values, as bf16 bits (above 0x7f7f: one
// of them is not finite).
__device__ __forceinline__ uint32_t bf16_amax8(const uint4 &x) {
    const uint32_t a = __vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu);
    const uint32_t m = __vmaxu2(a, __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
    return max(m & 0xffffu, m >> 16);
}

// E4M3 (nearest even, saturating at 448), and a byte's value.
__device__ __forceinline__ uint32_t e4m3_of(float v) {
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.f), "f"(v));
    return h & 0xffu;
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    return f16x2_to_float2(e4m3x2_to_f16x2(byte)).x;
}

// Eight fp32 values to E2M1 (nearest even, saturating at 6), the first in the
// lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8_of(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight E2M1 codes to four f16 pairs (exact).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Codes of eight values of a 16-element group whose largest magnitude is amax
// (bf16 bits), and the group's scale byte:
//   scale = e4m3(amax / (6 f)),  code = e2m1(x / (e4m3 value * f)),
// every quotient and product rounded to fp32 once; codes 0 where the scale is 0.
//
// The quotients are correctly rounded without the division's code: two steps
// of q + (x - q d) / d with the correctly rounded reciprocal (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990): the first makes q faithful, the second then rounds
// correctly unless d's significand is all ones.  A remainder that underflows
// belongs to a quotient far below the first code's border.  A scale that
// saturated (quotients of 8 and more, which may overflow) and that one
// significand take the division.
__device__ __forceinline__ uint32_t fp4_encode8(const uint4 &x, uint32_t amax, float f, uint32_t &scale) {
    scale = e4m3_of(__fdiv_rn(__uint_as_float(amax << 16), __fmul_rn(6.f, f)));
    if (scale == 0u) return 0u;
    const float d = __fmul_rn(e4m3_value(scale), f);
    const float v[8] = {bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y),
                        bf16_lo(x.z), bf16_hi(x.z), bf16_lo(x.w), bf16_hi(x.w)};
    float q[8];
    if (__uint_as_float(amax << 16) < 8.f * d && (__float_as_uint(d) & 0x7fffffu) != 0x7fffffu) {
        const float inv = __frcp_rn(d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            q[i] = __fmul_rn(v[i], inv);
            q[i] = __fmaf_rn(__fmaf_rn(-q[i], d, v[i]), inv, q[i]);
            q[i] = __fmaf_rn(__fmaf_rn(-q[i], d, v[i]), inv, q[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(v[i], d);
    }
    return e2m1x8_of(q);
}

}  // namespace svpa
