// wq_quotient.cuh -- arithmetic shared by the quantisers: correctly rounded
// quotients from a reciprocal, rounding by an addition, packed binary32
// pairs and the INT4 scale.
#pragma once

#include "wq_common.cuh"

namespace wq {

// Correctly rounded quotients w / s for the codes, without a division per weight.  Markstein's final
// correction step (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", IBM J. Res. Dev. 34(1), 1990): with r = RN(1/s) and q0 = RN(w * r), the residual
// e = w - q0 * s is exact (one fused multiply-add), and RN(q0 + e * r) = RN(w / s) provided the reciprocal
// and the quotient stay in the normal range.  The scales here are bf16 values; for every bf16 significand
// of s and every binary32 significand of w this identity was checked exhaustively (the check is part of
// the test suite).  A group whose scale or largest quotient could leave the normal range uses the IEEE
// division instead; quotients too small to be normal never change a code (t = RN(q + z) rounds to z, or
// to 0 when z = 0).
__device__ __forceinline__ bool quotients_by_reciprocal(float s, float maxabs)
{
    return s >= 0x1p-100f && s <= 0x1p100f && maxabs <= s * 0x1p100f;
}

__device__ __forceinline__ float quotient_rn(float w, float s, float r)
{
    const float q0 = __fmul_rn(w, r);
    const float e = __fmaf_rn(-q0, s, w);
    return __fmaf_rn(e, r, q0);
}

// RN(d / c) for a bf16-representable constant c (15 or 127) with rc = RN(1 / c): the same identity, with
// the IEEE division where d could leave its proven range (d non-finite, above 2^100, or tiny but not 0).
__device__ __forceinline__ float div_by_const_rn(float d, float c, float rc)
{
    const float ad = fabsf(d);
    return (ad <= 0x1p100f && (ad >= 0x1p-90f || ad == 0.0f)) ? quotient_rn(d, c, rc) : __fdiv_rn(d, c);
}
constexpr float kRcp15 = 0x1.111112p-4f;   // RN(1 / 15)
constexpr float kRcp7 = 0x1.24924ap-3f;    // RN(1 / 7)
constexpr float kRcp127 = 0x1.020408p-7f;  // RN(1 / 127)

// Round an integer-bound value t, already clipped to [-127, 127], to the nearest integer with ties to
// even, and return the binary32 bit pattern of 1.5 * 2^23 + round(t): the integer sits in the low bits
// (two's complement in the low byte for negative t).  Adding 1.5 * 2^23 leaves a unit in the last place
// of 1, so the addition itself is the rounding.
__device__ __forceinline__ uint32_t rint_bits(float t) { return __float_as_uint(__fadd_rn(t, 0x1.8p23f)); }
constexpr uint32_t kRintBase = 0x4B400000u;  // bits of 1.5 * 2^23

// Packed binary32 pairs (sm_100 f32x2 arithmetic; round to nearest, no fused contraction across the pair):
// the low 32 bits hold the first value.
__device__ __forceinline__ uint64_t f32x2_bits(float lo, float hi)
{
    return ((uint64_t)__float_as_uint(hi) << 32) | (uint64_t)__float_as_uint(lo);
}
__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// s of one INT4 group from its min and max (the library contract): RN((max - min) / 15) rounded to bf16;
// a zero range falls back to max(|min|, |max|), then to 1.
__device__ __forceinline__ float int4_scale(float mn, float mx)
{
    float s = round_bf16(div_by_const_rn(__fsub_rn(mx, mn), 15.0f, kRcp15));
    if (s == 0.0f) {
        s = round_bf16(fmaxf(fabsf(mn), fabsf(mx)));
        if (s == 0.0f) s = 1.0f;
    }
    return s;
}

// bf16x2 minimum (each half; a NaN half yields the other operand's half, as fminf does)
__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

}  // namespace wq
