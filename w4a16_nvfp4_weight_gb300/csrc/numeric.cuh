// Conversions shared by the kernels around the linears (norm, rotary positions,
// key-value cache, attention): 16-bit activations to and from 32 bits, and the
// E4M3 rows with one 32-bit scale that the norm and the cache write.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace nvfp4 {

constexpr float kE4m3Max = 448.f;
// Smallest scale of an E4M3 row.  It keeps x / scale defined for a row of
// zeros, and a scale times exp2 of a score inside the range of 32 bits.
constexpr float kMinScale = 0x1p-100f;

// 16 bytes that are read once and may be written later in the same kernel (in place).
__device__ __forceinline__ uint4 ldg_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

template <bool F16>
__device__ __forceinline__ float act_to_f32(uint16_t b) {
    return F16 ? f16_bits_to_f32(b) : __uint_as_float((uint32_t)b << 16);
}

// The two activations of a 32-bit word (low half first).
template <bool F16>
__device__ __forceinline__ float2 act2_to_f32(uint32_t w) {
    return make_float2(act_to_f32<F16>((uint16_t)w), F16 ? f16_bits_to_f32((uint16_t)(w >> 16))
                                                         : __uint_as_float(w & 0xffff0000u));
}

// Two FP32 values rounded to activations, `lo` in the low half.
template <bool F16>
__device__ __forceinline__ uint32_t f32_to_act2(float lo, float hi) {
    uint32_t d;
    if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// The same rounded towards zero.
template <bool F16>
__device__ __forceinline__ uint32_t f32_to_act2_down(float lo, float hi) {
    uint32_t d;
    if (F16) asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    else asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two FP32 values rounded to E4M3 (nearest even, saturating at +-448, NaN kept).
__device__ __forceinline__ uint16_t f32_to_e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two E4M3 codes as FP16 (exact: every E4M3 value is an FP16 value).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(c));
    return d;
}

// x / d by `inv`, d's reciprocal to a last bit or so: the quotient by it and one
// correction by its remainder (Markstein, IBM Journal of Research and Development
// 34, 1990).  Three operations where an IEEE division an element took a third of
// the E4M3 norm's time.  For finite d in [2^-100, 2^120] nothing under- or overflows
// on the way, and a quotient that is a value of 32 bits comes out as that.
__device__ __forceinline__ float quotient(float x, float d, float inv) {
    const float q = x * inv;
    return fmaf(fmaf(-q, d, x), inv, q);
}

// Scale of an E4M3 row whose largest magnitude is `amax`: amax / 448, rounded as
// IEEE division does (every significand was checked against it), so that scales and
// codes are the same on every path.
__device__ __forceinline__ float e4m3_scale(float amax) {
    const float s = amax < INFINITY ? quotient(amax, kE4m3Max, 1.f / kE4m3Max) : INFINITY;
    return fmaxf(s, kMinScale);
}
__device__ __forceinline__ float e4m3_inverse(float s) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
    return y;
}

// Two 32-bit values: products and fused ones take one instruction for both.
struct F2 { uint64_t v; };
__device__ __forceinline__ F2 make_f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 both(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
// Sums one value at a time: a packed addition after a packed product came out as
// one fused operation, with one rounding instead of two.
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    const float2 u = both(a), v = both(b);
    return make_f2(__fadd_rn(u.x, v.x), __fadd_rn(u.y, v.y));
}
__device__ __forceinline__ F2 sub2(F2 a, F2 b) {
    const float2 u = both(a), v = both(b);
    return make_f2(__fsub_rn(u.x, v.x), __fsub_rn(u.y, v.y));
}

// The two activations of a 32-bit word as a pair.
template <bool F16>
__device__ __forceinline__ F2 widen2(uint32_t w) {
    const float2 u = act2_to_f32<F16>(w);
    return make_f2(u.x, u.y);
}

// Code of x in a row of scale s, inv = e4m3_inverse(s).  An infinite scale gives NaN.
__device__ __forceinline__ uint8_t e4m3_code(float x, float s, float inv) { return (uint8_t)f32_to_e4m3x2(quotient(x, s, inv), 0.f); }

// Codes of two values, the first in the low byte.
__device__ __forceinline__ uint16_t e4m3_codes(F2 x, F2 minus_s, F2 inv) {
    const F2 q = mul2(x, inv);
    const float2 r = both(fma2(fma2(q, minus_s, x), inv, q));
    return f32_to_e4m3x2(r.x, r.y);
}

}  // namespace nvfp4
