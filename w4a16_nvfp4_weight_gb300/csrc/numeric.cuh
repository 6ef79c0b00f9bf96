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

// Scale of an E4M3 row whose largest magnitude is `amax`: one IEEE division, so
// that scales and codes are the same on every path.
__device__ __forceinline__ float e4m3_scale(float amax) { return fmaxf(__fdiv_rn(amax, kE4m3Max), kMinScale); }

// x / s for the codes of a row with scale s and inv = __frcp_rn(s): the quotient
// by the reciprocal and one correction by its remainder (Markstein, IBM Journal
// of Research and Development 34, 1990), three operations where an IEEE division
// an element took a third of the E4M3 norm's time.  Scales lie in [2^-100, 2^120],
// so nothing under- or overflows on the way; an infinite scale gives NaN.
__device__ __forceinline__ float e4m3_quotient(float x, float s, float inv) {
    const float q = x * inv;
    return fmaf(fmaf(-q, s, x), inv, q);
}

}  // namespace nvfp4
