// Rows as 16-byte pieces of eight bf16 values, and their quantisation to E4M3 codes with fp32 or E8M0 scales (shared by the
// kernels that make rows for the caches and for FP8 products, so that all make the same bytes).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace dsa {

// Two fp32 products, or products and sums, in one instruction (rounded like the single ones).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// Two E4M3 codes (a in the low byte), nearest-even, saturating at +-448.
__device__ __forceinline__ uint32_t codes2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Eight bf16 values of a 16-byte piece.
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(f2_to_bf2(x[0], x[1]), f2_to_bf2(x[2], x[3]), f2_to_bf2(x[4], x[5]), f2_to_bf2(x[6], x[7]));
}
__device__ __forceinline__ uint2 pack_codes(const float (&y)[8]) {
    return make_uint2(codes2(y[0], y[1]) | (codes2(y[2], y[3]) << 16), codes2(y[4], y[5]) | (codes2(y[6], y[7]) << 16));
}
// E4M3 codes of x / scale, the quotient rounded to fp32 first (so that both appends make the same codes).  With the
// correctly rounded reciprocal, y = x inv is within two units in the last place, y s - x is exact, and
// y - (y s - x) inv differs from the quotient by 2^-23 units before its rounding (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990): three packed operations a pair where a division
// takes ten a value.  (The signs are such that -0 stays -0.)  Scales whose products could leave fp32's range divide.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
    const float inv = __frcp_rn(scale);
    float y[8];
    if (scale > 0x1p-80f && scale < 0x1p80f) {
        const float2 inv2 = make_float2(inv, inv), minus2 = make_float2(-inv, -inv), scale2 = make_float2(scale, scale);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 v = mul2(make_float2(x[i], x[i + 1]), inv2);
            const float2 q = fma2(fma2(v, scale2, make_float2(-x[i], -x[i + 1])), minus2, v);
            y[i] = q.x;
            y[i + 1] = q.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], scale);
    }
    return pack_codes(y);
}
// The same for a scale of 2^e, -127 <= e <= 120: the product with 2^-e, a normal number, is the quotient.
__device__ __forceinline__ uint2 codes8_exp(const float (&x)[8], int e) {
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 v = mul2(make_float2(x[i], x[i + 1]), make_float2(inv, inv));
        y[i] = v.x;
        y[i + 1] = v.y;
    }
    return pack_codes(y);
}
__device__ __forceinline__ float absmax8(const float (&x)[8]) {
    const float a = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fabsf(x[2]));
    const float b = fmaxf(fmaxf(fabsf(x[3]), fabsf(x[4])), fabsf(x[5]));
    return fmaxf(fmaxf(fmaxf(a, b), fmaxf(fabsf(x[6]), fabsf(x[7]))), 0.f);  // (the 0: a group of NaN alone)
}
// absmax / 448 in fp32 (1 for an all-zero group); the product with 1/448 and one correction, as above (no quotient by 448
// comes closer to halfway between two fp32 numbers than a 14th of their distance)
__device__ __forceinline__ float group_scale(float amax) {
    if (!(amax > 0x1p-80f && amax < 0x1p120f)) return amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    const float c = 1.f / 448.f, y = amax * c;
    return __fmaf_rn(__fmaf_rn(-448.f, y, amax), c, y);
}

// Shared exponent of an MX group: floor(log2(absmax)) - 8 within the E8M0 range, 0 for an all-zero group.  (Subnormal
// maxima lie below the range either way; an infinity gives 120.)
__device__ __forceinline__ int mx_exponent(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    return bits == 0u ? 0 : max(-127, (int)(bits >> 23) - 127 - 8);
}

}  // namespace dsa
