// f32x2.cuh -- fp32 arithmetic on pairs and 2^x on the FMA pipe, for the kernels around the
// block that form many exponentials (prefill_attn.cu has its own, with the same coefficients,
// for arguments that are never above zero).
#pragma once

#include "common.cuh"

namespace hs2 {

// ---- packed fp32 pairs (one instruction for two lanes of arithmetic on sm_100)
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("{\n\t.reg .b64 ra, rb, rc;\n\t"
        "mov.b64 ra, {%1, %2};\n\tmov.b64 rb, {%3, %4};\n\tmov.b64 rc, {%5, %6};\n\t"
        "fma.rn.f32x2 %0, ra, rb, rc;\n\t}"
        : "=l"(d) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("{\n\t.reg .b64 ra, rb;\n\t"
        "mov.b64 ra, {%1, %2};\n\tmov.b64 rb, {%3, %4};\n\t"
        "add.rn.f32x2 %0, ra, rb;\n\t}"
        : "=l"(d) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float clamp_nan(float x, float lo, float hi) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(lo));
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(r) : "f"(hi));
    return r;
}

// sum + 2^x for a pair on the FMA pipe (where the exponential unit is the bottleneck, a
// share of the exponentials moves here): x = j + r with j the nearest integer (added to
// and taken back from 1.5 * 2^23, whose ulp is 1) and r in [-1/2, 1/2]; 2^r by a degree-5
// polynomial, the minimax relative-error fit of 2^r on that interval by Lawson's algorithm
// (least squares reweighted by the error until it equioscillates; exp2_poly_fit.py beside
// this package prints the coefficients): max relative error 2.1e-7 in fp32 Horner form,
// like the exponential unit's.  2^j, made of exponent bits, comes in with the addition, one
// multiply-add: 0 below x = -126.5 and infinity from 127.5 up (between them j is -126 ..
// 127), as fp32's own range ends, and a NaN stays one.  (Added to the polynomial's exponent
// bits instead, j wrapped around for large x and a NaN came out as a number.)
__device__ __forceinline__ float2 add_exp2_poly2(float2 x, float2 sum) {
    constexpr float kMagic = 12582912.f;                       // 1.5 * 2^23
    x.x = clamp_nan(x.x, -127.f, 128.f);
    x.y = clamp_nan(x.y, -127.f, 128.f);
    const float2 t = add2(x, make_float2(kMagic, kMagic));
    const float2 j = add2(t, make_float2(-kMagic, -kMagic));
    const float2 r = add2(x, make_float2(-j.x, -j.y));
    float2 p = make_float2(1.3276455e-3f, 1.3276455e-3f);
    p = fma2(p, r, make_float2(9.6755400e-3f, 9.6755400e-3f));
    p = fma2(p, r, make_float2(5.5507135e-2f, 5.5507135e-2f));
    p = fma2(p, r, make_float2(2.4022120e-1f, 2.4022120e-1f));
    p = fma2(p, r, make_float2(6.9314694e-1f, 6.9314694e-1f));
    p = fma2(p, r, make_float2(1.0000001f, 1.0000001f));
    // exponent bits j + 127 in [0, 255] (kMagic's lower bits are zero)
    const float2 s = make_float2(__int_as_float((__float_as_int(t.x) << 23) + 0x3f800000),
                                 __int_as_float((__float_as_int(t.y) << 23) + 0x3f800000));
    return fma2(p, s, sum);
}

}  // namespace hs2
