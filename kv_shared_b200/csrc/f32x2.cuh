// f32x2.cuh -- fp32 arithmetic on pairs and 2^x on the FMA pipe, for the kernels around the
// block that form many exponentials (prefill_attn.cu has its own, with the same coefficients).
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

// 2^x for a pair on the FMA pipe (where the exponential unit is the bottleneck, a
// share of the exponentials moves here): x = j + r with j the nearest integer (added to
// and taken back from 1.5 * 2^23, whose ulp is 1) and r in [-1/2, 1/2]; 2^r by a degree-5
// polynomial, the minimax relative-error fit of 2^r on that interval by Lawson's algorithm
// (least squares reweighted by the error until it equioscillates; exp2_poly_fit.py beside
// this package prints the coefficients): max relative error 2.1e-7 in fp32 Horner form,
// like the exponential unit's; 2^j enters through the exponent bits.  x is clamped at -125 so
// that the result stays a normal number (it is then below 2^-124, nothing beside the
// row maximum's 1).
__device__ __forceinline__ float2 exp2_poly2(float2 x) {
    constexpr float kMagic = 12582912.f;                       // 1.5 * 2^23
    x.x = fmaxf(x.x, -125.f);
    x.y = fmaxf(x.y, -125.f);
    const float2 t = add2(x, make_float2(kMagic, kMagic));
    const float2 j = add2(t, make_float2(-kMagic, -kMagic));
    const float2 r = add2(x, make_float2(-j.x, -j.y));
    float2 p = make_float2(1.3276455e-3f, 1.3276455e-3f);
    p = fma2(p, r, make_float2(9.6755400e-3f, 9.6755400e-3f));
    p = fma2(p, r, make_float2(5.5507135e-2f, 5.5507135e-2f));
    p = fma2(p, r, make_float2(2.4022120e-1f, 2.4022120e-1f));
    p = fma2(p, r, make_float2(6.9314694e-1f, 6.9314694e-1f));
    p = fma2(p, r, make_float2(1.0000001f, 1.0000001f));
    return make_float2(__int_as_float(__float_as_int(p.x) + (__float_as_int(t.x) << 23)),
                       __int_as_float(__float_as_int(p.y) + (__float_as_int(t.y) << 23)));
}

}  // namespace hs2
