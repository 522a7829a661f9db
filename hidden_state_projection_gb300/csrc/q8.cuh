// q8.cuh -- the 8-bit numbers of a quantised cache: e4m3 codes under a scale that is a power of two.
//
//   value = code * scale;  e4m3: 1 sign, 4 exponent, 3 mantissa bits, largest 448, no infinities, one NaN (0x7f)
//
// Scales go from 2^-60 to 2^60.  A value counts for its block's scale if it is at most 448 * 2^60; what is
// larger, infinite or NaN is stored as NaN.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "packed.cuh"

namespace hsp {

constexpr int kQ8MinExp = -60, kQ8MaxExp = 60;
constexpr float kQ8Top = 448.f;

// Two e4m3 codes as fp16 (exact: e4m3 has fewer bits of either kind).
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(codes));
    return *reinterpret_cast<const __half2 *>(&r);
}
// Rounded to the nearest e4m3 value, ties to the even code; `lo` in bits 0-7.  (NaN gives NaN; callers keep |x| <= 448.)
__device__ __forceinline__ uint32_t float2_to_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f32 c, %2, %1;\n\tcvt.u32.u16 %0, c;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
// x * inv as a code's float: NaN where it is out of the codes' range.
__device__ __forceinline__ float q8_scaled(float x, float inv) {
    const float y = x * inv;
    return fabsf(y) <= kQ8Top ? y : __uint_as_float(0x7fc00000u);
}

__device__ __forceinline__ float two_to(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // -126 .. 127

// Smallest e in -60 .. 60 with amax <= 448 * 2^e (amax >= 0, at most 448 * 2^60): 448 = 1.75 * 2^8.
__device__ __forceinline__ int q8_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(kQ8MinExp, min(kQ8MaxExp, e));
}

// x * s cut off to fp32 and, where something was cut off, its last bit set (rounded to odd): the rounding to fewer bits behind it is that of
// the exact product.
__device__ __forceinline__ float product_odd(float x, float s) {
    const float p = __fmul_rz(x, s);
    return __uint_as_float(__float_as_uint(p) | (__fmaf_rn(x, s, -p) != 0.f ? 1u : 0u));
}

// a c + b d rounded to odd, two at a time: floats whose last bits say whether something was cut off, so that the rounding to
// a code (which is shorter by far) is that of the exact sum.  The products' errors and the sum's are found with fused
// multiply-adds and the two-sum of Knuth (a few bits beyond 2^-70 of the larger product aside).
__device__ __forceinline__ float odd(float h, float l) {
    uint32_t u = __float_as_uint(h);
    if ((l > 0.f || l < 0.f) && (u & 1u) == 0) u = (l > 0.f) == (h > 0.f) ? u + 1 : u - 1;
    return __uint_as_float(u);
}
__device__ __forceinline__ float2 dot2_odd(float2 a, float2 c, float2 b, float2 d) {
    const float2 p = mul2(a, c), q = mul2(b, d);
    const float2 ep = fma2(a, c, make_float2(-p.x, -p.y)), eq = fma2(b, d, make_float2(-q.x, -q.y));
    const float2 s = sum2(p, q);
    const float2 bb = sub2(s, p);
    const float2 es = sum2(sub2(p, sub2(s, bb)), sub2(q, bb));
    const float2 rest = sum2(es, sum2(ep, eq));
    const float2 h = sum2(s, rest);
    const float2 l = sub2(rest, sub2(h, s));
    return make_float2(odd(h.x, l.x), odd(h.y, l.y));
}

}  // namespace hsp
