// append_common.cuh -- the rotary turn of bf16 pieces and the division by launch constants, shared by the
// kernels that write new tokens into a cache (kernels_append.cu, kernels_append_q8.cu) or read them (kernels_read_q8.cu).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace hsp {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Four interleaved pairs of one piece.
__device__ __forceinline__ uint4 turn_pairs(uint4 v, const float4 c, const float4 s) {
    uint4 o;
    o.x = pack_bf16(bf_lo(v.x) * c.x - bf_hi(v.x) * s.x, bf_hi(v.x) * c.x + bf_lo(v.x) * s.x);
    o.y = pack_bf16(bf_lo(v.y) * c.y - bf_hi(v.y) * s.y, bf_hi(v.y) * c.y + bf_lo(v.y) * s.y);
    o.z = pack_bf16(bf_lo(v.z) * c.z - bf_hi(v.z) * s.z, bf_hi(v.z) * c.z + bf_lo(v.z) * s.z);
    o.w = pack_bf16(bf_lo(v.w) * c.w - bf_hi(v.w) * s.w, bf_hi(v.w) * c.w + bf_lo(v.w) * s.w);
    return o;
}
// Two columns of either half: a (first half) and b (second half).
__device__ __forceinline__ void turn_halves(uint32_t &a, uint32_t &b, float c0, float c1, float s0, float s1) {
    const float a0 = bf_lo(a), a1 = bf_hi(a), b0 = bf_lo(b), b1 = bf_hi(b);
    a = pack_bf16(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
    b = pack_bf16(b0 * c0 + a0 * s0, b1 * c1 + a1 * s1);
}

// n / d for n < 2^31: multiply by floor(2^(32 + s) / d) + 1, s = floor(log2 d), and shift (the
// product is too large by at most n d <= 2^(32 + s), so the quotient is exact); a power of two
// only shifts.
struct FastDiv {
    uint32_t mul, shift;
    explicit FastDiv(int d) {
        shift = 0;
        while (d >> (shift + 1)) ++shift;
        mul = (d & (d - 1)) == 0 ? 0u : static_cast<uint32_t>((1ull << (32 + shift)) / static_cast<uint32_t>(d)) + 1u;
    }
    __device__ __forceinline__ int operator()(int n) const {
        return static_cast<int>(mul ? __umulhi(static_cast<uint32_t>(n), mul) >> shift : static_cast<uint32_t>(n) >> shift);
    }
};

}  // namespace hsp
