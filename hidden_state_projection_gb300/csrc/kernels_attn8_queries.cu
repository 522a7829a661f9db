// kernels_attn8_queries.cu -- the queries of an attention over a cache in 8 bits, in two pieces:
//
//   q 2^-e = Qh + Ql / 16,  Qh, Ql e4m3, e of the head: its largest |q| 2^-e is 224 to 448
//
// written as the attention's instructions read them from shared memory (attn8_kernel.cuh): rows in the order of the softmax
// threads' columns, 128 (64) columns to a swizzled line.  A warp takes a head of 512 or 576 columns, two of 128, four of
// 64; two bytes are read and two written per number.  The attention kernel starts as soon as every CTA here has seen the
// kernel before complete, and waits for the images alone: its own start (4.5 us) hides this kernel but for the launch (7 us by
// itself, with cold caches, for 6144 heads of 576 columns, 4.6 for 64).
#include <cuda_bf16.h>

#include "attn8_kernel.cuh"

namespace hsp {

constexpr int kQueryWarps = 4;

template <int DK>
__global__ void __launch_bounds__(32 * kQueryWarps) hsp_attn8_queries_kernel(const __grid_constant__ Attn8QueryArgs a) {
    constexpr int kLanes = DK / 8 < 32 ? DK / 8 : 32, kPer = 32 / kLanes, kRounds = (DK / 8 + kLanes - 1) / kLanes;
    constexpr int kW = DK >= 128 ? 128 : 64, kRope = DK == 576 ? 512 : DK;  // line, first column of the rotary ones
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, sub = lane / kLanes, at = lane % kLanes;
    const int64_t head = (static_cast<int64_t>(blockIdx.x) * kQueryWarps + (threadIdx.x >> 5)) * kPer + sub;
    const int64_t tile = head / a.N;  // of all sequences, kv heads and head tiles
    const int h = static_cast<int>(head - tile * a.N);
    const int64_t pair = tile / a.head_tiles;
    const int ht = static_cast<int>(tile - pair * a.head_tiles);
    const int64_t b = pair / a.kv_heads;
    const int kv = static_cast<int>(pair - b * a.kv_heads);
    const bool there = b < a.batch, real = there && ht * a.N + h < a.group;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + b * a.q_row + (static_cast<int64_t>(kv) * a.group + ht * a.N + h) * a.q_head;
    uint4 v[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int c = (r * kLanes + at) * 8;
        v[r] = make_uint4(0, 0, 0, 0);
        if (real && c < DK) v[r] = *reinterpret_cast<const uint4 *>(q + c);
    }
    __nv_bfloat162 most = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint32_t x[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) most = __hmax2(most, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&x[e])));  // (not NaN)
    }
    float amax = fmaxf(__low2float(most), __high2float(most));
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    if (!there) return;
    // the unit of what is smaller than 2^-118 is 2^-126
    const uint32_t u = __float_as_uint(amax);
    const int e2 = max(-126, min(126, static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0)));
    const float inv = two_to(-e2);
    // row of the head among the instruction's columns: a softmax thread has columns 8 j + 2 c + e of its 16, c its place
    // in four: those are heads 4 c + 2 j + e
    const int row = (h & ~15) + 8 * ((h >> 1) & 1) + 2 * ((h >> 2) & 3) + (h & 1);
    uint8_t *image = a.images + tile * attn8_image_bytes(DK, a.N);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int c = (r * kLanes + at) * 8;
        if (c >= DK) continue;
        const uint32_t x[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // (what is not finite makes its head's scores NaN)
            const float2 y = make_float2(q8_scaled(__uint_as_float(x[e] << 16), inv), q8_scaled(__uint_as_float(x[e] & 0xffff0000u), inv));
            const __half2 z = __floats2half2_rn(y.x, y.y);
            hi[e] = half2_to_e4m3x2(z);
            lo[e] = half2_to_e4m3x2(__hmul2(__hsub2(z, e4m3x2_to_half2(hi[e])), __float2half2_rn(16.f)));
        }
        const bool rope = c >= kRope;
        const int line = rope ? 64 : kW;
        uint8_t *to = rope ? image + 2 * a.N * kRope + row * 64 + swizzled<64>(row, (c - kRope) >> 4) + (c & 8)
                           : image + c / kW * (2 * a.N * kW) + row * kW + swizzled<kW>(row, c % kW >> 4) + (c & 8);
        *reinterpret_cast<uint2 *>(to) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
        *reinterpret_cast<uint2 *>(to + a.N * line) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);  // (N rows on: the same swizzle)
    }
    if (at == 0) image[2 * a.N * DK + h] = static_cast<uint8_t>(e2 + 127);
}

template <int DK>
cudaError_t launch_queries(const Attn8LaunchReq &r) {
    const Attn8QueryArgs &a = r.queries;
    constexpr int kPer = DK >= 256 ? 1 : 256 / DK;
    const int64_t heads = static_cast<int64_t>(a.batch) * a.kv_heads * a.head_tiles * a.N;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((heads + kQueryWarps * kPer - 1) / (kQueryWarps * kPer)), 1, 1);
    cfg.blockDim = dim3(32 * kQueryWarps, 1, 1);
    cfg.stream = r.stream;
    cudaLaunchAttribute attrs[1];
    unsigned n = 0;
    if (r.pdl) {
        attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attrs;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, hsp_attn8_queries_kernel<DK>, a);
}

cudaError_t launch_attn8_queries(const Attn8LaunchReq &r) {
    return r.DK == 576 ? launch_queries<576>(r) : r.DK == 512 ? launch_queries<512>(r) : r.DK == 128 ? launch_queries<128>(r) : launch_queries<64>(r);
}

}  // namespace hsp
