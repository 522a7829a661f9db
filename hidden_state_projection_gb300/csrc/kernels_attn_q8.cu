// kernels_attn_q8.cu -- attention of one new token per sequence over a cache held in 8 bits.
//
//   o[b, h] = sum_t p_t vs_t vc_t,  p = softmax_t(scale ks_t q[b, h] . kc_t),  t < len_b
//
// A CTA per sequence and query head; its four warps take the tokens in turn, a lane 16 columns or fewer, with
// the running maximum and sum of a softmax in fp32, and are joined at the end.
#include <cuda_bf16.h>
#include <stdint.h>

#include "append_common.cuh"
#include "cache_args.h"
#include "ptx.cuh"
#include "q8.cuh"

namespace hsp {

template <int DK, int DV>
__global__ void __launch_bounds__(128) hsp_attn_q8_simple_kernel(const __grid_constant__ AttnQ8Args a) {
    constexpr int kK = DK / 32, kV = DV / 32;
    __shared__ float acc_s[4][DV];
    __shared__ float m_s[4], l_s[4];
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x, b = blockIdx.y, heads = a.kv_heads * a.group, kvh = h / a.group;
    const int row = a.rows ? a.rows[b] : b;
    const bool row_ok = row >= 0 && row < a.num_rows;
    int len = row_ok ? a.lens[row] : 0;
    const int most = a.max_pages << a.page_shift;
    if ((!row_ok || len < 0 || len > most) && threadIdx.x == 0) atomicCAS(a.err_word, 0, kDeviceErrIndex);
    len = min(max(len, 0), most);
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + b * a.q_row + h * a.q_head;
    float qv[kK], acc[kV];
#pragma unroll
    for (int k = 0; k < kK; ++k) qv[k] = __bfloat162float(q[k * 32 + lane]) * a.scale_log2;
#pragma unroll
    for (int k = 0; k < kV; ++k) acc[k] = 0.f;
    float m = -3.0e38f, l = 0.f;
    const Q8Side &vs = a.v.codes ? a.v : a.k;
    for (int t = warp; t < len; t += 4) {
        int page = a.table[row * a.table_stride + (t >> a.page_shift)];
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) atomicCAS(a.err_word, 0, kDeviceErrIndex);
            page = 0;
        }
        const int line = t & ((1 << a.page_shift) - 1), blk = line >> a.block_shift;
        const uint8_t *kc = a.k.codes + page * a.k.page + line * a.k.token + kvh * a.k.head;
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kK; ++k) s += qv[k] * __low2float(e4m3x2_to_half2(kc[k * 32 + lane]));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.k.scales[page * a.k.s_page + blk * a.k.s_block + kvh * a.k.s_head];
        const float vscale = vs.scales[page * vs.s_page + blk * vs.s_block + kvh * vs.s_head];
        const float n = fmaxf(m, s), f = exp2f(m - n), p = exp2f(s - n);
        m = n;
        l = l * f + p;
        const uint8_t *vc = vs.codes + page * vs.page + line * vs.token + kvh * vs.head;
#pragma unroll
        for (int k = 0; k < kV; ++k) acc[k] = acc[k] * f + p * vscale * __low2float(e4m3x2_to_half2(vc[k * 32 + lane]));
    }
#pragma unroll
    for (int k = 0; k < kV; ++k) acc_s[warp][k * 32 + lane] = acc[k];
    if (lane == 0) {
        m_s[warp] = m;
        l_s[warp] = l;
    }
    __syncthreads();
    float M = -3.0e38f, L = 0.f;
    for (int w = 0; w < 4; ++w) M = fmaxf(M, m_s[w]);
    for (int w = 0; w < 4; ++w) L += l_s[w] * exp2f(m_s[w] - M);
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + (static_cast<int64_t>(b) * heads + h) * DV;
    for (int c = threadIdx.x; c < DV; c += 128) {
        float o = 0.f;
        for (int w = 0; w < 4; ++w) o += acc_s[w][c] * exp2f(m_s[w] - M);
        out[c] = __float2bfloat16_rn(len > 0 ? o / L : 0.f);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[static_cast<int64_t>(b) * heads + h] = len > 0 ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
    cta_release_and_trigger();
}

cudaError_t launch_attn_q8_simple(const AttnQ8Args &a, int pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.kv_heads * a.group), static_cast<unsigned>(a.batch), 1);
    cfg.blockDim = dim3(128, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attrs[1];
    unsigned n = 0;
    if (pdl) {
        attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attrs;
    cfg.numAttrs = n;
    if (a.k.dim == 576) return cudaLaunchKernelEx(&cfg, hsp_attn_q8_simple_kernel<576, 512>, a);
    if (a.k.dim == 512) return cudaLaunchKernelEx(&cfg, hsp_attn_q8_simple_kernel<512, 512>, a);
    if (a.k.dim == 128) return cudaLaunchKernelEx(&cfg, hsp_attn_q8_simple_kernel<128, 128>, a);
    if (a.k.dim == 64) return cudaLaunchKernelEx(&cfg, hsp_attn_q8_simple_kernel<64, 64>, a);
    return cudaErrorInvalidConfiguration;
}

}  // namespace hsp
