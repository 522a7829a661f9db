// attn_launch.cuh -- launch of one instance of the attention kernel and its join.
#pragma once

#include <atomic>

#include "attn_kernel.cuh"
#include "launch.h"

namespace hsp {

template <int KB, int VB, bool SHARED, int N>
cudaError_t launch_attn_variant(const AttnLaunchReq &r) {
    constexpr int kMaxDev = 64;
    auto kern = hsp_attn_kernel<KB, VB, SHARED, N>;
    static std::atomic<uint64_t> configured[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
    if (!set_up_in_current_context(configured[dev])) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
        if (e != cudaSuccess) return e;
        configured[dev].store(current_context_id(), std::memory_order_release);
    }
    cudaLaunchAttribute attrs[1];
    unsigned n = 0;
    if (r.pdl) {
        attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(r.head_tiles), static_cast<unsigned>(r.args.ctas), 1);
    cfg.blockDim = dim3(kAttnThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(r.smem_bytes);
    cfg.stream = r.stream;
    cfg.attrs = attrs;
    cfg.numAttrs = n;
    e = cudaLaunchKernelEx(&cfg, kern, r.tmap_q, r.tmap_k, r.tmap_v, r.args);
    if (e != cudaSuccess || !r.args.split) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(r.sms * kJoinPerSm), 1, 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, hsp_attn_join_kernel<VB * 64, N>, r.args);
}

}  // namespace hsp
