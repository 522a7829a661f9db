// attn8_launch.cuh -- launch of one instance of the attention kernel over a cache in 8 bits, the kernel that splits its
// queries in front and its join behind it.
#pragma once

#include <atomic>

#include "attn8_kernel.cuh"
#include "attn_kernel.cuh"
#include "launch.h"

namespace hsp {

template <int DK, int DV, bool SHARED, int N, int PER_SM>
cudaError_t launch_attn8_variant(const Attn8LaunchReq &r) {
    constexpr int kMaxDev = 64;
    auto kern = hsp_attn8_kernel<DK, DV, SHARED, N, PER_SM>;
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
    e = launch_attn8_queries(r);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attrs[1];
    unsigned n = 0;
    if (r.pdl) {
        attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(r.head_tiles), static_cast<unsigned>(r.args.line.ctas), 1);
    cfg.blockDim = dim3(attn8_threads(N), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(r.smem_bytes);
    cfg.stream = r.stream;
    cfg.attrs = attrs;
    cfg.numAttrs = n;
    e = cudaLaunchKernelEx(&cfg, kern, r.tmap_k, r.tmap_v, r.args);
    if (e != cudaSuccess || !r.args.line.split) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(r.sms * kJoinPerSm), 1, 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, hsp_attn_join_kernel<DV, N>, r.args.line);
}

}  // namespace hsp
