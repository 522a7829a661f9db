// kernels_attn8_grouped.cu -- attention over a cache in 8 bits of keys and values with 64 or 128 columns per kv head.
#include "attn8_launch.cuh"

namespace hsp {

cudaError_t launch_attn8_grouped(const Attn8LaunchReq &r) {
    if (r.args.line.slots < 4 || r.args.line.slots % 2 != 0) return cudaErrorInvalidConfiguration;
    if (r.DK == 128) {
        if (r.N == 16) return r.per_sm == 3 ? launch_attn8_variant<128, 128, false, 16, 3>(r) : launch_attn8_variant<128, 128, false, 16, 2>(r);
        if (r.N == 32) return launch_attn8_variant<128, 128, false, 32, 2>(r);
        if (r.N == 64) return launch_attn8_variant<128, 128, false, 64, 1>(r);
    } else if (r.DK == 64) {
        if (r.N == 16) return r.per_sm == 3 ? launch_attn8_variant<64, 64, false, 16, 3>(r) : launch_attn8_variant<64, 64, false, 16, 2>(r);
        if (r.N == 32) return launch_attn8_variant<64, 64, false, 32, 2>(r);
        if (r.N == 64) return launch_attn8_variant<64, 64, false, 64, 1>(r);
    }
    return cudaErrorInvalidConfiguration;
}

}  // namespace hsp
