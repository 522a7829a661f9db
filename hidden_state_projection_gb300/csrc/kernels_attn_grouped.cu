// kernels_attn_grouped.cu -- attention over a cache of keys and values with 64 or 128 columns
// per kv head.
#include "attn_launch.cuh"

namespace hsp {

cudaError_t launch_attn_grouped(const AttnLaunchReq &r) {
    if (r.args.slots < 4 || r.args.slots % 2 != 0) return cudaErrorInvalidConfiguration;
    if (r.KB == 2) {
        if (r.N == 16) return launch_attn_variant<2, 2, false, 16>(r);
        if (r.N == 32) return launch_attn_variant<2, 2, false, 32>(r);
        if (r.N == 64) return launch_attn_variant<2, 2, false, 64>(r);
    } else if (r.KB == 1) {
        if (r.N == 16) return launch_attn_variant<1, 1, false, 16>(r);
        if (r.N == 32) return launch_attn_variant<1, 1, false, 32>(r);
        if (r.N == 64) return launch_attn_variant<1, 1, false, 64>(r);
    }
    return cudaErrorInvalidConfiguration;
}

}  // namespace hsp
