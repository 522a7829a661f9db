// kernels_attn8_latent.cu -- attention over a latent cache in 8 bits: keys of 576 or 512 columns, the first 512 of them
// the values.
#include "attn8_launch.cuh"

namespace hsp {

cudaError_t launch_attn8_latent(const Attn8LaunchReq &r) {
    if (r.DK == 576) {
        if (r.N == 16) return launch_attn8_variant<576, 512, true, 16, 1>(r);
        if (r.N == 32) return launch_attn8_variant<576, 512, true, 32, 1>(r);
        if (r.N == 64) return launch_attn8_variant<576, 512, true, 64, 1>(r);
    } else if (r.DK == 512) {
        if (r.N == 16) return launch_attn8_variant<512, 512, true, 16, 1>(r);
        if (r.N == 32) return launch_attn8_variant<512, 512, true, 32, 1>(r);
        if (r.N == 64) return launch_attn8_variant<512, 512, true, 64, 1>(r);
    }
    return cudaErrorInvalidConfiguration;
}

}  // namespace hsp
