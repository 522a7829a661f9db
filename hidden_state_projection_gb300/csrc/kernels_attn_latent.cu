// kernels_attn_latent.cu -- attention over a latent cache: keys of 576 or 512 columns, the
// first 512 of them the values.
#include "attn_launch.cuh"

namespace hsp {

cudaError_t launch_attn_latent(const AttnLaunchReq &r) {
    if (r.KB == 9) {
        if (r.N == 16) return launch_attn_variant<9, 8, true, 16>(r);
        if (r.N == 32) return launch_attn_variant<9, 8, true, 32>(r);
        if (r.N == 64) return launch_attn_variant<9, 8, true, 64>(r);
    } else if (r.KB == 8) {
        if (r.N == 16) return launch_attn_variant<8, 8, true, 16>(r);
        if (r.N == 32) return launch_attn_variant<8, 8, true, 32>(r);
        if (r.N == 64) return launch_attn_variant<8, 8, true, 64>(r);
    }
    return cudaErrorInvalidConfiguration;
}

}  // namespace hsp
