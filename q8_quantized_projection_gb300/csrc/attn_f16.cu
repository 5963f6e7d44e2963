// attn_f16.cu -- the attention kernels over f16 caches.
#include "attn_mma.cuh"

namespace q8 {

cudaError_t launch_attn_f16(const AttnParams& p, const LaunchCtx& ctx) {
    return launch_attn_16<Q8_KV_F16>(p, ctx);
}

}  // namespace q8
