// attn_f32.cu -- the attention kernels over f32 caches.
#include "attn.cuh"

namespace q8 {

cudaError_t launch_attn_f32(const AttnParams& p, const LaunchCtx& ctx) {
    return launch_attn_type<Q8_KV_F32>(p, ctx);
}

}  // namespace q8
