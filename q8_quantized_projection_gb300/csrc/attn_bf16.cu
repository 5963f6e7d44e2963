// attn_bf16.cu -- the attention kernels over bf16 caches.
#include "attn_mma.cuh"

namespace q8 {

cudaError_t launch_attn_bf16(const AttnParams& p, const LaunchCtx& ctx) {
    return launch_attn_16<Q8_KV_BF16>(p, ctx);
}

}  // namespace q8
