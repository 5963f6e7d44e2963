// attn_kvq_u4_4.cu -- the attention kernels over Q8_KVQ_U4 caches, up to 4 query heads a block.
#include "attn_kvq.cuh"

namespace q8 {

cudaError_t launch_attn_kvq_u4_4(const AttnParams& p, const LaunchCtx& ctx) {
    return launch_attn_kvq_heads<Q8_KVQ_U4, 1>(p, ctx);
}

}  // namespace q8
