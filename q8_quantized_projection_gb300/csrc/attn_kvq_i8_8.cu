// attn_kvq_i8_8.cu -- the attention kernels over Q8_KVQ_I8 caches, up to 8 query heads a block.
#include "attn_kvq.cuh"

namespace q8 {

cudaError_t launch_attn_kvq_i8_8(const AttnParams& p, const LaunchCtx& ctx) {
    return launch_attn_kvq_heads<Q8_KVQ_I8, 2>(p, ctx);
}

}  // namespace q8
