// attn_kvq.cu -- the choice of kernel for attention over quantised caches.
#include "attn_kvq.cuh"

namespace q8 {

cudaError_t launch_attn_kvq(const AttnParams& p, const LaunchCtx& ctx) {
    if (p.a.kv_type == kKvQuantised + Q8_KVQ_I8) return launch_attn_kvq_kind<Q8_KVQ_I8>(p, ctx);
    return launch_attn_kvq_kind<Q8_KVQ_U4>(p, ctx);
}

}  // namespace q8
