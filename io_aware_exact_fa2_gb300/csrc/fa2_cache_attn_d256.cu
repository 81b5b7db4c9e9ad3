// fa2_cache_attn_d256.cu -- fa2_cache_attn for head dimension 256.
#include "fa2_cache_attn.cuh"

namespace fa2 {
namespace cache {

// One 16-row block: its accumulators are 128 registers a thread.
fa2_status launch_attn_d256(const AttnArgs &a) { return launch_attn<AttnCfg<256, 1>>(a); }

size_t attn_workspace_d256(long long, int num_sms) { return attn_workspace<AttnCfg<256, 1>>(num_sms); }

}  // namespace cache
}  // namespace fa2
