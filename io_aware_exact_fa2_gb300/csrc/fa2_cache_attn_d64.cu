// fa2_cache_attn_d64.cu -- fa2_cache_attn for head dimension 64.
#include "fa2_cache_attn.cuh"

namespace fa2 {
namespace cache {

// Query rows of a key/value head: 16 fill one matrix block; more share each key's
// conversion in a block of 32.
fa2_status launch_attn_d64(const AttnArgs &a)
{
    if (static_cast<long long>(a.Lq) * a.G <= 16)
        return launch_attn<AttnCfg<64, 1>>(a);
    return launch_attn<AttnCfg<64, 2>>(a);
}

size_t attn_workspace_d64(long long rows, int num_sms)
{
    return rows <= 16 ? attn_workspace<AttnCfg<64, 1>>(num_sms) : attn_workspace<AttnCfg<64, 2>>(num_sms);
}

}  // namespace cache
}  // namespace fa2
