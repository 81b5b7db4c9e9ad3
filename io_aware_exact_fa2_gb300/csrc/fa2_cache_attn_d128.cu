// fa2_cache_attn_d128.cu -- fa2_cache_attn for head dimension 128.
#include "fa2_cache_attn.cuh"

namespace fa2 {
namespace cache {

// Query rows of a key/value head: 16 fill one matrix block; more share each key's
// conversion in a block of 32.
fa2_status launch_attn_d128(const AttnArgs &a)
{
    if (static_cast<long long>(a.Lq) * a.G <= 16)
        return launch_attn<AttnCfg<128, 1>>(a);
    return launch_attn<AttnCfg<128, 2>>(a);
}

size_t attn_workspace_d128(long long rows, int num_sms)
{
    return rows <= 16 ? attn_workspace<AttnCfg<128, 1>>(num_sms) : attn_workspace<AttnCfg<128, 2>>(num_sms);
}

}  // namespace cache
}  // namespace fa2
