// fa2_cache_attn_d64.cu -- fa2_cache_attn for head dimension 64.
#include "fa2_cache_attn.cuh"

namespace fa2 {
namespace cache {

template fa2_status launch_attn<64>(const AttnArgs &a);
template size_t attn_workspace_bytes<64>(long long rows, int num_sms);

}  // namespace cache
}  // namespace fa2
