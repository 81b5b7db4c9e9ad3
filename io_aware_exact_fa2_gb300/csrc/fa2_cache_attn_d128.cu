// fa2_cache_attn_d128.cu -- fa2_cache_attn for head dimension 128.
#include "fa2_cache_attn.cuh"

namespace fa2 {
namespace cache {

template fa2_status launch_attn<128>(const AttnArgs &a);
template size_t attn_workspace_bytes<128>(long long rows, int num_sms);

}  // namespace cache
}  // namespace fa2
