// fa2_cache_attn_d64.cu -- fa2_cache_attn for head dimension 64.
#include "fa2_cache_attn.cuh"
#include "fa2_cache_chunk.cuh"

namespace fa2 {
namespace cache {

namespace {
// Query rows of a key/value head up to which a step's kernel takes them.
constexpr long long kFewRows = 32;

template <class F>
auto dispatch(long long rows, F f)
{
    if (rows <= 16)   // one matrix block; more share each key's conversion in two
        return f(AttnCfg<64, 1>{});
    if (rows <= kFewRows)
        return f(AttnCfg<64, 2>{});
    return f(ChunkCfg<64>{});
}

template <int D, int MT>
fa2_status launch(AttnCfg<D, MT>, const AttnArgs &a)
{
    return launch_attn<AttnCfg<D, MT>>(a);
}
template <int D>
fa2_status launch(ChunkCfg<D>, const AttnArgs &a)
{
    return launch_chunk<ChunkCfg<D>>(a);
}
}  // namespace

fa2_status launch_attn_d64(const AttnArgs &a)
{
    return dispatch(static_cast<long long>(a.Lq) * a.G, [&](auto c) { return launch(c, a); });
}

size_t attn_workspace_d64(long long rows, int num_sms)
{
    return dispatch(rows, [&](auto c) { return attn_workspace<decltype(c)>(num_sms); });
}

}  // namespace cache
}  // namespace fa2
