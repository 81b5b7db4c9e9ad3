// fa2_cache_attn_d256.cu -- fa2_cache_attn for head dimension 256.
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
    if (rows <= kFewRows)   // blocks of 16: their accumulators are 128 registers a thread
        return f(AttnCfg<256, 1>{});
    return f(ChunkCfg<256>{});
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

fa2_status launch_attn_d256(const AttnArgs &a)
{
    return dispatch(static_cast<long long>(a.Lq) * a.G, [&](auto c) { return launch(c, a); });
}

size_t attn_workspace_d256(long long rows, int num_sms)
{
    return dispatch(rows, [&](auto c) { return attn_workspace<decltype(c)>(num_sms); });
}

}  // namespace cache
}  // namespace fa2
