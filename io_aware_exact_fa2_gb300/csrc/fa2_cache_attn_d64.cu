// fa2_cache_attn_d64.cu -- fa2_cache_attn for head dimension 64.
#include "fa2_cache_chunk.cuh"
#include "fa2_cache_step.cuh"

namespace fa2 {
namespace cache {

namespace {
template <class F>
auto dispatch(long long rows, F f)
{
    if (rows <= kStepRows / 2)
        return f(StepCfg<64, 8>{});
    if (rows <= kStepRows)
        return f(StepCfg<64, 16>{});
    return f(ChunkCfg<64>{});
}

template <int D, int R>
fa2_status launch(StepCfg<D, R>, const AttnArgs &a)
{
    return launch_step<StepCfg<D, R>>(a);
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
