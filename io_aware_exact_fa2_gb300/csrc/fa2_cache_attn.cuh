// fa2_cache_attn.cuh -- fa2_cache_attn for one head dimension: which kernel takes a call.  Each
// fa2_cache_attn_d*.cu instantiates it for a dimension of its own, so that they compile together.
#pragma once

#include "fa2_cache_chunk.cuh"
#include "fa2_cache_step.cuh"

namespace fa2 {
namespace cache {

// f(configuration) for `rows` query rows a key/value head (see kStepRows).
template <int D, class F>
auto for_rows(long long rows, F f)
{
    if (rows <= kStepRows / 2)
        return f(StepCfg<D, 8>{});
    if (rows <= kStepRows)
        return f(StepCfg<D, 16>{});
    return f(ChunkCfg<D>{});
}

template <int D, int R>
fa2_status launch_with(StepCfg<D, R>, const AttnArgs &a)
{
    return launch_step<StepCfg<D, R>>(a);
}
template <int D>
fa2_status launch_with(ChunkCfg<D>, const AttnArgs &a)
{
    return launch_chunk<ChunkCfg<D>>(a);
}

template <int D>
fa2_status launch_attn(const AttnArgs &a)
{
    return for_rows<D>(static_cast<long long>(a.Lq) * a.G, [&](auto c) { return launch_with(c, a); });
}

template <int D>
size_t attn_workspace_bytes(long long rows, int num_sms)
{
    return for_rows<D>(rows, [&](auto c) { return attn_workspace<decltype(c)>(num_sms); });
}

}  // namespace cache
}  // namespace fa2
