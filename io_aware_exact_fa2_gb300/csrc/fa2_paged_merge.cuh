// fa2_paged_merge.cuh -- the parts of a row whose keys several CTAs share (fa2_paged_line.cuh),
// put together: fa2_paged_step.cuh and fa2_paged_chunk.cuh.  (The 8-bit cache's merge_row, in
// fa2_cache_line.cuh, is this one with parts that carry their log2-sum-exp2 as two floats: what is
// mended in one is to be looked at in the other.)
//
// A part says what it computed as O / l and two floats: M, a score as the products gave it, and
// y = log2 of the sum of 2^((S - M) c).  Scores stay scores: a difference of two M times c is exact
// where it matters, whatever their size, where M c as a float would be off by 2^-24 of it, 2^19 at
// scores of 2^43.  Parts count by weights of the same size as a key's (Weight::UNIT).
#pragma once

#include "fa2_cache_line.cuh"
#include "fa2_paged.cuh"

namespace fa2 {
namespace paged {

#ifdef __CUDACC__
constexpr float NONE = -3.402823466e38f;   // M of nothing: no finite score lies below it

// log2 of the sum of a row's exponentials.
__device__ __forceinline__ float log2_sum(float M, float c, float y)
{
    const float top = __fmul_rn(M, c);
    return top + (fmaf(M, c, -top) + y);
}

// Merges what ranges c0 .. c1 computed of N quadruples of one row of a unit, always in that
// order: place(k) is quadruple k's offset in a slot.  Returns the row's log2-sum-exp2.  (One
// pass, W parts at a time, so that their loads are under way together.)
template <class C, int N, int W, class P>
__device__ __forceinline__ float merge_row(const cache::Parts &parts, float c, int c0, int c1, int row, P place, float4 (&v)[N])
{
    const size_t slot_floats = cache::Parts::slot_floats(C::R, C::D);
    auto slot = [&](int i) { return parts.data + (2 * static_cast<size_t>(i) + (i == c0 ? 1 : 0)) * slot_floats; };
    float top = NONE, l = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k)
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i = c0; i <= c1; i += W) {
        float2 sum[W];
        float4 x[W][N];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const bool there = i + w <= c1;
            const float *const s = slot(i + w);
            sum[w] = there ? __ldcg(reinterpret_cast<const float2 *>(s + C::R * C::D) + row) : make_float2(NONE, -INFINITY);
#pragma unroll
            for (int k = 0; k < N; ++k)
                x[w][k] = there ? __ldcg(reinterpret_cast<const float4 *>(s + place(k))) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float before = top;
#pragma unroll
        for (int w = 0; w < W; ++w)
            top = fmaxf(top, sum[w].x);
        const float f = ptx::ex2_approx((before - top) * c);
        l *= f;
#pragma unroll
        for (int k = 0; k < N; ++k)
            v[k].x *= f, v[k].y *= f, v[k].z *= f, v[k].w *= f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float g = ptx::ex2_approx(fmaf(sum[w].x - top, c, sum[w].y)) * Weight<C::F16>::UNIT;
            l += g;
#pragma unroll
            for (int k = 0; k < N; ++k)
                v[k].x += x[w][k].x * g, v[k].y += x[w][k].y * g, v[k].z += x[w][k].z * g, v[k].w += x[w][k].w * g;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int k = 0; k < N; ++k)
        v[k].x *= inv, v[k].y *= inv, v[k].z *= inv, v[k].w *= inv;
    return l == 0.f ? -INFINITY : log2_sum(top, c, ptx::lg2_approx(l * (1.f / Weight<C::F16>::UNIT)));
}
#endif

}  // namespace paged
}  // namespace fa2
