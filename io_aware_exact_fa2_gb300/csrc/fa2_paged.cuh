// fa2_paged.cuh -- what the kernels of the 16-bit key/value cache and of the position rotation
// (include/fa2_paged.h) share: argument blocks, tensor maps, bf16 and fp16 pairs.  The cache
// itself is the 8-bit one's View without scales, and attention's arguments are its AttnArgs.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "fa2_cache.cuh"
#include "fa2_cache_tile.cuh"
#include "fa2_paged.h"

namespace fa2 {
namespace paged {

using cache::AttnArgs;
using cache::Half;
using cache::View;

struct Rotation {
    const float *cos, *sin;         // [positions, R]
    int positions, R;               // R = 0: none
    int interleaved, inverse;
};

// Rows [B, heads, L, D] that one call moves: where they lie and where they go.
struct Rows {
    const uint16_t *x;
    uint16_t *out;                  // null: into the cache
    long long sb, sh, sl, out_sb, out_sh, out_sl;   // element strides
    int heads;
    int rotated, side;              // turned on the way; cache: 0 keys, 1 values
};

struct MoveArgs {                   // fa2_rope, fa2_paged_append
    View c;                         // (append)
    Rows rows[3];
    int kinds;                      // of rows
    Rotation r;
    const int *starts, *counts;     // may be null: 0, L
    int B, L, D;
};

// A weight is 2^LIFT of the type where its score is the row's reference (a score up to 8 below its
// largest, in the exponent), and UNIT is that number.
// fp16: weights up to 2^14, of which the type keeps those 2^-31 below the largest's.
// bf16 has the range of fp32, in which O is held until it is divided: weights up to 2^-4, so that a row's
// sum stays finite with values of any finite size, unless sum_j exp(s_j - max) |v_j| passes 2^131 (a
// reference past 2^24 may be off by 1: fa2_paged_chunk.cuh), and small ones up to 2^-114 below the
// reference's still count.  (With 6, values of 2^122 made O infinite over one key.)
template <bool F16>
struct Weight {
    static constexpr float LIFT = F16 ? 6.f : -12.f, UNIT = F16 ? 64.f : 1.f / 4096;
};

// Blocks of a move, which a launch counts in an int (of more only where there are few).
long long move_blocks(const MoveArgs &a);
fa2_status launch_move(const MoveArgs &a, bool f16, int num_sms, cudaStream_t stream);
// Head dimension D, 64, 128 or 256 (fa2_paged_attn_d*.cu).
template <int D>
fa2_status launch_attn(const AttnArgs &a, bool f16);
// Workspace bytes for `rows` query rows a key/value head.
template <int D>
size_t attn_workspace_bytes(long long rows, int num_sms);

// A page and head's rows: boxes of `rows` rows by 64 numbers, swizzled over their 128 bytes.
inline bool page_map(cache::EncodeTiled encode, CUtensorMap *m, const Half &x, const View &c, int D, int rows)
{
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), 1ull << c.page_shift, static_cast<cuuint64_t>(c.H),
                                static_cast<cuuint64_t>(c.num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(x.s_slot), static_cast<cuuint64_t>(x.s_head),
                                   static_cast<cuuint64_t>(x.s_page)};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1}, step[4] = {1, 1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, x.codes, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// kind::f16 with fp32 accumulators; operands bf16 or fp16.
__host__ __device__ constexpr uint32_t idesc(bool f16, int m, int n, bool a_mn, bool b_mn)
{
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

#ifdef __CUDACC__
// Two fp32 as a packed pair (round to nearest even), `lo` in bits [0,16).
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    return F16 ? cache::pack_f16x2(lo, hi) : ptx::pack_bf16x2(lo, hi);
}
// ... and back (exact).
template <bool F16>
__device__ __forceinline__ void unpack2(uint32_t w, float &lo, float &hi)
{
    if constexpr (F16) {
        cache::unpack_f16x2(w, lo, hi);
    } else {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xffff0000u);
    }
}
// Bits of a pair that are all ones in an infinity or a NaN.
template <bool F16>
__device__ __forceinline__ uint32_t exponent_bits()
{
    return F16 ? 0x7c007c00u : 0x7f807f80u;
}
// An infinity or NaN in the low, in the high half.
template <bool F16>
__device__ __forceinline__ bool odd_lo(uint32_t w)
{
    return (~w & exponent_bits<F16>() & 0xffffu) == 0;
}
template <bool F16>
__device__ __forceinline__ bool odd_hi(uint32_t w)
{
    return (~w & exponent_bits<F16>() & 0xffff0000u) == 0;
}
// Infinities and NaN as zeros.
template <bool F16>
__device__ __forceinline__ uint32_t finite(uint32_t w)
{
    return w & ((odd_lo<F16>(w) ? 0u : 0xffffu) | (odd_hi<F16>(w) ? 0u : 0xffff0000u));
}
// acc + 0 w: NaN, in one half or the other, once any of the pairs so added holds an infinity or a NaN.
template <bool F16>
__device__ __forceinline__ uint32_t add_odd(uint32_t acc, uint32_t w)
{
    if constexpr (F16)
        asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w), "r"(0));
    else
        asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w), "r"(0));
    return acc;
}
// An infinity or NaN among N quadruples of pairs: at(i) is where quadruple i lies.
template <bool F16, int N, class P>
__device__ __forceinline__ bool any_odd(P at)
{
    uint32_t acc[2] = {};
#pragma unroll
    for (int i0 = 0; i0 < N; i0 += 8) {   // (eight loads under way together)
        uint4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = *reinterpret_cast<const uint4 *>(at(i0 + i));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            acc[i & 1] = add_odd<F16>(add_odd<F16>(acc[i & 1], w[i].x), w[i].y);
            acc[i & 1] = add_odd<F16>(add_odd<F16>(acc[i & 1], w[i].z), w[i].w);
        }
    }
    return odd_lo<F16>(acc[0]) || odd_hi<F16>(acc[0]) || odd_lo<F16>(acc[1]) || odd_hi<F16>(acc[1]);
}
template <bool F16>
__device__ __forceinline__ uint4 finite4(const uint4 &w)
{
    return make_uint4(finite<F16>(w.x), finite<F16>(w.y), finite<F16>(w.z), finite<F16>(w.w));
}
#endif

}  // namespace paged
}  // namespace fa2
