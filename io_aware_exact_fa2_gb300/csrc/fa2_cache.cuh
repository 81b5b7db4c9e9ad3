// fa2_cache.cuh -- what the kernels of the 8-bit key/value cache (include/fa2_cache.h)
// share: the cache as they see it, scales and code conversions, argument blocks.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "fa2_cache.h"

namespace fa2 {
namespace cache {

// The cache's keys or its values.  Strides in bytes (a code is a byte).
struct Half {
    uint8_t *codes;
    uint8_t *scale;                 // e8m0 [num_pages, H]
    long long s_page, s_head, s_slot;
};

struct View {
    Half k, v;
    const int *table;               // [B, max_pages]
    int num_pages, H, page_shift;   // page_size = 1 << page_shift
    int B, max_pages;
};

struct MoveArgs {                   // fa2_cache_write, fa2_cache_read
    View c;
    void *x[2];                     // bf16 [B, H, L, D]: keys, values
    long long sb[2], sh[2], sl[2];  // their element strides
    const int *starts, *counts;     // counts may be null: L
    int L, D;
};

// Tests only (FA2_TEST_STALL=2, read on every call): some warps take naps of about half a microsecond,
// the few-row kernel's loading warp before it begins, and, where two warps of the many-row kernel have
// met to exchange a row's largest |q|, the second of the last row tile's.  (A count, and no test of
// it, in the kernels: the many-row one took 387 us instead of 384 with a branch there.)
constexpr int TEST_NAPS = 64;

struct AttnArgs {
    View c;
    const void *q;
    void *o;
    float *lse;
    long long q_sb, q_sh, q_sl, o_sb, o_sh, o_sl;   // element strides
    const int *kv_lens, *q_lens;    // q_lens may be null: Lq
    int Hq, Lq, D;
    int G;                          // query heads a key/value head
    int causal, window;
    float scale;
    void *workspace;
    size_t workspace_bytes;
    int num_sms;
    int *err;                       // device error word
    unsigned long long wait_limit_ns, drain_limit_ns;   // of waits between warps; for a CTA's own copies and products
    int naps;                       // tests only: TEST_NAPS or 0
    cudaStream_t stream;
};

// Blocks of a write or read, which a launch counts in an int.
long long write_blocks(const MoveArgs &a);
long long read_blocks(const MoveArgs &a);
fa2_status launch_write(const MoveArgs &a, cudaStream_t stream);
fa2_status launch_read(const MoveArgs &a, cudaStream_t stream);
// Head dimension D, 64, 128 or 256 (fa2_cache_attn_d*.cu).
template <int D>
fa2_status launch_attn(const AttnArgs &a);
// Workspace bytes for `rows` query rows a key/value head.
template <int D>
size_t attn_workspace_bytes(long long rows, int num_sms);

constexpr int kMinExponent = -96;   // of a scale that fa2_cache_write sets
constexpr int kMaxExponent = 119;   // 448 * 2^119 is the largest finite product in fp32 and bf16

#ifdef __CUDACC__
// 2^n in fp32 for whole n: exact down to the subnormals, infinity above 127.
__device__ __forceinline__ float pow2i(int n)
{
    if (n >= -126)
        return __uint_as_float(n > 127 ? 0x7f800000u : static_cast<uint32_t>(n + 127) << 23);
    return __uint_as_float(n < -149 ? 0u : 0x00400000u >> (-127 - n));
}

// The number an e8m0 byte stands for.
__device__ __forceinline__ float e8m0(uint32_t byte)
{
    return byte == 255 ? __uint_as_float(0x7fc00000u) : pow2i(static_cast<int>(byte) - 127);
}

// Two e4m3 codes in the low 16 bits of w -> packed f16 pair (exact; the NaN code gives NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(r)
        : "r"(w));
    return r;
}

// ... in the high 16 bits.
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
        : "=r"(r)
        : "r"(w));
    return r;
}

__device__ __forceinline__ void unpack_f16x2(uint32_t w, float &lo, float &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.f32.f16 %0, a;\n\t"
        "cvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(w));
}

// Two fp32 -> packed f16 pair (round to nearest even); `lo` lands in bits [0,16).
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// e4m3 NaN codes of four as zeros.
__device__ __forceinline__ uint32_t without_nan(uint32_t w)
{
    const uint32_t nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;   // high bit of each NaN's byte
    return w & ~((nan >> 7) * 0xffu);
}

// Page that entry `j` of sequence b's table names, or -1.
__device__ __forceinline__ int page_of(const View &c, int b, int j)
{
    const int id = c.table[static_cast<long long>(b) * c.max_pages + j];
    return static_cast<unsigned>(id) < static_cast<unsigned>(c.num_pages) ? id : -1;
}
#endif

}  // namespace cache
}  // namespace fa2
