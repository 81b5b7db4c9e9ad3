// fa2_cache_tile.cuh -- what the kernels that bring the cache's pages into shared memory by
// TMA share: tensor maps, matrix descriptors, and values as sums of e4m3 terms.
#pragma once

#include <cuda.h>

#include "fa2_cache.cuh"
#include "sm103_ptx.cuh"

namespace fa2 {
namespace cache {

// A page's scales as a loading warp hands them on: key byte, value byte, this bit (0: no page).
constexpr uint32_t PAGE_BIT = 1u << 16;

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled();   // the driver's cuTensorMapEncodeTiled, or null

// Codes of a page and head: boxes of `rows` rows by `row` bytes, swizzled over `row`.
inline bool page_map(EncodeTiled encode, CUtensorMap *m, const Half &x, const View &c, int D, int rows, int row)
{
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), 1ull << c.page_shift, static_cast<cuuint64_t>(c.H),
                                static_cast<cuuint64_t>(c.num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(x.s_slot), static_cast<cuuint64_t>(x.s_head),
                                   static_cast<cuuint64_t>(x.s_page)};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(row), static_cast<cuuint32_t>(rows), 1, 1}, step[4] = {1, 1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, x.codes, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

#ifdef __CUDACC__
// Waits for the phase of parity `parity` of an mbarrier to complete, as a whole warp; false
// (and `code` in *err, first writer wins) when `limit_ns` passes first.  The hint lets the
// hardware suspend the warp for up to 20 us at a time: without one the waits of a kernel whose
// warps each do one part of the work took a third of its issue slots.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, int *err, int code, uint64_t limit_ns)
{
    auto done = [&]() -> bool {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(bar), "r"(parity), "n"(20000)
                     : "memory");
        return __all_sync(0xffffffffu, ok);
    };
    if (done())
        return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!done())
        if (__any_sync(0xffffffffu, ptx::globaltimer_ns() - t0 > limit_ns)) {
            atomicCAS(err, 0, code);
            return false;
        }
    return true;
}

// `bytes` more to come in an mbarrier's present phase, which an arrival has to follow.
__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// N consecutive 32-bit columns of this warp's 32 tensor-memory lanes; valid after the wait.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[4])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
                 "%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[4])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Keeps uses of loaded registers below the wait.
template <int N>
__device__ __forceinline__ void tmem_pin(uint32_t (&r)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+r"(r[i]));
}

// Shared-memory matrix descriptor for rows of 64 bytes swizzled over 64 (layout type 4),
// otherwise as ptx::sdesc_sw128.
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr, uint32_t lbo, uint32_t sbo)
{
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(lbo >> 4 & 0x3FFFu) << 16 |
           static_cast<uint64_t>(sbo >> 4 & 0x3FFFu) << 32 | 1ull << 46 | 4ull << 61;
}

// 1 / x to within 2^-23 of it, also where it is subnormal.
__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Takes the next e4m3 term off an f16 pair: its codes (round to nearest even, saturating),
// and SCALE (16 or 1) times what is left, exactly: the rounding error of four bits' worth of
// eleven.
template <int SCALE>
__device__ __forceinline__ uint32_t take_term(uint32_t &pair)
{
    uint32_t codes, rest;
    asm("{\n\t.reg .b16 c;\n\t.reg .b32 x;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 c, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 x, c;\n\t"
        "sub.rn.f16x2 x, %2, x;\n\t"
        "mul.rn.f16x2 %1, x, %3;\n\t"
        "cvt.u32.u16 %0, c;\n\t}"
        : "=r"(codes), "=r"(rest)
        : "r"(pair), "r"(SCALE == 16 ? 0x4c004c00u : 0x3c003c00u));   // SCALE, SCALE
    pair = rest;
    return codes;
}

#endif

}  // namespace cache
}  // namespace fa2
