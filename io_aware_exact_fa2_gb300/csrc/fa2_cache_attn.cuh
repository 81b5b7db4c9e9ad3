// fa2_cache_attn.cuh -- attention of a few query rows over the paged e4m3 cache
// (fa2_cache_attn in include/fa2_cache.h), for one head dimension.
//
// Mathematics.  The query heads that share a key/value head and the query tokens of a
// sequence are the rows of one small matrix: row r is token r / G, head r % G of the
// group, so a cache byte is read once for all of them.  For a block of R = 16 or 32
// rows a warp takes 16 keys at a time:
//     S = Q K^T            mma.sync m16n8k16, f16 operands, fp32 sums
//     x = S * scale * log2 e * 2^ek          (ek: the page's key exponent)
//     p = 2^(x - m),  l += sum p             m: running maximum of x
//     O += (p 2^(m + ev - M + 6)) V          M: running maximum of x + ev
// A code is exact in f16, and so is a bf16 row of Q once it is multiplied by a power
// of two that puts its largest magnitude in [2^14, 2^15).  The weights of V carry the
// value scale's exponent ev and have a reference M of their own, so pages of any
// strength meet in one accumulator and a weight loses bits only 2^-20 below the
// largest |p 2^ev| seen (f16 subnormals); l is fp32 throughout.  m and M are raised
// only when a chunk exceeds them by more than 2^8 (exact: all terms use the same m, M).
//
// What bounds it.  One token of a group of 8 does 16 operations a cache byte: the card
// could do 290, so the cache's bytes are the time.  Hence: every warp streams its own
// 16-key chunks through a private ring of cp.async stages (no barrier in the loop),
// codes go from shared memory straight into the matrix instructions' register layout
// (d and key orders are permuted to make every shared load 16 bytes a lane), and the
// keys of all sequences, heads and row blocks are one line of 64-key tiles that is cut
// into equal ranges, one for each CTA.  A block of rows cut by a range's end is
// computed in parts; the CTA that finishes last merges them, always in key order.
#pragma once

#include <atomic>

#include "fa2_cache_line.cuh"
#include "sm103_ptx.cuh"

namespace fa2 {
namespace cache {

template <int D_, int MT_>
struct AttnCfg {
    static constexpr int D = D_;
    static constexpr int MT = MT_;                   // 16-row blocks of query rows
    static constexpr int R = 16 * MT;                // query rows of a unit
    static constexpr int NW = 4;                     // warps
    static constexpr int T = 32 * NW;
    static constexpr int TILE = CHUNK * NW;          // keys
    static constexpr int CTAS = 2;                   // an SM
    // stages of 16 keys and values: 96 KB a CTA (64 KB at D = 64)
    static constexpr int ST = D == 64 ? 8 : D == 128 ? 6 : 3;
    static constexpr int STAGE_BYTES = 2 * CHUNK * D;
    static constexpr int RING_BYTES = ST * STAGE_BYTES;      // one warp's
    static constexpr int SMEM_BYTES = NW * RING_BYTES;
    static_assert(RING_BYTES >= R * D * 4, "a warp's partial O lies in its ring");
};

#ifdef __CUDACC__

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes global -> shared; `bytes` 0 fills the 16 with zeros and reads nothing.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float quad_max(float v)
{
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v)
{
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// Where a 16-byte column of a chunk's row lies in the chunk: lines of 128 bytes hold
// one row (D = 128), two (64) or half of one (256); the column is XORed within its
// line so that the lanes of one shared load meet all banks.
//   K: eight rows and four neighbouring columns a load (lanes 4 g + t: row g, column t)
//   V: rows 2t, columns g (D = 64: halves of columns g / 2)
template <int D, bool V>
__device__ __forceinline__ uint32_t chunk_offset(int row, int col)
{
    if (D == 64) {
        const int line = row >> 1, c = ((row & 1) << 2) | col;
        return line * 128 + ((c ^ (V ? (line & 3) << 1 : 0)) << 4);
    }
    const int line = D == 128 ? row : row * 2 + (col >> 3);
    const int x = V ? row & 6 : ((row & 1) << 2) | ((row >> 1) & 3);
    return line * 128 + (((col & 7) ^ x) << 4);
}

// Everything a warp knows of its rows: row mt * 16 + g + 8 * half of the unit for
// the lane 4 g + t.
template <class C>
struct Rows {
    uint32_t q[C::MT][C::D / 16][4];   // A fragments
    int e[C::MT][2];                   // Q was multiplied by 2^-e
    int hi[C::MT][2], lo[C::MT][2];    // keys lo <= j < hi are visible
    float m[C::MT][2], M[C::MT][2], l[C::MT][2];
    float o[C::MT][C::D / 8][4];
};

template <class C>
__device__ __forceinline__ void load_rows(Rows<C> &w, const AttnArgs &a, const Seq &s, int b, int h, int rb, int g, int t)
{
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = rb * C::R + mt * 16 + half * 8 + g;
            const bool live = r < s.n * a.G;
            const int i = r / a.G, hq = h * a.G + r % a.G;
            const int pos = s.kv - s.n + i;
            w.hi[mt][half] = !live ? 0 : a.causal ? pos + 1 : s.kv;
            const long long lo = static_cast<long long>(pos) - a.window;
            w.lo[mt][half] = a.window >= 0 && lo > 0 ? static_cast<int>(lo) : 0;
            w.m[mt][half] = w.M[mt][half] = -INFINITY;
            w.l[mt][half] = 0.f;
            const uint16_t *q = static_cast<const uint16_t *>(a.q) + b * a.q_sb + hq * a.q_sh + i * a.q_sl;
            uint32_t raw[C::D / 64][8];
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < C::D / 64; ++c) {
                uint4 x = make_uint4(0, 0, 0, 0), y = x;
                if (live) {
                    x = __ldg(reinterpret_cast<const uint4 *>(q + c * 64 + t * 16));
                    y = __ldg(reinterpret_cast<const uint4 *>(q + c * 64 + t * 16) + 1);
                }
                raw[c][0] = x.x, raw[c][1] = x.y, raw[c][2] = x.z, raw[c][3] = x.w;
                raw[c][4] = y.x, raw[c][5] = y.y, raw[c][6] = y.z, raw[c][7] = y.w;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t u = raw[c][k] & 0x7fffu, v = (raw[c][k] >> 16) & 0x7fffu;
                    top = top > u ? top : u;
                    top = top > v ? top : v;
                }
            }
            uint32_t other = __shfl_xor_sync(0xffffffffu, top, 1);
            top = top > other ? top : other;
            other = __shfl_xor_sync(0xffffffffu, top, 2);
            top = top > other ? top : other;
            // a row with an infinity or NaN has no finite scores: make it NaN
            int e = static_cast<int>(top >> 7) - 127 - 14;
            e = e < -126 ? -126 : e;   // 2^126 is as far as fp32 goes (zero and subnormal rows)
            w.e[mt][half] = e;
            const float f = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : pow2i(-e);
#pragma unroll
            for (int c = 0; c < C::D / 64; ++c)
#pragma unroll
                for (int k = 0; k < 8; ++k)   // step c * 4 + k / 2; its first or second pair of d
                    w.q[mt][c * 4 + k / 2][half + 2 * (k & 1)] =
                        pack_f16x2(__uint_as_float(raw[c][k] << 16) * f, __uint_as_float(raw[c][k] & 0xffff0000u) * f);
        }
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
        for (int j = 0; j < C::D / 8; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w.o[mt][j][k] = 0.f;
}

// A value chunk's NaN codes, in a chunk that some rows see in part: the product below
// would carry them (0 * NaN) into rows that do not see their keys.  They are replaced
// by zeros for the product, and this puts the NaN into the rows that do see them.
template <class C>
__device__ __forceinline__ void nan_values(Rows<C> &w, const uint8_t *v, int pos0, int t)
{
#pragma unroll 1
    for (int key = 0; key < CHUNK; ++key)
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int j = pos0 + key;
                if (j < w.lo[mt][half] || j >= w.hi[mt][half])
                    continue;
#pragma unroll
                for (int n = 0; n < C::D / 8; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        // the d of accumulator column 2t + k of n-tile n (see the product with V)
                        const int g = 2 * t + k;
                        const int d = C::D == 64 ? 8 * g + n : (n >> 4) * 128 + 16 * g + (n & 15);
                        if ((v[chunk_offset<C::D, true>(key, d >> 4) + (d & 15)] & 0x7f) == 0x7f)
                            w.o[mt][n][half * 2 + k] = __uint_as_float(0x7fc00000u);
                    }
            }
}

// 16 keys and values in shared memory, at positions pos0 .. pos0 + 15.
template <class C>
__device__ __forceinline__ void consume(Rows<C> &w, uint32_t kv, const uint8_t *v_ptr, int pos0, bool whole, int ek, int ev,
                                        float scale_log2, int g, int t)
{
    constexpr int D = C::D, MT = C::MT;
    const bool nan_scale = ev == 128;   // (that of the keys: below)
    ev = nan_scale ? 0 : ev;
    float s[MT][2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                s[mt][nt][k] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            uint32_t k[4];
            ptx::ld_shared_v4(kv + chunk_offset<D, false>(nt * 8 + g, c * 4 + t), k[0], k[1], k[2], k[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t b0 = e4m3x2_to_f16x2(k[i]), b1 = e4m3x2_hi_to_f16x2(k[i]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    mma_f16(s[mt][nt], w.q[mt][c * 4 + i], b0, b1);
            }
        }
    }
    // scores in log2 units, masked
    float top[MT][2];
    bool raise = false;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float f = ek == 128 ? __uint_as_float(0x7fc00000u) : scale_log2 * pow2i(w.e[mt][half] + ek);
            float x = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float &y = s[mt][nt][half * 2 + k];
                    y *= f;
                    if (!whole) {
                        const int j = pos0 + nt * 8 + 2 * t + k;
                        y = j >= w.lo[mt][half] && j < w.hi[mt][half] ? y : -INFINITY;
                    }
                    x = fmaxf(x, y);
                }
            x = quad_max(x);
            top[mt][half] = x;
            raise |= x > w.m[mt][half] + 8.f || x + ev > w.M[mt][half] + 8.f;
        }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float x = top[mt][half];
                if (x > w.m[mt][half] + 8.f) {
                    w.l[mt][half] *= ptx::ex2_approx(w.m[mt][half] - x);
                    w.m[mt][half] = x;
                }
                float f = 1.f;
                if (x + ev > w.M[mt][half] + 8.f) {
                    f = ptx::ex2_approx(w.M[mt][half] - (x + ev));
                    w.M[mt][half] = x + ev;
                }
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    w.o[mt][j][half * 2] *= f;
                    w.o[mt][j][half * 2 + 1] *= f;
                }
            }
    }
    // weights
    uint32_t p[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float m = w.m[mt][half] == -INFINITY ? 0.f : w.m[mt][half];
            const float M = w.M[mt][half] == -INFINITY ? 0.f : w.M[mt][half];
            const float f = ptx::ex2_approx(fminf(m + ev - M + 6.f, 127.f));
            float y[2][2], sum = 0.f;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    y[nt][k] = ptx::ex2_approx(s[mt][nt][half * 2 + k] - m);
                    sum += y[nt][k];
                }
            w.l[mt][half] += sum;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
                p[mt][half + 2 * nt] = pack_f16x2(y[nt][0] * f, y[nt][1] * f);
        }
    // O += P V: lane 4 g + t holds keys 2t, 2t + 1, 2t + 8, 2t + 9 and, as column g of
    // n-tile j, d = 16 g + j of each 128 (8 g + j at D = 64)
    constexpr int W = D == 64 ? 2 : 4;   // words of four d a lane reads of a row
    bool nan = false;
#pragma unroll
    for (int c = 0; c < (D == 256 ? 2 : 1); ++c) {
        uint32_t v[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = 2 * t + (k & 1) + (k >> 1) * 8;
            if (D == 64) {
                const uint32_t at = kv + CHUNK * D + chunk_offset<D, true>(row, g >> 1) + (g & 1) * 8;
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[k][0]), "=r"(v[k][1]) : "r"(at) : "memory");
            } else {
                ptx::ld_shared_v4(kv + CHUNK * D + chunk_offset<D, true>(row, c * 8 + g), v[k][0], v[k][1], v[k][2],
                                  v[k][3]);
            }
            if (!whole)
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const uint32_t z = without_nan(v[k][i]);
                    nan |= z != v[k][i];
                    v[k][i] = z;
                }
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
            // pairs of keys for each of four d
            const uint32_t a01 = __byte_perm(v[0][i], v[1][i], 0x5140), a23 = __byte_perm(v[0][i], v[1][i], 0x7362);
            const uint32_t b01 = __byte_perm(v[2][i], v[3][i], 0x5140), b23 = __byte_perm(v[2][i], v[3][i], 0x7362);
            const uint32_t b0[4] = {e4m3x2_to_f16x2(a01), e4m3x2_hi_to_f16x2(a01), e4m3x2_to_f16x2(a23),
                                    e4m3x2_hi_to_f16x2(a23)};
            const uint32_t b1[4] = {e4m3x2_to_f16x2(b01), e4m3x2_hi_to_f16x2(b01), e4m3x2_to_f16x2(b23),
                                    e4m3x2_hi_to_f16x2(b23)};
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    mma_f16(w.o[mt][c * 16 + i * 4 + d], p[mt], b0[d], b1[d]);
        }
    }
    if (!whole && __any_sync(0xffffffffu, nan))
        nan_values<C>(w, v_ptr, pos0, t);
    if (nan_scale)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half)
                if (w.lo[mt][half] < pos0 + CHUNK && w.hi[mt][half] > pos0)   // the row sees one of the keys
#pragma unroll
                    for (int j = 0; j < D / 8; ++j)
                        w.o[mt][j][half * 2] = w.o[mt][j][half * 2 + 1] = __uint_as_float(0x7fc00000u);
}

// Where the D / 4 four-float units of a row lie in a warp's partial O [R, D]: the lanes
// that store (row g, 32 or 16 consecutive d each) meet all banks.
template <int D>
__device__ __forceinline__ int unit_offset(int row, int u)
{
    if (D == 64) {
        const int blk = row * 4 + (u >> 2);
        return blk * 4 + ((u & 3) ^ ((blk >> 1) & 3));
    }
    return row * (D / 4) + (u & ~7) + ((u & 7) ^ (((u >> 3) & 3) | ((row & 1) << 2)));
}

template <class C>
__global__ void __launch_bounds__(C::T, C::CTAS) attn_kernel(const AttnArgs a, const Parts parts)
{
    constexpr int D = C::D, R = C::R, NW = C::NW, ST = C::ST;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LineShared sh_line;
    __shared__ float sh_m[NW][R], sh_l[NW][R];
    __shared__ float sh_lse[R];
    __shared__ int sh_last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const bool cut = parts.data != nullptr;
    const int cta = blockIdx.x;
    Range range;
    long long first, end;
    Line<C> line;
    if (!find_range<C>(a, cut, sh_line, range, first, end, line))
        return;

    const uint32_t ring = ptx::smem_u32(smem) + warp * C::RING_BYTES;
    uint8_t *const ring_ptr = smem + warp * C::RING_BYTES;
    float *const mine_o = reinterpret_cast<float *>(ring_ptr);
    const float scale_log2 = a.scale * 1.4426950408889634f;
    Rows<C> w;

    for (;;) {
        const int b = line.b, h = line.h, rb = line.rb;
        const Seq s = line.s;
        const Span span = line.span;
        const int tile0 = cut && first > line.at ? static_cast<int>(first - line.at) : 0;
        const int tile1 = cut && end < line.at + span.tiles ? static_cast<int>(end - line.at) : span.tiles;
        load_rows<C>(w, a, s, b, h, rb, g, t);
        int all_lo, all_hi;
        line.seen_by_all(a, all_lo, all_hi);
        const int from = span.lo & ~(CHUNK - 1);
        // this warp's chunks: number k at position chunk0 + k * TILE
        const int chunk0 = from + tile0 * C::TILE + warp * CHUNK;
        const int stop = from + tile1 * C::TILE < span.hi ? from + tile1 * C::TILE : span.hi;
        const int n = stop > chunk0 ? (stop - chunk0 + C::TILE - 1) / C::TILE : 0;

        // Pages and scales of 32 chunks at a time, one a lane: the table's entries are
        // loaded a batch ahead, the scales when their batch begins to be copied.
        auto table_batch = [&](int k) {
            const int pos = chunk0 + (k + lane) * C::TILE;
            return k + lane < n ? page_of(a.c, b, pos >> a.c.page_shift) : -1;
        };
        auto scale_batch = [&](int id) -> uint32_t {   // 0: no page
            if (id < 0)
                return 0;
            const long long i = static_cast<long long>(id) * a.c.H + h;
            return a.c.k.scale[i] | static_cast<uint32_t>(a.c.v.scale[i]) << 8 | 1u << 16;
        };
        int id_now = table_batch(0), id_next = table_batch(32);
        uint32_t sc_new = scale_batch(id_now), sc_now = sc_new;

        auto issue = [&](int k) {
            if (k > 0 && (k & 31) == 0) {
                id_now = id_next;
                sc_new = scale_batch(id_now);
                id_next = table_batch(k + 32);
            }
            const int id = __shfl_sync(0xffffffffu, id_now, k & 31);
            if (k < n && id >= 0) {
                const int pos = chunk0 + k * C::TILE, slot = pos & ((1 << a.c.page_shift) - 1);
                const uint32_t dst = ring + (k % ST) * C::STAGE_BYTES;
                const uint8_t *kp = a.c.k.codes + id * a.c.k.s_page + h * a.c.k.s_head + slot * a.c.k.s_slot;
                const uint8_t *vp = a.c.v.codes + id * a.c.v.s_page + h * a.c.v.s_head + slot * a.c.v.s_slot;
                constexpr int COLS = D / 16, STEP = 32 / COLS;
                const int col = lane % COLS;
#pragma unroll
                for (int i = 0; i < CHUNK / STEP; ++i) {
                    const int row = lane / COLS + i * STEP;
                    // rows that no query of the block sees are zeros
                    const int bytes = pos + row >= span.lo && pos + row < span.hi ? 16 : 0;
                    cp_async16(dst + chunk_offset<D, false>(row, col), kp + row * a.c.k.s_slot + col * 16, bytes);
                    cp_async16(dst + CHUNK * D + chunk_offset<D, true>(row, col), vp + row * a.c.v.s_slot + col * 16, bytes);
                }
            }
            cp_async_commit();
        };
        for (int k = 0; k < ST - 1; ++k)
            issue(k);
        for (int k = 0; k < n; ++k) {
            cp_async_wait<ST - 2>();
            __syncwarp();
            if (k > 0 && (k & 31) == 0)
                sc_now = sc_new;
            issue(k + ST - 1);
            const uint32_t sc = __shfl_sync(0xffffffffu, sc_now, k & 31);
            if (sc) {   // a page that does not exist is passed over
                const int pos = chunk0 + k * C::TILE;
                const bool whole = pos >= all_lo && pos + CHUNK <= all_hi;
                const int stage = (k % ST) * C::STAGE_BYTES;
                consume<C>(w, ring + stage, ring_ptr + stage + CHUNK * D, pos, whole, static_cast<int>(sc & 255) - 127,
                           static_cast<int>(sc >> 8 & 255) - 127, scale_log2, g, t);
            }
        }
        cp_async_wait<0>();
        __syncwarp();

        // ---- merge the warps: rows of this CTA's part of the unit
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float l = quad_sum(w.l[mt][half]);
                if (t == 0) {
                    const int r = mt * 16 + half * 8 + g;
                    sh_m[warp][r] = w.m[mt][half];
                    sh_l[warp][r] = l;
                }
            }
        __syncthreads();
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int r = mt * 16 + half * 8 + g;
                float m = -INFINITY, l = 0.f;
#pragma unroll
                for (int i = 0; i < NW; ++i)
                    m = fmaxf(m, sh_m[i][r]);
                m = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int i = 0; i < NW; ++i)
                    l += sh_l[i][r] * ptx::ex2_approx(sh_m[i][r] - m);
                // O of this warp stands for O * 2^(M - 6); divide by the unit's l * 2^m
                const float f = l == 0.f || w.M[mt][half] == -INFINITY ? 0.f : ptx::ex2_approx(w.M[mt][half] - 6.f - m) / l;
#pragma unroll
                for (int j = 0; j < D / 8; j += 4)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int gg = 2 * t + k;   // the accumulator's column
                        const int d = D == 64 ? 8 * gg + j : (j >> 4) * 128 + 16 * gg + (j & 15);
                        const float4 v = make_float4(w.o[mt][j][half * 2 + k] * f, w.o[mt][j + 1][half * 2 + k] * f,
                                                     w.o[mt][j + 2][half * 2 + k] * f, w.o[mt][j + 3][half * 2 + k] * f);
                        reinterpret_cast<float4 *>(mine_o)[unit_offset<D>(r, d >> 2)] = v;
                    }
                if (warp == 0 && t == 0)
                    sh_lse[r] = l == 0.f ? -INFINITY : m + ptx::lg2_approx(l);
            }
        __syncthreads();
        const int c0 = cut ? range.owner(line.at) : cta;
        const int c1 = cut ? range.owner(line.at + span.tiles - 1) : cta;
        const int rows = s.n * a.G;
        auto write_o = [&](int r, int u, const float4 &v) {   // unit u of row r
            const int rr = rb * R + r;
            if (rr >= rows)
                return;
            uint16_t *o = static_cast<uint16_t *>(a.o) + b * a.o_sb + (h * a.G + rr % a.G) * a.o_sh +
                          static_cast<long long>(rr / a.G) * a.o_sl;
            *reinterpret_cast<uint2 *>(o + u * 4) = make_uint2(ptx::pack_bf16x2(v.x, v.y), ptx::pack_bf16x2(v.z, v.w));
        };
        auto write_lse = [&](int r, float lse2) {
            const int rr = rb * R + r;
            if (rr < rows)
                a.lse[(static_cast<long long>(b) * a.Hq + h * a.G + rr % a.G) * a.Lq + rr / a.G] = lse2 * 0.69314718055994531f;
        };
        const size_t slot_floats = Parts::slot_floats(R, D);
        float *part = cut ? parts.data + (2 * static_cast<size_t>(cta) + (cta == c0 ? 1 : 0)) * slot_floats : nullptr;
        for (int i = tid; i < R * (D / 4); i += C::T) {
            const int r = i / (D / 4), u = i % (D / 4);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                const float4 x = reinterpret_cast<const float4 *>(smem + k * C::RING_BYTES)[unit_offset<D>(r, u)];
                v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            }
            if (c0 == c1)
                write_o(r, u, v);
            else
                reinterpret_cast<float4 *>(part)[i] = v;
        }
        for (int r = tid; r < R; r += C::T) {
            if (c0 == c1)
                write_lse(r, sh_lse[r]);
            else
                part[R * D + r] = sh_lse[r];
        }
        if (c0 != c1) {
            __threadfence();
            __syncthreads();
            if (tid == 0)
                sh_last = atomicAdd(parts.counters + c0, 1) == c1 - c0;
            __syncthreads();
            if (sh_last) {   // every part of the unit is there: merge them in key order
                __threadfence();
                merge_parts<C>(parts, c0, c1, tid, C::T, write_o, write_lse);
                if (tid == 0)
                    parts.counters[c0] = 0;
            }
        }
        __syncthreads();   // the rings and sh_* are free again
        if (!line.next(a) || line.at >= end)
            break;
    }
}

template <class C>
fa2_status launch_attn(const AttnArgs &a)
{
    Parts parts;
    if (!parts_of<C>(a, parts))
        return FA2_ERR_INVALID_ARG;
    const int grid = line_grid<C>(a, parts.data != nullptr);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return FA2_ERR_CUDA;
    static std::atomic<unsigned long long> configured{0};
    const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
    if (!bit || !(configured.load() & bit)) {
        if (cudaFuncSetAttribute(attn_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess) {
            (void)cudaGetLastError();
            return FA2_ERR_CUDA;
        }
        configured.fetch_or(bit);
    }
    attn_kernel<C><<<grid, C::T, C::SMEM_BYTES, a.stream>>>(a, parts);
    return cudaGetLastError() == cudaSuccess ? FA2_OK : FA2_ERR_CUDA;
}
#endif

}  // namespace cache
}  // namespace fa2
