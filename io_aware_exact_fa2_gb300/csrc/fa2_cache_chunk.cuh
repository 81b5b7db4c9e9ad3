// fa2_cache_chunk.cuh -- attention of many query rows over the paged e4m3 cache
// (fa2_cache_attn in include/fa2_cache.h): blocks of 128 rows on the 5th-generation
// tensor cores.
//
// Mathematics.  As in fa2_cache_attn.cuh, rows are the tokens of a sequence times the
// query heads that share a key/value head, codes and rows of Q (times a power of two)
// are exact in f16, and one accumulator takes pages of any strength: for key j of a
// page with exponents ek, ev
//     x_j = S_j * scale * log2 e * 2^ek,   p'_j = 2^(x_j + ev - M + 6)   (f16 for P V)
//     O += P' V,   l += 2^-ev sum p'       M: running maximum of x + ev
// so both exponents ride in the one multiply-add before the exponential, at no cost.
// M is raised only when a tile exceeds it by more than 2^8: p' stays within 2^14.
//
// What bounds it.  4 D operations a (row, key) pair against D / 64 cache bytes a row
// and key: the tensor pipe.  Two f16 products of 128 rows x 64 keys x D = 128 take
// some 540 cycles; the exponentials and the rest of the softmax cost about as much
// issue time, and each code has to be converted once a block of rows.  So the three
// run on warps of their own,
//     4 warps   softmax: one row a thread, S from and P to tensor memory
//     4 warps   codes from global memory to f16 operands in shared memory (swizzled),
//               a tile ahead in registers
//     1 warp    issues the products
// with two buffers of K, V and S each, and at D <= 128 two CTAs share an SM (256
// columns of tensor memory each), so that one's exponentials run under the other's
// products.  Work is cut and merged as in fa2_cache_line.cuh.
#pragma once

#include <atomic>

#include "fa2_cache_line.cuh"

namespace fa2 {
namespace cache {

template <int D_>
struct ChunkCfg {
    static constexpr int D = D_;
    static constexpr int R = 128;                    // query rows of a unit
    static constexpr int TILE = 64;                  // keys
    static constexpr int UNIT_COST = 4, MIN_TILES = 4;   // see fa2_cache_line.cuh
    static constexpr int ALIGN = CHUNK;              // where a unit's first tile may begin
    static constexpr int CTAS = D <= 128 ? 2 : 1;    // an SM
    static constexpr int WARP_CONVERT = 4, WARP_MMA = 8;
    static constexpr int T = 32 * 12;                // (the last warpgroup: one issuing warp and three idle ones)
    // With two CTAs an SM the launch leaves 80 registers a thread, 240 for the three
    // warpgroups' lanes together: the softmax rises, the issuing warpgroup gives.
    static constexpr bool REG_SPLIT = CTAS == 2;
    static constexpr int REG_SOFTMAX = 120, REG_CONVERT = 80, REG_ISSUE = 40;
    static_assert(REG_SOFTMAX + REG_CONVERT + REG_ISSUE <= 3 * 80, "the split draws on the launch's registers");
    static constexpr int GROUPS = TILE / CHUNK;      // 16-key groups of a tile, each in one page

    static constexpr int Q_PANEL = R * 128, KV_PANEL = TILE * 128;   // 64 columns of f16, 128-byte rows
    static constexpr int Q_BYTES = D / 64 * Q_PANEL, KV_BYTES = D / 64 * KV_PANEL;
    static constexpr int OFF_Q = 0, OFF_K = Q_BYTES, OFF_V = OFF_K + 2 * KV_BYTES;
    // rings of four: a tile's group scales and flags, its NaN values by key
    static constexpr int NAN_WORDS = D / 32;
    static constexpr int OFF_INFO = OFF_V + 2 * KV_BYTES, INFO_BYTES = GROUPS * 16 + 16;
    static constexpr int OFF_NAN = OFF_INFO + 4 * INFO_BYTES, NAN_BYTES = TILE * NAN_WORDS * 4;
    static constexpr int OFF_BAR = OFF_NAN + 4 * NAN_BYTES;
    static constexpr int NUM_BAR = 18;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BAR * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;          // 1024: operand alignment

    static constexpr int TM_S = 0, TM_O = 2 * TILE;
    static constexpr int TMEM_COLS = D <= 128 ? 256 : 512;

    static constexpr int BAR_Q_FULL = 0, BAR_Q_EMPTY = 1, BAR_K_FULL = 2, BAR_K_EMPTY = 4, BAR_V_FULL = 6, BAR_V_EMPTY = 8,
                         BAR_S_FULL = 10, BAR_P_FULL = 12, BAR_O_DONE = 14, BAR_O_FREE = 15, BAR_GROUP = 16, BAR_DRAIN = 17;

    // kind::f16 with f16 A and B (formats 0), fp32 accumulator
    static constexpr uint32_t idesc(int n, bool b_mn)
    {
        return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(R >> 4) << 24);
    }
    static_assert(CTAS * SMEM_BYTES <= 227 * 1024 && CTAS * TMEM_COLS <= 512 && 2 * TILE + D <= TMEM_COLS, "an SM holds CTAS of them");
};

// Error codes of waits that ran out (bits 8-11 the waiting role).
constexpr int CHUNK_ERR_SOFTMAX = 8 << 8, CHUNK_ERR_CONVERT = 9 << 8, CHUNK_ERR_MMA = 10 << 8, CHUNK_ERR_DRAIN = 11 << 8;

#ifdef __CUDACC__

// What the converting warps tell the softmax warps of a tile.
// For each group of 16 keys: 2^ek, ev, 2^-ev, and a word of the key and value scales' bytes
// and this bit (0: no page); then a flag byte from each converting warp.
constexpr uint32_t INFO_PAGE = 1u << 16;
constexpr uint32_t FLAG_WHOLE = 1, FLAG_NAN = 2;

// Sixteen codes as f16 into two 16-byte columns of a 128-byte-swizzled row.  (Eight lanes
// that store together have eight rows of one column: the swizzle spreads them over all banks.)
__device__ __forceinline__ void store_f16(uint32_t row_addr, int row, int c, const uint4 &w)
{
    ptx::st_shared_v4(row_addr + ((c ^ (row & 7)) << 4), e4m3x2_to_f16x2(w.x), e4m3x2_hi_to_f16x2(w.x), e4m3x2_to_f16x2(w.y),
                      e4m3x2_hi_to_f16x2(w.y));
    ptx::st_shared_v4(row_addr + (((c + 1) ^ (row & 7)) << 4), e4m3x2_to_f16x2(w.z), e4m3x2_hi_to_f16x2(w.z),
                      e4m3x2_to_f16x2(w.w), e4m3x2_hi_to_f16x2(w.w));
}

// NaN codes among four: bit i for byte i.
__device__ __forceinline__ uint32_t nan_bits(uint32_t w)
{
    const uint32_t m = (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
    return (m | m >> 7 | m >> 14 | m >> 21) & 15u;
}

template <class C>
__global__ void __launch_bounds__(C::T, C::CTAS) chunk_kernel(const AttnArgs a, const Parts parts)
{
    using namespace ptx;
    constexpr int D = C::D, R = C::R, TILE = C::TILE, GROUPS = C::GROUPS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ LineShared sh_line;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool cut = parts.data != nullptr;
    const int cta = blockIdx.x;
    Range range;
    long long first, end;
    Line<C> line;
    if (!find_range<C>(a, cut, sh_line, range, first, end, line))
        return;

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *const smem = smem_raw + (base - smem_u32(smem_raw));
    auto bar = [&](int i) { return base + C::OFF_BAR + 8 * i; };
    if (tid == 0) {
        for (int i = 0; i < C::NUM_BAR; ++i) {
            const bool by_warps = i == C::BAR_Q_FULL || i / 2 == C::BAR_K_FULL / 2 || i / 2 == C::BAR_V_FULL / 2 ||
                                  i / 2 == C::BAR_P_FULL / 2 || i == C::BAR_O_FREE || i == C::BAR_GROUP;
            mbar_init(bar(i), by_warps ? 4 : 1);
        }
        fence_mbar_init();
    }
    if (warp == C::WARP_MMA) {
        tmem_alloc(base + C::OFF_MISC, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + C::OFF_MISC);

    const uint64_t limit = a.wait_limit_ns;
    auto warp_wait = [&](int i, uint32_t parity, int code) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar(i), parity, a.err, code | i, limit));
    };
    auto warp_arrive = [&](int i) {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(i));
    };
    // the tiles of the unit `line` that lie in this CTA's range
    auto part_of = [&](int &tile0, int &tile1) {
        tile0 = cut && first > line.at ? static_cast<int>(first - line.at) : 0;
        tile1 = cut && end < line.at + line.span.tiles ? static_cast<int>(end - line.at) : line.span.tiles;
    };
    auto next_unit = [&]() { return line.next(a) && line.at < end; };
    uint32_t it = 0;       // tiles before the present unit's first: buffers alternate by tile
    uint32_t unit = 0;

    if (warp >= C::WARP_MMA) {
        // ============================================ one thread issues the products
        if constexpr (C::REG_SPLIT)
            setmaxnreg_dec<C::REG_ISSUE>();
        if (warp == C::WARP_MMA) {
            // (all lanes wait: a lone lane would have to poll)
            const bool leader = elect_one();
            const uint64_t desc_q = sdesc_sw128(base + C::OFF_Q, 16, 1024);
            const uint64_t desc_k = sdesc_sw128(base + C::OFF_K, 16, 1024);
            const uint64_t desc_v = sdesc_sw128(base + C::OFF_V, C::KV_PANEL, 1024);
            auto issue_s = [&](uint32_t g, bool last) -> bool {   // S = Q K^T of tile g
                const uint32_t buf = g & 1;
                if (!warp_wait(C::BAR_K_FULL + buf, g >> 1 & 1, CHUNK_ERR_MMA))
                    return false;
                tc_fence_after();
                if (leader) {
                    const uint64_t dk = desc_k + (buf * C::KV_BYTES >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_ss(tmem + C::TM_S + buf * TILE, desc_q + (((kk >> 2) * C::Q_PANEL + (kk & 3) * 32) >> 4),
                               dk + (((kk >> 2) * C::KV_PANEL + (kk & 3) * 32) >> 4), C::idesc(TILE, false), kk > 0);
                    mma_commit(bar(C::BAR_S_FULL + buf));
                    mma_commit(bar(C::BAR_K_EMPTY + buf));
                    if (last)
                        mma_commit(bar(C::BAR_Q_EMPTY));
                }
                __syncwarp();
                return true;
            };
            auto issue_pv = [&](uint32_t g, bool start) -> bool {   // O += P V of tile g
                const uint32_t buf = g & 1;
                // a unit's first product overwrites O: the one before has been read out
                if (!warp_wait(C::BAR_V_FULL + buf, g >> 1 & 1, CHUNK_ERR_MMA) ||
                    !warp_wait(C::BAR_P_FULL + buf, g >> 1 & 1, CHUNK_ERR_MMA) ||
                    (start && unit > 0 && !warp_wait(C::BAR_O_FREE, (unit - 1) & 1, CHUNK_ERR_MMA)))
                    return false;
                tc_fence_after();
                if (leader) {
                    const uint64_t dv = desc_v + (buf * C::KV_BYTES >> 4);
#pragma unroll
                    for (int kk = 0; kk < TILE / 16; ++kk)
                        mma_ts(tmem + C::TM_O, tmem + C::TM_S + buf * TILE + kk * 8, dv + (kk * 16 * 128 >> 4),
                               C::idesc(D, true), !start || kk > 0);
                    mma_commit(bar(C::BAR_O_DONE));
                    mma_commit(bar(C::BAR_V_EMPTY + buf));
                }
                __syncwarp();
                return true;
            };
            bool ok = true;
            do {
                int tile0, tile1;
                part_of(tile0, tile1);
                const int n = tile1 - tile0;
                ok = warp_wait(C::BAR_Q_FULL, unit & 1, CHUNK_ERR_MMA);
                for (int j = 0; j < 2 && j < n && ok; ++j)
                    ok = issue_s(it + j, j == n - 1);
                for (int j = 0; j < n && ok; ++j) {
                    ok = issue_pv(it + j, j == 0);
                    if (ok && j + 2 < n)
                        ok = issue_s(it + j + 2, j + 2 == n - 1);
                }
                it += n;
                ++unit;
            } while (ok && next_unit());
            // nothing issued is still running when tensor memory is given back
            if (leader)
                mma_commit(bar(C::BAR_DRAIN));
            __syncwarp();
            warp_wait(C::BAR_DRAIN, 0, CHUNK_ERR_DRAIN);
        }
    } else if (warp >= C::WARP_CONVERT) {
        // ============================================ codes -> f16 operands
        // A warp takes blocks of 8 rows by 64 bytes: rows 8 w .. and 8 (w + 4) .. of every
        // panel, so two 16-key groups a tile.
        constexpr int NL = D / 32;                       // 16-byte pieces a thread takes of K
        const int w = warp - C::WARP_CONVERT, c = lane >> 3;
        const int row0 = w * 8 + (lane & 7);             // piece i: row row0 + 32 (i & 1), panel i / 2
        auto piece = [&](int off, uint32_t buf, int i) {
            return base + off + buf * C::KV_BYTES + (i >> 1) * C::KV_PANEL + (row0 + 32 * (i & 1)) * 128;
        };
        bool ok = true;
        do {
            int tile0, tile1;
            part_of(tile0, tile1);
            const int n = tile1 - tile0, b = line.b, h = line.h;
            const int from = (line.span.lo & ~(C::ALIGN - 1)) + tile0 * TILE;
            const int stop = line.span.hi < from + n * TILE ? line.span.hi : from + n * TILE;
            int all_lo, all_hi;
            line.seen_by_all(a, all_lo, all_hi);
            // Pages and scales of 32 groups (eight tiles) at a time, one a lane, loaded one
            // and two batches ahead.
            auto table_batch = [&](int k) {
                const long long pos = from + static_cast<long long>(k + lane) * CHUNK;
                return pos < stop ? page_of(a.c, b, static_cast<int>(pos) >> a.c.page_shift) : -1;
            };
            auto scale_batch = [&](int id) -> uint32_t {
                if (id < 0)
                    return 0;
                const long long i = static_cast<long long>(id) * a.c.H + h;
                return a.c.k.scale[i] | static_cast<uint32_t>(a.c.v.scale[i]) << 8 | INFO_PAGE;
            };
            int id_now = table_batch(0), id_next = table_batch(32), id_after = table_batch(64);
            uint32_t sc_now = scale_batch(id_now), sc_next = scale_batch(id_next);

            uint4 k_reg[NL], v_reg[NL];
            uint32_t info = 0;                           // lane i < GROUPS: group i of the tile to come
            int id_row[2];                               // pages of this thread's two rows
            auto advance = [&](int j) {                  // to tile j
                if (j > 0 && (j & 7) == 0) {
                    id_now = id_next;
                    id_next = id_after;
                    sc_now = sc_next;
                    sc_next = scale_batch(id_next);
                    id_after = table_batch(j * GROUPS + 64);
                }
                info = __shfl_sync(0xffffffffu, sc_now, (j & 7) * GROUPS + (lane & (GROUPS - 1)));
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    id_row[r] = __shfl_sync(0xffffffffu, id_now, (j & 7) * GROUPS + (w >> 1) + 2 * r);
            };
            auto load = [&](uint4 (&reg)[NL], const Half &half, int j) {
                const uint8_t *p[2];
                bool seen[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int pos = from + j * TILE + row0 + 32 * r, slot = pos & ((1 << a.c.page_shift) - 1);
                    // positions that no row of the block sees are zeros
                    seen[r] = id_row[r] >= 0 && pos >= line.span.lo && pos < stop;
                    p[r] = half.codes + id_row[r] * half.s_page + h * half.s_head + slot * half.s_slot + c * 16;
                }
#pragma unroll
                for (int i = 0; i < NL; ++i)
                    reg[i] = seen[i & 1] ? __ldg(reinterpret_cast<const uint4 *>(p[i & 1] + (i >> 1) * 64)) : make_uint4(0, 0, 0, 0);
            };
            advance(0);
            load(k_reg, a.c.k, 0);
            load(v_reg, a.c.v, 0);
            for (int j = 0; j < n && ok; ++j) {
                const uint32_t g = it + j, buf = g & 1, par = (g >> 1 & 1) ^ 1, slot = g & 3;
                const int pos0 = from + j * TILE;
                if (g >= 2 && !(ok = warp_wait(C::BAR_K_EMPTY + buf, par, CHUNK_ERR_CONVERT)))
                    break;
                const bool pages = __all_sync(0xffffffffu, (info & INFO_PAGE) && (info & 255) != 255 && (info >> 8 & 255) != 255);
                const bool whole = pages && pos0 >= all_lo && pos0 + TILE <= all_hi;
                bool nan = false;
                if (!whole) {
                    // Rows of the block see different keys of this tile, and a NaN value
                    // times a weight of 0 is NaN: such values become zeros here, and their
                    // places go to the softmax warps.
                    uint16_t *const map = reinterpret_cast<uint16_t *>(smem + C::OFF_NAN + slot * C::NAN_BYTES);
#pragma unroll
                    for (int i = 0; i < NL; ++i) {
                        const int row = row0 + 32 * (i & 1);
                        const uint32_t sc = __shfl_sync(0xffffffffu, info, row >> 4);
                        uint32_t m = nan_bits(v_reg[i].x) | nan_bits(v_reg[i].y) << 4 | nan_bits(v_reg[i].z) << 8 |
                                     nan_bits(v_reg[i].w) << 12;
                        const int pos = pos0 + row;
                        if ((sc & INFO_PAGE) && (sc >> 8 & 255) == 255 && pos >= line.span.lo && pos < stop)
                            m = 0xffffu;   // a NaN scale
                        if (m)
                            v_reg[i] = make_uint4(without_nan(v_reg[i].x), without_nan(v_reg[i].y),
                                                  without_nan(v_reg[i].z), without_nan(v_reg[i].w));
                        nan |= m != 0;
                        map[row * (D / 16) + (i >> 1) * 4 + c] = static_cast<uint16_t>(m);
                    }
                    nan = __any_sync(0xffffffffu, nan);
                }
                uint32_t *const words = reinterpret_cast<uint32_t *>(smem + C::OFF_INFO + slot * C::INFO_BYTES);
                if (w == 0 && lane < GROUPS) {
                    // (a NaN scale: the softmax warps go by its byte)
                    const int kb = info & 255, vb = info >> 8 & 255;
                    const int ek = kb == 255 ? 0 : kb - 127, ev = vb == 255 ? 0 : vb - 127;
                    reinterpret_cast<float4 *>(words)[lane] =
                        make_float4(pow2i(ek), static_cast<float>(ev), pow2i(-ev), __uint_as_float(info));
                }
                if (lane == 0)   // flags, one byte a warp
                    reinterpret_cast<uint8_t *>(words + GROUPS * 4)[w] = (whole ? FLAG_WHOLE : 0) | (nan ? FLAG_NAN : 0);
#pragma unroll
                for (int i = 0; i < NL; ++i)
                    store_f16(piece(C::OFF_K, buf, i), row0, c * 2, k_reg[i]);
                fence_proxy_async_shared();
                warp_arrive(C::BAR_K_FULL + buf);
                if (j + 1 < n) {   // the next tile's keys come in while these values are converted
                    advance(j + 1);
                    load(k_reg, a.c.k, j + 1);
                }
                if (g >= 2 && !(ok = warp_wait(C::BAR_V_EMPTY + buf, par, CHUNK_ERR_CONVERT)))
                    break;
#pragma unroll
                for (int i = 0; i < NL; ++i)
                    store_f16(piece(C::OFF_V, buf, i), row0, c * 2, v_reg[i]);
                fence_proxy_async_shared();
                warp_arrive(C::BAR_V_FULL + buf);
                if (j + 1 < n)
                    load(v_reg, a.c.v, j + 1);
            }
            it += n;
        } while (ok && next_unit());
    } else {
        // ============================================ softmax: one row a thread
        if constexpr (C::REG_SPLIT)
            setmaxnreg_inc<C::REG_SOFTMAX>();
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        const int row = tid;
        const float scale_log2 = a.scale * 1.4426950408889634f;
        const uint32_t o_addr = tmem + lanes + C::TM_O;
        uint32_t group_phase = 0;
        bool ok = true;
        do {
            int tile0, tile1;
            part_of(tile0, tile1);
            const int n = tile1 - tile0, b = line.b, h = line.h, rb = line.rb;
            const Seq s = line.s;
            const int from = (line.span.lo & ~(C::ALIGN - 1)) + tile0 * TILE;
            const int rr = rb * R + row;
            const bool live = rr < s.n * a.G;
            const int tok = rr / a.G, hq = h * a.G + rr % a.G;
            const int pos = s.kv - s.n + tok;
            const int hi = !live ? 0 : a.causal ? pos + 1 : s.kv;
            int lo = 0;
            if (a.window >= 0) {
                const long long x = static_cast<long long>(pos) - a.window;
                lo = x > 0 ? static_cast<int>(x) : 0;
            }
            // ---- this row of Q, times the power of two that brings its largest
            // magnitude to [2^14, 2^15), as f16
            int e;
            {
                const uint16_t *q = static_cast<const uint16_t *>(a.q) + b * a.q_sb + hq * a.q_sh + tok * a.q_sl;
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 x = live ? __ldg(reinterpret_cast<const uint4 *>(q) + c) : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t u = w[k] & 0x7fffu, v = (w[k] >> 16) & 0x7fffu;
                        top = top > u ? top : u;
                        top = top > v ? top : v;
                    }
                }
                e = static_cast<int>(top >> 7) - 127 - 14;
                e = e < -126 ? -126 : e;
                // a row with an infinity or NaN has no finite scores: make it NaN
                const float f = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : pow2i(-e);
                if (unit > 0 && !(ok = warp_wait(C::BAR_Q_EMPTY, (unit - 1) & 1, CHUNK_ERR_SOFTMAX)))
                    break;
#pragma unroll 8
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 x = live ? __ldg(reinterpret_cast<const uint4 *>(q) + c) : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    uint32_t y[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        y[k] = pack_f16x2(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xffff0000u) * f);
                    st_shared_v4(base + C::OFF_Q + (c >> 3) * C::Q_PANEL + row * 128 + (((c & 7) ^ (row & 7)) << 4), y[0], y[1],
                                 y[2], y[3]);
                }
                fence_proxy_async_shared();
                warp_arrive(C::BAR_Q_FULL);
            }

            const float scale_row = scale_log2 * pow2i(e);
            float M = -INFINITY, l = 0.f;
            uint32_t nan[C::NAN_WORDS];   // values of O that a visible NaN value makes NaN
#pragma unroll
            for (int k = 0; k < C::NAN_WORDS; ++k)
                nan[k] = 0;
            for (int j = 0; j < n; ++j) {
                const uint32_t g = it + j, buf = g & 1;
                if (!(ok = warp_wait(C::BAR_S_FULL + buf, g >> 1 & 1, CHUNK_ERR_SOFTMAX)))
                    break;
                tc_fence_after();
                const uint32_t s_addr = tmem + lanes + C::TM_S + buf * TILE;
                uint32_t r0[32], r1[32];
                tmem_ld32(s_addr, r0);
                tmem_ld32(s_addr + 32, r1);
                const float4 *const info = reinterpret_cast<const float4 *>(smem + C::OFF_INFO + (g & 3) * C::INFO_BYTES);
                const uint32_t flags = __float_as_uint(info[GROUPS].x);
                float c[GROUPS], ev[GROUPS], lf[GROUPS];      // x = S * c
#pragma unroll
                for (int q = 0; q < GROUPS; ++q) {
                    const float4 f = info[q];
                    c[q] = fmaxf(scale_row * f.x, 1.17549435e-38f);   // (not 0: a hidden score is -inf * c)
                    ev[q] = f.y;
                    lf[q] = f.z;
                }
                tmem_ld_wait(r0);
                tmem_ld_wait(r1);
                const bool whole = flags & FLAG_WHOLE;
                if (!whole) {             // scores that the row does not see
                    const int pos0 = from + j * TILE;
#pragma unroll
                    for (int q = 0; q < GROUPS; ++q) {
                        const uint32_t word = __float_as_uint(info[q].w);
                        const bool page = word & INFO_PAGE, nan_scale = (word & 255) == 255;
#pragma unroll
                        for (int k = q * CHUNK; k < (q + 1) * CHUNK; ++k) {
                            uint32_t &x = k < 32 ? r0[k & 31] : r1[k & 31];
                            const bool see = page && pos0 + k >= lo && pos0 + k < hi;
                            x = !see ? 0xff800000u : nan_scale ? 0x7fc00000u : x;
                        }
                    }
                    if (flags & 0x02020202u) {
                        const uint32_t *map = reinterpret_cast<const uint32_t *>(smem + C::OFF_NAN + (g & 3) * C::NAN_BYTES);
#pragma unroll 1
                        for (int k = 0; k < TILE; ++k)
                            if (pos0 + k >= lo && pos0 + k < hi)
#pragma unroll
                                for (int q = 0; q < C::NAN_WORDS; ++q)
                                    nan[q] |= map[k * C::NAN_WORDS + q];
                    }
                }
                // running maximum of x + ev
                float top = -INFINITY;
#pragma unroll
                for (int q = 0; q < GROUPS; ++q) {
                    const uint32_t *r = q < 2 ? r0 + q * CHUNK : r1 + (q - 2) * CHUNK;
                    float t = __uint_as_float(r[0]);
#pragma unroll
                    for (int k = 1; k < 15; k += 2)
                        t = max3(t, __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
                    t = fmaxf(t, __uint_as_float(r[15]));
                    top = fmaxf(top, fmaf(t, c[q], ev[q]));
                }
                const bool raise = top > M + 8.f, any = __any_sync(0xffffffffu, raise);
                float f = 1.f;
                if (raise) {
                    f = ex2_approx(M - top);
                    M = top;
                    l *= f;
                }
                // A parity tells a phase from the one before only, so the wait below for the
                // last tile's product needs this one taken for the last but one's, before
                // the last can complete.
                if (j > 0 && (any || j == n - 1)) {
                    if (!(ok = warp_wait(C::BAR_O_DONE, (g - 1) & 1, CHUNK_ERR_SOFTMAX)))
                        break;
                    tc_fence_after();
                    if (any) {            // O in tensor memory stands for the old maximum
#pragma unroll 1
                        for (int cc = 0; cc < D / 32; ++cc) {
                            uint32_t o[32];
                            tmem_ld32(o_addr + 32 * cc, o);
                            tmem_ld_wait(o);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st32(o_addr + 32 * cc, o);
                        }
                    }
                }
                // weights, over the first half of this S buffer as f16 pairs
                const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t p[16];
#pragma unroll
                    for (int q = 0; q < GROUPS / 2; ++q) {
                        const uint32_t *r = (half ? r1 : r0) + q * CHUNK;
                        const int grp = half * 2 + q;
                        const float add = ev[grp] + 6.f - ref;
                        const uint64_t c2 = f32x2(c[grp], c[grp]), add2 = f32x2(add, add);
                        uint64_t sum2 = 0;
#pragma unroll
                        for (int k = 0; k < CHUNK; k += 2) {
                            float x0, x1;
                            unpack_f32x2(fma_f32x2(f32x2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), c2, add2), x0, x1);
                            x0 = ex2_approx(x0);
                            x1 = ex2_approx(x1);
                            sum2 = add_f32x2(sum2, f32x2(x0, x1));
                            p[q * 8 + k / 2] = pack_f16x2(x0, x1);
                        }
                        float sum0, sum1;
                        unpack_f32x2(sum2, sum0, sum1);
                        l = fmaf(sum0 + sum1, lf[grp], l);
                    }
                    tmem_st16(s_addr + half * 16, p);
                }
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(C::BAR_P_FULL + buf);
            }
            if (!ok)
                break;

            // ---- O out of tensor memory: the unit's rows, or this part of them
            it += n;
            if (!(ok = warp_wait(C::BAR_O_DONE, (it - 1) & 1, CHUNK_ERR_SOFTMAX)))
                break;
            tc_fence_after();
            const int first_cta = cut ? range.owner(line.at) : cta;
            const int last_cta = cut ? range.owner(line.at + line.span.tiles - 1) : cta;
            const bool alone = first_cta == last_cta;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const float lse2 = l == 0.f ? -INFINITY : M - 6.f + lg2_approx(l);
            uint16_t *const o = static_cast<uint16_t *>(a.o) + b * a.o_sb + hq * a.o_sh + tok * a.o_sl;
            float *const part =
                cut ? parts.data + (2 * static_cast<size_t>(cta) + (cta == first_cta ? 1 : 0)) * Parts::slot_floats(R, D) : nullptr;
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t r[32];
                tmem_ld32(o_addr + 32 * cc, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    r[k] = (nan[cc] >> k & 1) ? 0x7fc00000u : __float_as_uint(__uint_as_float(r[k]) * inv);
                if (alone && live) {
#pragma unroll
                    for (int k = 0; k < 32; k += 8)
                        *reinterpret_cast<uint4 *>(o + cc * 32 + k) =
                            make_uint4(pack_bf16x2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])),
                                       pack_bf16x2(__uint_as_float(r[k + 2]), __uint_as_float(r[k + 3])),
                                       pack_bf16x2(__uint_as_float(r[k + 4]), __uint_as_float(r[k + 5])),
                                       pack_bf16x2(__uint_as_float(r[k + 6]), __uint_as_float(r[k + 7])));
                } else if (!alone) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        *reinterpret_cast<uint4 *>(part + row * D + cc * 32 + k) = make_uint4(r[k], r[k + 1], r[k + 2], r[k + 3]);
                }
            }
            tc_fence_before();
            warp_arrive(C::BAR_O_FREE);
            auto write_lse = [&](int r, float v) {
                const int x = rb * R + r;
                if (x < s.n * a.G)
                    a.lse[(static_cast<long long>(b) * a.Hq + h * a.G + x % a.G) * a.Lq + x / a.G] = v * 0.69314718055994531f;
            };
            if (alone) {
                write_lse(row, lse2);
            } else {
                part[R * D + row] = lse2;
                // the CTA whose part is the last to arrive merges them
                auto group = [&]() -> bool {
                    warp_arrive(C::BAR_GROUP);
                    return warp_wait(C::BAR_GROUP, group_phase++ & 1, CHUNK_ERR_SOFTMAX);
                };
                __threadfence();
                if (!(ok = group()))
                    break;
                volatile int *const last = reinterpret_cast<int *>(smem + C::OFF_MISC + 4);
                if (tid == 0) {
                    *last = atomicAdd(parts.counters + first_cta, 1) == last_cta - first_cta;
                    if (*last)
                        parts.counters[first_cta] = 0;
                }
                if (!(ok = group()))
                    break;
                if (*last) {
                    __threadfence();
                    auto write_o = [&](int r, int u, const float4 &v) {
                        const int x = rb * R + r;
                        if (x >= s.n * a.G)
                            return;
                        uint16_t *to = static_cast<uint16_t *>(a.o) + b * a.o_sb + (h * a.G + x % a.G) * a.o_sh +
                                       static_cast<long long>(x / a.G) * a.o_sl;
                        *reinterpret_cast<uint2 *>(to + u * 4) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                    };
                    const int live_rows = s.n * a.G - rb * R;
                    merge_parts<C>(parts, first_cta, last_cta, live_rows < R ? live_rows : R, tid, 128, write_o, write_lse);
                }
            }
            ++unit;
        } while (next_unit());
        tmem_st_wait();   // a loop left early may leave stores in flight
    }

    tc_fence_before();
    __syncthreads();
    if (warp == C::WARP_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

template <class C>
fa2_status launch_chunk(const AttnArgs &a)
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
        if (cudaFuncSetAttribute(chunk_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess) {
            (void)cudaGetLastError();
            return FA2_ERR_CUDA;
        }
        configured.fetch_or(bit);
    }
    chunk_kernel<C><<<grid, C::T, C::SMEM_BYTES, a.stream>>>(a, parts);
    return cudaGetLastError() == cudaSuccess ? FA2_OK : FA2_ERR_CUDA;
}
#endif

}  // namespace cache
}  // namespace fa2
