// fa2_cache_chunk.cuh -- attention of many query rows over the paged e4m3 cache
// (fa2_cache_attn in include/fa2_cache.h): blocks of up to 256 rows on the 5th-generation
// tensor cores.
//
// Mathematics.  As in fa2_cache_step.cuh, rows are the tokens of a sequence times the query
// heads that share a key/value head.  The scores are e4m3 products, the cache's codes as
// they are and q as two terms,
//     q 2^-e = q0 + q1          (e: largest magnitude of the row in [224, 448))
// exact but for elements below 2^-9 of their row's largest, which are off by up to 2^-17 of
// that.  For key j of a page with exponents ek, ev
//     x_j = S_j * scale * log2 e * 2^(e + ek),   p'_j = 2^(x_j + ev - M + 6)
//     O += P' V,   l += 2^-ev sum p'             M: a maximum of x + ev so far
// so both exponents ride in the one multiply-add before the exponential, at no cost, and one
// accumulator takes pages of any strength.  P' is f16 (two terms of e4m3 would not span a
// long context's weights) and V is converted to f16, exactly.  M is raised only when the
// weights that a tile has by it would leave f16's range, which their sum tells: most tiles
// need no maximum at all.  (Past 2^20 the multiply-add is exact where M is rounded: there a
// tile's scores are replaced by their differences from its maximum first.)  l sums the weights
// before their rounding to f16, 2^-11 at most: LSE needs that sum, and one of the rounded
// weights for O alone would cost a conversion back of each.
//
// What bounds it.  4 D operations a (row, key) pair against D / 64 cache bytes a row and
// key: the tensor pipe.  (Two e4m3 products take the time of one of f16, and K needs no
// conversion.)  128 rows x 128 keys x D = 128 take some 1100 cycles of it; the exponentials
// and the rest of the softmax cost about as much issue time, and V's conversion is shared by
// the 256 rows of a unit (128 at D = 256, where tensor memory holds no more).  So the work
// has warps of its own,
//     8 or 16 warps  softmax: two threads a row, each half of a tile's keys; S from and P to
//                    tensor memory
//     4 warps        values' codes to f16 operands in shared memory (swizzled)
//     1 warp         issues the products: one 128-row tile's run under the other's softmax
//     1 warp         pages into shared memory by TMA
// on one CTA an SM.  Work is cut and merged as in fa2_cache_line.cuh.
// Measured (several inputs in turn, so that none is in L2): 2048 tokens at the end of 16384, 32
// heads on 8 of 128: 515 GFLOP in 377 us, 1366 TFLOP/s, 71 % of the measured bf16 rate, the
// tensor pipe busy for 58 % of the cycles; no unit is saturated (issue slots 51 %): a row
// tile's chain of products, scores, exponentials and weights, some 3600 cycles for 256 rows by
// 128 keys, has only the other tile's to hide under.  That is not the limit of two row tiles:
// the dense forward (fa2_fwd_kernel.cuh) has two as well and takes some 2700 cycles.  It does
// without what stands in this chain: scores read 16 columns at a time with a wait for each, a
// vote of two warps before a weight may be stored, two threads a row, converted values.  With
// two CTAs of one row tile an SM, which convert the values twice: 499 us.  One thread a row
// instead of two: 435 us.  At D = 64 the chain is as long for half the work: 258 GFLOP of the
// same lengths in 300 us, six ragged prompts' chunks, 24.5 GFLOP, in 60.  At D = 256, 16 heads
// on 4: 515 GFLOP in 482 us, 1069 TFLOP/s.  Units of up to 128 rows take as long as full ones:
// 32 rows, 16 sequences of 4000, 8 heads of 128, 133 MB in 54 us for a floor of 20.
#pragma once

#include <atomic>

#include "fa2_cache_line.cuh"
#include "fa2_cache_tile.cuh"

namespace fa2 {
namespace cache {

template <int D_>
struct ChunkCfg {
    static constexpr int D = D_;
    static constexpr int NQ = D == 256 ? 1 : 2;      // 128-row tiles of a unit
    static constexpr int R = 128 * NQ;               // its query rows
    static constexpr int TILE = 128;                 // keys
    static constexpr int UNIT_COST = 4, MIN_TILES = 3;   // see fa2_cache_line.cuh
    static constexpr int ALIGN = TILE;               // a tile begins at a multiple
    static constexpr int CTAS = 1;                   // an SM
    static constexpr int WARP_CONVERT = 8 * NQ, WARP_MMA = WARP_CONVERT + 4, WARP_LOAD = WARP_MMA + 1;
    static constexpr int T = 32 * (WARP_MMA + 4);    // (the last warpgroup: two idle warps)
    // With six warpgroups the launch leaves 80 registers a thread, 480 for the warpgroups'
    // lanes together: the softmax rises, the others give.
    static constexpr bool REG_SPLIT = NQ == 2;
    static constexpr int REG_SOFTMAX = 88, REG_CONVERT = 56, REG_ISSUE = 72;
    static_assert(4 * REG_SOFTMAX + REG_CONVERT + REG_ISSUE <= 6 * 80, "the split draws on the launch's registers");
    static constexpr int GROUPS = TILE / CHUNK;      // 16-key groups of a tile, each in one page

    static constexpr int ROW = D == 64 ? 64 : 128;   // bytes of a row of codes: its swizzle span
    static constexpr int PANELS = D / ROW, PANEL = TILE * ROW;       // of a stage of codes
    static constexpr int STAGE = TILE * D;
    // Stages of keys, of values: as many as there is room for.  (What is loaded when a stage
    // comes free takes 2 us from memory; D = 64, 32 rows, 98 MB of cache: 57 us, 63 with two.)
    static constexpr int KS = D == 64 ? 4 : D == 128 ? 2 : 1, VS = KS;
    static constexpr int Q_PANEL = 128 * ROW, Q_TERM = 128 * D, Q_TILE = 2 * Q_TERM;   // Q: two terms of codes a row tile
    // V in f16, half a tile's keys a buffer: panels of 64 columns, 128-byte rows
    static constexpr int HALF = TILE / 2, V_PANEL = HALF * 128, V_BYTES = HALF * D * 2, VB = D == 256 ? 2 : 4;
    static constexpr int OFF_Q = 0, OFF_V = NQ * Q_TILE, OFF_K = OFF_V + VB * V_BYTES, OFF_RAW = OFF_K + KS * STAGE;
    // Rings of tiles: group scales of eight; NaN flags, NaN values by key of four.  (Tile g is
    // loaded when the values of g - VS have been read, which waits for the products of g - VS -
    // VB / 2.)
    static constexpr int NAN_WORDS = D / 32;
    static constexpr int OFF_INFO = OFF_RAW + VS * STAGE, INFO_BYTES = GROUPS * 16 + 16, RING = 8;
    static constexpr int OFF_FLAGS = OFF_INFO + RING * INFO_BYTES;
    static constexpr int OFF_NAN = OFF_FLAGS + 16, NAN_BYTES = TILE * NAN_WORDS * 4;
    static constexpr int OFF_MARK = OFF_NAN + 4 * NAN_BYTES;         // values of O that are NaN, by row
    static constexpr int OFF_PAIR = OFF_MARK + R * NAN_WORDS * 4;    // a float of each softmax thread
    static constexpr int OFF_SUM = OFF_PAIR + 2 * R * 4;             // maximum and sum of a row, by row tile
    static constexpr int OFF_BAR = OFF_SUM + R * 8;
    // (the first five: one for each row tile)
    static constexpr int BAR_Q_FULL = 0, BAR_Q_EMPTY = 2, BAR_S_FULL = 4, BAR_P_FULL = 6, BAR_O_DONE = 8, BAR_DRAIN = 10,
                         BAR_V_FULL = 11, BAR_V_EMPTY = BAR_V_FULL + VB, BAR_K_FULL = BAR_V_EMPTY + VB,
                         BAR_K_EMPTY = BAR_K_FULL + KS, BAR_RAW_FULL = BAR_K_EMPTY + KS, BAR_RAW_EMPTY = BAR_RAW_FULL + VS,
                         NUM_BAR = BAR_RAW_EMPTY + VS;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BAR * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;          // 1024: operand alignment
    static_assert(VS + VB / 2 <= RING && VB / 2 + 1 <= 4, "the rings hold the tiles under way");

    // The weights lie over the scores at D = 128, where they fill tensor memory with O; else
    // beside them, and a tile's scores are computed before the product of the one before
    // (ragged chunks at D = 64: 58.0 us over the scores, 53.6 apart).
    static constexpr bool P_APART = D != 128;
    static constexpr int TM_S = 0, TM_O = NQ * TILE, TM_P = P_APART ? TM_O + NQ * D : TM_S, P_STEP = P_APART ? TILE / 2 : TILE;
    static constexpr int TMEM_COLS = 512;
    // kind::f16 with f16 A and B (formats 0), fp32 accumulator
    static constexpr uint32_t idesc(int n, bool b_mn)
    {
        return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (128u >> 4 << 24);
    }
    static_assert(SMEM_BYTES + 1024 + 1024 <= 228 * 1024 && NQ * (TILE + D + (P_APART ? P_STEP : 0)) <= TMEM_COLS, "an SM holds it");
};

// Scores (times log2 e) past which a row's reference is too coarse for what is subtracted from it
// exactly: its last place is 2^-3 there.
constexpr float LARGE = 1 << 20;

// Error codes of waits that ran out (bits 8-11 the waiting role).
constexpr int CHUNK_ERR_SOFTMAX = 8 << 8, CHUNK_ERR_CONVERT = 9 << 8, CHUNK_ERR_MMA = 10 << 8, CHUNK_ERR_LOAD = 11 << 8,
              CHUNK_ERR_DRAIN = 7 << 8;

#ifdef __CUDACC__

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
__global__ void __launch_bounds__(C::T, C::CTAS)
    chunk_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const AttnArgs a,
                 const Parts parts)
{
    using namespace ptx;
    constexpr int D = C::D, R = C::R, TILE = C::TILE, GROUPS = C::GROUPS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ LineShared sh_line;
    // Each warp's place on the line: it changes with the unit only, and would cost the roles
    // registers in their loops over tiles.
    __shared__ struct {
        Range range;
        int first, end;
        Line<C> line[C::T / 32];
    } sh;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool cut = parts.data != nullptr;
    const int cta = blockIdx.x;
    {
        Range range;
        int first, end;
        Line<C> line;
        if (!find_range<C>(a, cut, sh_line, range, first, end, line))
            return;
        if (lane == 0)
            sh.line[warp] = line;
        if (tid == 0) {
            sh.range = range;
            sh.first = first;
            sh.end = end;
        }
    }
    const Line<C> &line = sh.line[warp];

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *const smem = smem_raw + (base - smem_u32(smem_raw));
    auto bar = [&](int i) { return base + C::OFF_BAR + 8 * i; };
    if (tid == 0) {
        for (int i = 0; i < C::NUM_BAR; ++i) {
            const bool rows = i / 2 == C::BAR_Q_FULL / 2 || i / 2 == C::BAR_P_FULL / 2;
            const bool convert = (i >= C::BAR_V_FULL && i < C::BAR_V_EMPTY) || i >= C::BAR_RAW_EMPTY;
            mbar_init(bar(i), rows ? 8 : convert ? 4 : 1);
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
        return wait_phase(bar(i), parity, a.err, code | i, limit);
    };
    auto drain_wait = [&](int i, uint32_t parity) {
        wait_phase(bar(i), parity, a.err, CHUNK_ERR_DRAIN | i, a.drain_limit_ns);
    };
    auto warp_arrive = [&](int i) {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(i));
    };
    // the tiles of the unit `line` that lie in this CTA's range
    auto part_of = [&](int &tile0, int &tile1) {
        tile0 = cut && sh.first > line.at ? sh.first - line.at : 0;
        tile1 = cut && sh.end < line.at + line.span.tiles ? sh.end - line.at : line.span.tiles;
    };
    auto next_unit = [&]() -> bool {     // by a whole warp
        __syncwarp();
        bool more = false;
        if (lane == 0)
            more = sh.line[warp].next(a, sh.end);
        __syncwarp();                    // (a shuffle orders no memory)
        return __shfl_sync(0xffffffffu, more, 0);
    };
    // what the loading warp says of tile g: a group's scales, and whether every row sees every key
    auto group_word = [](const uint8_t *smem, uint32_t g, int q) {
        return reinterpret_cast<const uint32_t *>(smem + C::OFF_INFO + g % C::RING * C::INFO_BYTES)[q * 4 + 3];
    };
    auto is_whole = [](const uint8_t *smem, uint32_t g) {
        return *reinterpret_cast<const uint32_t *>(smem + C::OFF_INFO + g % C::RING * C::INFO_BYTES + GROUPS * 16) != 0;
    };
    uint32_t it = 0;               // tiles before the present unit's first
    // A unit of no more than 128 rows: the row tiles are the same rows, one with the even
    // tiles of keys, one with the odd ones, and are put together at the end.  (32 rows, 131 MB
    // of cache, D = 128: 61 us, 70 with one row tile idle.)
    auto is_twin = [&] { return C::NQ > 1 && line.s.n * a.G - line.rb * R <= 128; };

    if (warp >= C::WARP_MMA) {
        // ============================================ one thread issues the products
        if constexpr (C::REG_SPLIT)
            setmaxnreg_dec<C::REG_ISSUE>();
        if (warp == C::WARP_MMA) {
            // (the whole loop in one lane: groups of products issued from a branch that the
            // warp's other lanes skip took twice the time of the products)
            if (elect_one()) {
                const uint64_t desc_q = D == 64 ? sdesc_sw64(base + C::OFF_Q, 16, 512) : sdesc_sw128(base + C::OFF_Q, 16, 1024);
                const uint64_t desc_k = D == 64 ? sdesc_sw64(base + C::OFF_K, 16, 512) : sdesc_sw128(base + C::OFF_K, 16, 1024);
                const uint64_t desc_v = sdesc_sw128(base + C::OFF_V, C::V_PANEL, 1024);
                bool ok = true;
                auto wait = [&](int i, uint32_t parity) {
                    if (ok)
                        ok = lone_wait(bar(i), parity, a.err, CHUNK_ERR_MMA | i, limit);
                };
                // S = Q K^T of row tile q (rows q_at of Q) and tile g of keys, the last to read
                // this tile of keys, of Q
                auto issue_s = [&](int q, int q_at, uint32_t g, bool last_k, bool last_q) {
                    const uint32_t stage = g % C::KS;
                    const uint64_t dk = desc_k + (stage * C::STAGE >> 4), dq = desc_q + (q_at * C::Q_TILE >> 4);
#pragma unroll
                    for (int term = 0; term < 2; ++term)
#pragma unroll
                        for (int kk = 0; kk < D / 32; ++kk) {
                            const int panel = kk * 32 / C::ROW, col = kk * 32 % C::ROW;
                            mma_ss<true>(tmem + C::TM_S + q * TILE, dq + ((term * C::Q_TERM + panel * C::Q_PANEL + col) >> 4),
                                         dk + ((panel * C::PANEL + col) >> 4), idesc_e4m3_f32(128, TILE, false, false),
                                         term > 0 || kk > 0);
                        }
                    mma_commit(bar(C::BAR_S_FULL + q));
                    if (last_k)
                        mma_commit(bar(C::BAR_K_EMPTY + stage));
                    if (last_q)
                        mma_commit(bar(C::BAR_Q_EMPTY + q_at));
                };
                auto issue_pv = [&](int q, uint32_t g, bool start, bool last_v) {   // O += P V
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t buf = (2 * g + half) % C::VB;
                        const uint64_t dv = desc_v + (buf * C::V_BYTES >> 4);
                        const uint32_t p = tmem + C::TM_P + q * C::P_STEP + half * (C::HALF / 2);
#pragma unroll
                        for (int kk = 0; kk < C::HALF / 16; ++kk)
                            mma_ts(tmem + C::TM_O + q * D, p + kk * 8, dv + (kk * 16 * 128 >> 4), C::idesc(D, true),
                                   !start || half > 0 || kk > 0);
                        if (last_v)
                            mma_commit(bar(C::BAR_V_EMPTY + buf));
                    }
                    mma_commit(bar(C::BAR_O_DONE + q));
                };
                auto wait_k = [&](uint32_t g) { wait(C::BAR_K_FULL + g % C::KS, g / C::KS & 1); };
                auto wait_v = [&](uint32_t item) { wait(C::BAR_V_FULL + item % C::VB, item / C::VB & 1); };
                // of each row tile: tiles of keys, and loads of Q, before the present unit
                uint32_t done[C::NQ] = {}, loads[C::NQ] = {};
                bool more;
                do {
                    int tile0, tile1;
                    part_of(tile0, tile1);
                    const int n = tile1 - tile0;
                    const bool twin = is_twin();
                    // The first tiles' scores; then for each tile and row tile the product with the
                    // values, and the scores of the tile after.  What the first of these reads
                    // beside the weights is waited for before them: they go out in one run.  (A
                    // unit's first product overwrites O: the warps whose weights it waits for
                    // have read out the one before.)
                    wait_k(it);
                    if (twin && n > 1)
                        wait_k(it + 1);
#pragma unroll
                    for (int q = 0; q < C::NQ; ++q) {
                        if (q == 0 || !twin)
                            wait(C::BAR_Q_FULL + q, loads[q] & 1);
                        if (ok && (q == 0 || !twin || n > 1)) {
                            tc_fence_after();
                            if (twin)
                                issue_s(q, 0, it + q, true, n <= q + 1);
                            else
                                issue_s(q, q, it, q == C::NQ - 1, n == 1);
                        }
                    }
                    const int ahead = twin ? 2 : 1;
                    for (int j = 0; j < n && ok; ++j) {
                        wait_v(2 * (it + j));
                        wait_v(2 * (it + j) + 1);
                        if (C::P_APART && j + ahead < n)
                            wait_k(it + j + ahead);
#pragma unroll
                        for (int q = 0; q < C::NQ; ++q)
                            if (!twin || q == (j & 1)) {
                                wait(C::BAR_P_FULL + q, (done[q] + (twin ? j >> 1 : j)) & 1);
                                if (ok) {
                                    const bool next = j + ahead < n;
                                    tc_fence_after();
                                    if (C::P_APART && next)
                                        issue_s(q, twin ? 0 : q, it + j + ahead, twin || q == C::NQ - 1, j + ahead == n - 1);
                                    issue_pv(q, it + j, j < ahead, twin || q == C::NQ - 1);
                                    if (!C::P_APART && next) {
                                        wait_k(it + j + ahead);
                                        if (!ok)
                                            break;
                                        tc_fence_after();
                                        issue_s(q, twin ? 0 : q, it + j + ahead, twin || q == C::NQ - 1, j + ahead == n - 1);
                                    }
                                }
                            }
                    }
                    it += n;
#pragma unroll
                    for (int q = 0; q < C::NQ; ++q) {
                        done[q] += twin ? (n + 1 - q) >> 1 : n;
                        loads[q] += q == 0 || !twin;
                    }
                    Line<C> &mine = sh.line[C::WARP_MMA];
                    more = ok && mine.next(a, sh.end);
                } while (more);
                // nothing issued is still running when tensor memory is given back
                mma_commit(bar(C::BAR_DRAIN));
                lone_wait(bar(C::BAR_DRAIN), 0, a.err, CHUNK_ERR_DRAIN | C::BAR_DRAIN, a.drain_limit_ns);
            }
            __syncwarp();
        } else if (warp == C::WARP_LOAD) {
            // ======================================== pages -> stages
            const int box_shift = a.c.page_shift;              // rows of a box: a page
            const int boxes_shift = 7 - box_shift;             // boxes of a tile
            const uint32_t box_bytes = static_cast<uint32_t>(D) << box_shift;
            const int in_tile = lane & ((1 << boxes_shift) - 1);
            const uint32_t offset = static_cast<uint32_t>(in_tile) * C::ROW << box_shift;   // in each panel
            const int batch_tiles = 32 >> boxes_shift;
            uint32_t issued = 0;                               // tiles
            bool ok = true;
            do {
                int tile0, tile1;
                part_of(tile0, tile1);
                const int n = tile1 - tile0, h = line.h;
                const int from = (line.span.lo & ~(C::ALIGN - 1)) + tile0 * TILE;
                const int stop = line.span.hi < from + n * TILE ? line.span.hi : from + n * TILE;
                int all_lo, all_hi;
                line.seen_by_all(a, all_lo, all_hi);
                // A lane has one of 32 boxes, those of the next 4 to 32 tiles: the table's
                // entries come two such batches ahead, their scales one.
                auto pos_at = [&](int tile) { return from + tile * TILE + (lane << box_shift); };
                auto pages = [&](int tile) {                   // -1: none, or not seen
                    if (tile >= n)
                        return -1;
                    const int pos = pos_at(tile);
                    return pos < stop && pos + (1 << box_shift) > line.span.lo ? page_of(a.c, line.b, pos >> a.c.page_shift) : -1;
                };
                auto scales = [&](int page) -> uint32_t {
                    if (page < 0)
                        return 0;
                    const long long i = static_cast<long long>(page) * a.c.H + h;
                    return a.c.k.scale[i] | static_cast<uint32_t>(a.c.v.scale[i]) << 8 | PAGE_BIT;
                };
                int id = pages(0), id_next = pages(batch_tiles), id_after = pages(2 * batch_tiles);
                uint32_t sc = scales(id), sc_next = scales(id_next);
                float4 info = make_float4(0.f, 0.f, 0.f, 0.f);
                bool fine = false;
                for (int j = 0; j < n; ++j) {
                    const int jj = j & (batch_tiles - 1);
                    if (jj == 0) {
                        if (j > 0) {
                            id = id_next;
                            sc = sc_next;
                            id_next = id_after;
                            sc_next = scales(id_next);
                            id_after = pages(j + 2 * batch_tiles);
                        }
                        // for the box's groups of 16 keys: 2^ek, ev, 2^-ev, and the scales' word
                        // (which tells a NaN scale)
                        const int kb = sc & 255, vb = sc >> 8 & 255;
                        const int ek = kb == 255 ? 0 : kb - 127, ev = vb == 255 ? 0 : vb - 127;
                        info = make_float4(pow2i(ek), static_cast<float>(ev), pow2i(-ev), __uint_as_float(sc));
                        fine = (sc & PAGE_BIT) && kb != 255 && vb != 255;
                    }
                    const bool mine = lane >> boxes_shift == jj;
                    const uint32_t g = it + j, ks = g % C::KS, vs = g % C::VS;
                    if ((g >= C::KS && !(ok = warp_wait(C::BAR_K_EMPTY + ks, (g / C::KS - 1) & 1, CHUNK_ERR_LOAD))) ||
                        (g >= C::VS && !(ok = warp_wait(C::BAR_RAW_EMPTY + vs, (g / C::VS - 1) & 1, CHUNK_ERR_LOAD))))
                        break;
                    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine && id >= 0)) * box_bytes;
                    const int pos0 = from + j * TILE;
                    const bool whole = __all_sync(0xffffffffu, !mine || fine) && pos0 >= all_lo && pos0 + TILE <= all_hi;
                    uint8_t *const to = smem + C::OFF_INFO + g % C::RING * C::INFO_BYTES;
                    if (mine)
                        for (int k = 0; k < 1 << (box_shift - 4); ++k)
                            reinterpret_cast<float4 *>(to)[(in_tile << (box_shift - 4)) + k] = info;
                    if (lane == 0)               // whether every row sees every key of the tile
                        *reinterpret_cast<uint32_t *>(to + GROUPS * 16) = whole;
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar(C::BAR_K_FULL + ks), bytes);
                        mbar_arrive_expect_tx(bar(C::BAR_RAW_FULL + vs), bytes);
                    }
                    __syncwarp();
                    if (mine && id >= 0)
#pragma unroll
                        for (int p = 0; p < C::PANELS; ++p) {
                            tma_load_4d(base + C::OFF_K + ks * C::STAGE + p * C::PANEL + offset, &k_map, p * 128, 0, h, id,
                                        bar(C::BAR_K_FULL + ks));
                            tma_load_4d(base + C::OFF_RAW + vs * C::STAGE + p * C::PANEL + offset, &v_map, p * 128, 0, h, id,
                                        bar(C::BAR_RAW_FULL + vs));
                        }
                    __syncwarp();
                    issued = g + 1;
                }
                it += n;
            } while (ok && next_unit());
            // the copies in flight have landed before the CTA goes
            for (uint32_t g = issued > C::VS ? issued - C::VS : 0; g < issued; ++g) {
                drain_wait(C::BAR_RAW_FULL + g % C::VS, g / C::VS & 1);
                if (g + C::KS >= issued)
                    drain_wait(C::BAR_K_FULL + g % C::KS, g / C::KS & 1);
            }
        }
    } else if (warp >= C::WARP_CONVERT) {
        // ============================================ values' codes -> f16 operands
        if constexpr (C::REG_SPLIT)
            setmaxnreg_dec<C::REG_CONVERT>();
        // Eight lanes take eight rows of one 16-byte column: the swizzles of both sides spread
        // them over all banks.
        constexpr int NL = D / 32;                       // 16-byte pieces a thread takes of half a tile
        const int w = warp - C::WARP_CONVERT;
        const int row0 = w * 8 + (lane & 7);             // piece i: row row0 + 32 (i & 1), column 4 (i / 2) + c
        const int c = lane >> 3;
        auto raw_at = [&](uint32_t stage, int half, int i) {
            const int row = half * C::HALF + row0 + 32 * (i & 1), col = (i >> 1) * 4 + c;
            const int panel = col * 16 / C::ROW, x = C::ROW == 64 ? row >> 1 & 3 : row & 7;
            return base + C::OFF_RAW + stage * C::STAGE + panel * C::PANEL + row * C::ROW + ((col % (C::ROW / 16) ^ x) << 4);
        };
        bool ok = true;
        do {
            int tile0, tile1;
            part_of(tile0, tile1);
            const int n = tile1 - tile0;
            const int from = (line.span.lo & ~(C::ALIGN - 1)) + tile0 * TILE;
            const int stop = line.span.hi < from + n * TILE ? line.span.hi : from + n * TILE;
            for (int j = 0; j < n && ok; ++j) {
                const uint32_t g = it + j, stage = g % C::VS;
                if (!(ok = warp_wait(C::BAR_RAW_FULL + stage, g / C::VS & 1, CHUNK_ERR_CONVERT)))
                    break;
                const bool whole = is_whole(smem, g);
                bool nan = false;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint4 v[NL];
#pragma unroll
                    for (int i = 0; i < NL; ++i)
                        ld_shared_v4(raw_at(stage, half, i), v[i].x, v[i].y, v[i].z, v[i].w);
                    if (!whole) {
                        // Rows of the block see different keys of this tile, and a NaN value
                        // times a weight of 0 is NaN: such values become zeros here, and their
                        // places go to the softmax warps.  Keys that no row sees are zeros, too
                        // (without a page, what lies in their place may be anything).
                        uint16_t *const map = reinterpret_cast<uint16_t *>(smem + C::OFF_NAN + (g & 3) * C::NAN_BYTES);
#pragma unroll
                        for (int i = 0; i < NL; ++i) {
                            const int row = half * C::HALF + row0 + 32 * (i & 1), pos = from + j * TILE + row;
                            const uint32_t sc = group_word(smem, g, row >> 4);
                            const bool seen = (sc & PAGE_BIT) && pos >= line.span.lo && pos < stop;
                            uint32_t m = nan_bits(v[i].x) | nan_bits(v[i].y) << 4 | nan_bits(v[i].z) << 8 | nan_bits(v[i].w) << 12;
                            m = !seen ? 0 : (sc >> 8 & 255) == 255 ? 0xffffu : m;
                            v[i] = seen ? make_uint4(without_nan(v[i].x), without_nan(v[i].y), without_nan(v[i].z), without_nan(v[i].w))
                                        : make_uint4(0, 0, 0, 0);
                            nan |= m != 0;
                            map[row * (D / 16) + (i >> 1) * 4 + c] = static_cast<uint16_t>(m);
                        }
                        if (half) {
                            nan = __any_sync(0xffffffffu, nan);
                            if (lane == 0)   // one byte a warp
                                smem[C::OFF_FLAGS + (g & 3) * 4 + w] = nan;
                        }
                    }
                    if (half)
                        warp_arrive(C::BAR_RAW_EMPTY + stage);
                    const uint32_t item = 2 * g + half, buf = item % C::VB;
                    if (item >= C::VB && !(ok = warp_wait(C::BAR_V_EMPTY + buf, (item / C::VB - 1) & 1, CHUNK_ERR_CONVERT)))
                        break;
#pragma unroll
                    for (int i = 0; i < NL; ++i)
                        store_f16(base + C::OFF_V + buf * C::V_BYTES + (i >> 1) * C::V_PANEL + (row0 + 32 * (i & 1)) * 128, row0,
                                  c * 2, v[i]);
                    fence_proxy_async_shared();
                    warp_arrive(C::BAR_V_FULL + buf);
                }
            }
            it += n;
        } while (ok && next_unit());
    } else {
        // ============================================ softmax: two threads a row
        if constexpr (C::REG_SPLIT)
            setmaxnreg_inc<C::REG_SOFTMAX>();
        // row tile, row in it; keys 64 half .. of a tile, columns D / 2 half .. of O
        const int rt = warp >> 3, row = tid & 127, half = warp >> 2 & 1;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float scale_log2 = a.scale * 1.4426950408889634f;
        const uint32_t o_addr = tmem + lanes + C::TM_O + rt * D, s_addr = tmem + lanes + C::TM_S + rt * TILE,
                       p_addr = tmem + lanes + C::TM_P + rt * C::P_STEP;
        // the row tile's warps; all of them
        auto tile_sync = [&] { asm volatile("bar.sync %0, 256;" ::"r"(1 + rt) : "memory"); };
        auto all_sync = [] { asm volatile("bar.sync 11, %0;" ::"n"(256 * C::NQ) : "memory"); };
        // the two warps of the same rows
        const int pair_id = 3 + rt * 4 + (warp & 3);
        auto pair_sync = [&] { asm volatile("bar.sync %0, 64;" ::"r"(pair_id) : "memory"); };
        auto pair_any = [&](bool x) -> bool {
            uint32_t r;
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
                         "bar.red.or.pred p, %1, 64, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                         : "=r"(r)
                         : "r"(pair_id), "r"(static_cast<uint32_t>(x))
                         : "memory");
            return r != 0;
        };
        float *const pair = reinterpret_cast<float *>(smem + C::OFF_PAIR);   // by thread
        // A wait that ran out is recorded and not waited for again: the role runs on to its end
        // without waiting (its outputs are undefined), so that barriers between warps still match.
        bool ok = true;
        auto wait = [&](int i, uint32_t parity) {
            if (ok)
                ok = warp_wait(i, parity, CHUNK_ERR_SOFTMAX);
        };
        uint32_t n_done = 0, loads = 0;                        // of this row tile: tiles of keys, and loads of Q
        do {
            int tile0, tile1;
            part_of(tile0, tile1);
            const int n = tile1 - tile0;
            const bool twin = is_twin();
            const int every = twin ? 2 : 1, j0 = twin ? rt : 0;   // this row tile's tiles of keys
            const int row_at = twin ? row : rt * 128 + row;       // its row in the unit
            const int from = (line.span.lo & ~(C::ALIGN - 1)) + tile0 * TILE;
            const int rr = line.rb * R + row_at;
            const bool live = rr < line.s.n * a.G;
            const int tok = rr / a.G, hq = line.h * a.G + rr % a.G;
            int lo = 0, hi = 0;                                  // keys the row sees
            {
                const int pos = line.s.kv - line.s.n + tok;
                if (live)
                    hi = a.causal ? pos + 1 : line.s.kv;
                const long long x = static_cast<long long>(pos) - a.window;
                lo = a.window >= 0 && x > 0 ? static_cast<int>(x) : 0;
            }
            // ---- this row of Q as two e4m3 terms, times the power of two that brings its
            // largest magnitude to [224, 448); each thread stores half of it
            int e;
            {
                const uint16_t *q =
                    static_cast<const uint16_t *>(a.q) + line.b * a.q_sb + hq * a.q_sh + tok * a.q_sl + half * (D / 2);
                uint4 x[D / 16];
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
                    x[c] = live ? __ldg(reinterpret_cast<const uint4 *>(q) + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        top = max(top, max(w[k] & 0x7fffu, w[k] >> 16 & 0x7fffu));
                }
                pair[tid] = __uint_as_float(top);
                pair_sync();
#pragma unroll 1
                for (int i = warp >= C::WARP_CONVERT - 4 ? a.naps : 0; i > 0; --i)
                    __nanosleep(500);
                top = max(top, __float_as_uint(pair[tid ^ 128]));
                // 448 = 1.75 * 2^8
                e = static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7fu) >= 0x60u ? 1 : 0);
                e = e < -126 ? -126 : e;
                // a row with an infinity or NaN has no finite scores: make it NaN
                const float f = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : pow2i(-e);
                const bool loads_q = !twin || rt == 0;
                // (both have read before either writes the next number there: the scores wait
                // for the warps that store q, but not for a twin's second)
                if (!loads_q)
                    pair_sync();
                if (loads_q && loads > 0)
                    wait(C::BAR_Q_EMPTY + rt, (loads - 1) & 1);
                if (loads_q) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t t0[4], t1[4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t w[4] = {x[c * 2 + i].x, x[c * 2 + i].y, x[c * 2 + i].z, x[c * 2 + i].w};
#pragma unroll
                            for (int k = 0; k < 4; k += 2) {
                                uint32_t y0 = pack_f16x2(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xffff0000u) * f);
                                uint32_t y1 = pack_f16x2(__uint_as_float(w[k + 1] << 16) * f, __uint_as_float(w[k + 1] & 0xffff0000u) * f);
                                t0[i * 2 + k / 2] = take_term<1>(y0) | take_term<1>(y1) << 16;
                                t1[i * 2 + k / 2] = take_term<1>(y0) | take_term<1>(y1) << 16;
                            }
                        }
                        const int col = half * (D / 32) + c, panel = col * 16 / C::ROW, swizzle = C::ROW == 64 ? row >> 1 & 3 : row & 7;
                        const uint32_t at = base + C::OFF_Q + rt * C::Q_TILE + panel * C::Q_PANEL + row * C::ROW +
                                            ((col % (C::ROW / 16) ^ swizzle) << 4);
                        st_shared_v4(at, t0[0], t0[1], t0[2], t0[3]);
                        st_shared_v4(at + C::Q_TERM, t1[0], t1[1], t1[2], t1[3]);
                    }
                    fence_proxy_async_shared();
                    warp_arrive(C::BAR_Q_FULL + rt);
                    ++loads;
                }
            }

            const float scale_row = scale_log2 * pow2i(e);
            float M = -INFINITY, l = 0.f;                        // (M: the same in both threads)
            // values of O that a visible NaN value makes NaN (the first thread's to set)
            uint32_t *const mark = reinterpret_cast<uint32_t *>(smem + C::OFF_MARK) + rt * 128 + row;   // word w: [w * R]
            if (half == 0)
#pragma unroll
                for (int w = 0; w < C::NAN_WORDS; ++w)
                    mark[w * R] = 0;
            for (int j = j0; j < n; j += every) {
                const uint32_t g = it + j, d = n_done + (twin ? j >> 1 : j);
                const bool fresh = j < every, last = j + every >= n;   // the first of them, the last
                wait(C::BAR_S_FULL + rt, d & 1);
                tc_fence_after();
                const float4 *const info = reinterpret_cast<const float4 *>(smem + C::OFF_INFO + g % C::RING * C::INFO_BYTES);
                const int pos0 = from + j * TILE;
                const bool whole = is_whole(smem, g);
                if (!whole) {            // NaN values, once the tile's are converted
                    for (uint32_t item = 2 * g; item < 2 * g + 2; ++item)
                        wait(C::BAR_V_FULL + item % C::VB, item / C::VB & 1);
                    if (half == 0 && *reinterpret_cast<const uint32_t *>(smem + C::OFF_FLAGS + (g & 3) * 4)) {
                        const uint32_t *map = reinterpret_cast<const uint32_t *>(smem + C::OFF_NAN + (g & 3) * C::NAN_BYTES);
#pragma unroll 1
                        for (int k = 0; k < TILE; ++k)
                            if (pos0 + k >= lo && pos0 + k < hi)
#pragma unroll
                                for (int w = 0; w < C::NAN_WORDS; ++w)
                                    mark[w * R] |= map[k * C::NAN_WORDS + w];
                    }
                }
                // Scores that the row does not see become -inf where they are: the passes over them
                // below, the same for every tile, then have no branch to keep their parts apart.
                if (!whole) {
#pragma unroll 1
                    for (int i = 0; i < GROUPS / 2; ++i) {
                        uint32_t r[CHUNK];
                        tmem_ld(s_addr + half * C::HALF + i * CHUNK, r);
                        tmem_wait_ld();
                        tmem_pin(r);
                        const uint32_t word = __float_as_uint(info[half * (GROUPS / 2) + i].w);
                        const bool page = word & PAGE_BIT, nan_scale = (word & 255) == 255;
                        const int key0 = pos0 + half * C::HALF + i * CHUNK;
#pragma unroll
                        for (int k = 0; k < CHUNK; ++k) {
                            const bool see = page && key0 + k >= lo && key0 + k < hi;
                            r[k] = !see ? 0xff800000u : nan_scale ? 0x7fc00000u : r[k];
                        }
                        tmem_st16(s_addr + half * C::HALF + i * CHUNK, r);
                    }
                    tmem_st_wait();
                }
                // this thread's scores, 16 at a time
                auto for_groups = [&](auto f) {
                    uint32_t r[2][CHUNK];
                    tmem_ld(s_addr + half * C::HALF, r[0]);
#pragma unroll
                    for (int i = 0; i < GROUPS / 2; ++i) {
                        tmem_wait_ld();
                        tmem_pin(r[i & 1]);
                        if (i + 1 < GROUPS / 2)
                            tmem_ld(s_addr + half * C::HALF + (i + 1) * CHUNK, r[(i + 1) & 1]);
                        const float4 scales = info[half * (GROUPS / 2) + i];
                        // (not 0: a hidden score is -inf * c)
                        f(i, r[i & 1], fmaxf(scale_row * scales.x, 1.17549435e-38f), scales.y, scales.z);
                    }
                };
                // Weights as f16 pairs, by the maximum so far.  Their sum tells whether one is
                // too large for it: only then (and for a row's first keys, and scores past LARGE) is
                // the tile's maximum taken, O and l brought to it, and the weights taken again.
                uint32_t p[32];
                float sum, add_l;
                bool waited = fresh;
                float ref = 6.f - (M == -INFINITY ? 0.f : M);
                bool again = __any_sync(0xffffffffu, fabsf(M) > LARGE);   // (or no maximum yet)
                for (int attempt = 0; attempt < 2; ++attempt) {
                    if (again) {
                        float top = -INFINITY;   // of x + ev
                        for_groups([&](int, const uint32_t (&r)[CHUNK], float c, float ev, float) {
                            float t = __uint_as_float(r[0]);
#pragma unroll
                            for (int k = 1; k < CHUNK - 1; k += 2)
                                t = max3(t, __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
                            t = fmaxf(t, __uint_as_float(r[CHUNK - 1]));
                            top = fmaxf(top, fmaf(t, c, ev));
                        });
                        pair[tid] = top;
                        pair_sync();
                        top = fmaxf(top, pair[tid ^ 128]);
                        float f = 1.f;
                        if (top > M) {
                            f = ex2_approx(M - top);
                            M = top;
                            l *= f;
                        }
                        if (!fresh) {            // O in tensor memory stands for the old maximum
                            if (!waited)
                                wait(C::BAR_O_DONE + rt, (d - 1) & 1);
                            waited = true;
                            tc_fence_after();
#pragma unroll 1
                            for (int cc = half * (D / 32); cc < (half + 1) * (D / 32); ++cc) {
                                uint32_t o[16];
                                tmem_ld(o_addr + 16 * cc, o);
                                tmem_wait_ld();
                                tmem_pin(o);
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                                tmem_st16(o_addr + 16 * cc, o);
                            }
                        }
                        // M is rounded, and S c + ev - M below is not: at scores past 2^20 the two would
                        // be apart by more than a little.  There the scores become those of x - M, x + ev
                        // rounded as M was, where they are, and the reference 0.  (M is the tile's own
                        // maximum or above it by now, so no further attempt finds them changed.)
                        const bool moved = fabsf(M) > LARGE && M != -INFINITY;
                        ref = 6.f - (M == -INFINITY || moved ? 0.f : M);
                        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll 1
                            for (int i = 0; i < TILE / 8; ++i) {   // (four at a time: registers)
                                uint32_t r[4];
                                tmem_ld(s_addr + half * C::HALF + i * 4, r);
                                tmem_wait_ld();
                                tmem_pin(r);
                                const float4 scales = info[half * (GROUPS / 2) + i / 4];
                                const float c = fmaxf(scale_row * scales.x, 1.17549435e-38f), inv = rcp_approx(c);
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const float x = (fmaf(__uint_as_float(r[k]), c, scales.y) - M - scales.y) * inv;
                                    r[k] = moved ? __float_as_uint(x) : r[k];
                                }
                                tmem_st(s_addr + half * C::HALF + i * 4, r);
                            }
                            tmem_st_wait();
                        }
                    }
                    // weights apart go where the tile before's were, as they are made
                    if (C::P_APART && !waited) {
                        wait(C::BAR_O_DONE + rt, (d - 1) & 1);
                        waited = true;
                        tc_fence_after();
                    }
                    sum = add_l = 0.f;
                    for_groups([&](int i, const uint32_t (&r)[CHUNK], float c, float ev, float lf) {
                        const float add = ev + ref;
                        const uint64_t c2 = f32x2(c, c), add2 = f32x2(add, add);
                        uint64_t sum2 = 0;
#pragma unroll
                        for (int k = 0; k < CHUNK; k += 2) {
                            float x0, x1;
                            unpack_f32x2(fma_f32x2(f32x2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), c2, add2), x0, x1);
                            x0 = ex2_approx(x0);
                            x1 = ex2_approx(x1);
                            sum2 = add_f32x2(sum2, f32x2(x0, x1));
                            p[i * 8 + k / 2] = pack_f16x2(x0, x1);
                        }
                        if (C::P_APART && i % 2)
                            tmem_st16(p_addr + half * 32 + i / 2 * 16, p + i / 2 * 16);
                        float sum0, sum1;
                        unpack_f32x2(sum2, sum0, sum1);
                        sum += sum0 + sum1;
                        add_l = fmaf(sum0 + sum1, lf, add_l);
                    });
                    // (f16 ends at 65504; by the tile's own maximum the sum is 2^12 at most.)  Both
                    // threads have read their scores after this, which the weights may go over.
                    again = pair_any(sum > 32768.f);
                    if (!again)
                        break;
                }
                l += add_l;
                if (!C::P_APART) {
                    // Over the scores: the products that made these came after the tile before's.
                    // But a parity tells a phase from the one before only, so the wait for the
                    // last tile's product (below) needs that for the last but one's, before the
                    // last can complete.
                    if (!waited && last)
                        wait(C::BAR_O_DONE + rt, (d - 1) & 1);
                    tmem_st32(p_addr + half * 32, p);
                }
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(C::BAR_P_FULL + rt);
            }

            // ---- O out of tensor memory: the unit's rows, or this part of them
            it += n;
            const int mine = twin ? (n + 1 - rt) >> 1 : n;
            n_done += mine;
            pair[tid] = l;
            pair_sync();
            l = (half ? pair[tid ^ 128] : l) + (half ? l : pair[tid ^ 128]);   // (in one order)
            if (mine > 0)
                wait(C::BAR_O_DONE + rt, (n_done - 1) & 1);
            // Twins: both tiles' maxima and sums; each tile's warps then take half of the columns.
            float f0 = 1.f, f1 = 0.f;
            if (twin) {
                float2 *const sums = reinterpret_cast<float2 *>(smem + C::OFF_SUM) + row;
                if (half == 0)
                    sums[rt * 128] = make_float2(M, l);
                tc_fence_before();
                all_sync();
                const float2 x = sums[0], y = sums[128];
                M = fmaxf(x.x, y.x);
                const float ref = M == -INFINITY ? 0.f : M;
                f0 = ex2_approx(x.x - ref);
                f1 = ex2_approx(y.x - ref);
                l = x.y * f0 + y.y * f1;
            }
            tc_fence_after();
            const int first_cta = cut ? sh.range.owner(line.at) : cta;
            const int last_cta = cut ? sh.range.owner(line.at + line.span.tiles - 1) : cta;
            const bool alone = first_cta == last_cta;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const float2 lse2 = l == 0.f ? make_float2(-INFINITY, 0.f) : two_floats(M, lg2_approx(l) - 6.f);
            uint16_t *const o = static_cast<uint16_t *>(a.o) + line.b * a.o_sb + hq * a.o_sh + tok * a.o_sl;
            float *const part =
                cut ? parts.data + (2 * static_cast<size_t>(cta) + (cta == first_cta ? 1 : 0)) * Parts::slot_floats(R, D) : nullptr;
            // a part's quadruple u of columns: neighbouring threads' rows lie next to each other
            auto place = [&](int u) { return (u * R + row_at) * 4; };
            const int chunk0 = twin ? rt * 2 + half : half, chunks = twin ? 4 : 2;   // of 16 columns: the first, every
#pragma unroll 1
            for (int cc = chunk0; cc < D / 16; cc += chunks) {
                uint32_t r[16];
                tmem_ld((twin ? o_addr - rt * D : o_addr) + 16 * cc, r);
                tmem_wait_ld();
                tmem_pin(r);
                uint32_t marked = mark[(cc >> 1) * R];
                if (twin) {
                    marked |= mark[(cc >> 1) * R + (rt ? -128 : 128)];
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        r[k] = __float_as_uint(__uint_as_float(r[k]) * f0);
                    if (n > 1) {
                        uint32_t r1[16];
                        tmem_ld(o_addr + (1 - rt) * D + 16 * cc, r1);
                        tmem_wait_ld();
                        tmem_pin(r1);
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            r[k] = __float_as_uint(fmaf(__uint_as_float(r1[k]), f1, __uint_as_float(r[k])));
                    }
                }
                marked >>= (cc & 1) * 16;
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    r[k] = (marked >> k & 1) ? 0x7fc00000u : __float_as_uint(__uint_as_float(r[k]) * inv);
                if (alone && live) {
#pragma unroll
                    for (int k = 0; k < 16; k += 8)
                        *reinterpret_cast<uint4 *>(o + cc * 16 + k) =
                            make_uint4(pack_bf16x2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])),
                                       pack_bf16x2(__uint_as_float(r[k + 2]), __uint_as_float(r[k + 3])),
                                       pack_bf16x2(__uint_as_float(r[k + 4]), __uint_as_float(r[k + 5])),
                                       pack_bf16x2(__uint_as_float(r[k + 6]), __uint_as_float(r[k + 7])));
                } else if (!alone) {
#pragma unroll
                    for (int k = 0; k < 16; k += 4)
                        *reinterpret_cast<uint4 *>(part + place(cc * 4 + k / 4)) = make_uint4(r[k], r[k + 1], r[k + 2], r[k + 3]);
                }
            }
            tc_fence_before();
            auto write_lse = [&](float v) {
                a.lse[(static_cast<long long>(line.b) * a.Hq + hq) * a.Lq + tok] = v * 0.69314718055994531f;
            };
            if (alone) {
                if (chunk0 == 0 && live)
                    write_lse(lse2.x);
            } else {
                if (chunk0 == 0)
                    reinterpret_cast<float2 *>(part + R * D)[row_at] = lse2;
                // the CTA whose part is the last to arrive merges them, each row tile by itself
                // (twins together)
                auto sync = [&] {
                    if (twin)
                        all_sync();
                    else
                        tile_sync();
                };
                __threadfence();
                sync();
                const int tile = twin ? 0 : rt;
                volatile int *const last = reinterpret_cast<int *>(smem + C::OFF_MISC + 4) + tile;
                if ((tid & 255) == 0 && rt == tile) {
                    int *const counter = parts.counters + 2 * first_cta + tile;
                    *last = atomicAdd(counter, 1) == last_cta - first_cta;
                    if (*last)
                        *counter = 0;
                }
                sync();
                if (*last) {
                    __threadfence();
#pragma unroll 1
                    for (int cc = chunk0; cc < D / 16; cc += chunks) {
                        float4 v[4];
                        const float merged =
                            merge_row<C, 4, 2>(parts, first_cta, last_cta, row_at, [&](int k) { return place(cc * 4 + k); }, v);
                        if (live) {
#pragma unroll
                            for (int k = 0; k < 4; k += 2)
                                *reinterpret_cast<uint4 *>(o + cc * 16 + k * 4) =
                                    make_uint4(pack_bf16x2(v[k].x, v[k].y), pack_bf16x2(v[k].z, v[k].w),
                                               pack_bf16x2(v[k + 1].x, v[k + 1].y), pack_bf16x2(v[k + 1].z, v[k + 1].w));
                            if (cc == 0)
                                write_lse(merged);
                        }
                    }
                }
            }
            // the marks and O are read
            if (twin)
                all_sync();
            else
                pair_sync();
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
    if (grid == 0)
        return FA2_ERR_UNSUPPORTED;
    const EncodeTiled encode = encode_tiled();
    CUtensorMap k_map, v_map;
    const int rows = 1 << a.c.page_shift;
    if (!encode || !page_map(encode, &k_map, a.c.k, a.c, C::D, rows, C::ROW) ||
        !page_map(encode, &v_map, a.c.v, a.c, C::D, rows, C::ROW))
        return FA2_ERR_CUDA;
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
    chunk_kernel<C><<<grid, C::T, C::SMEM_BYTES, a.stream>>>(k_map, v_map, a, parts);
    return cudaGetLastError() == cudaSuccess ? FA2_OK : FA2_ERR_CUDA;
}
#endif

}  // namespace cache
}  // namespace fa2
