// fa2_cache_step.cuh -- attention of a few query rows over the paged e4m3 cache
// (fa2_cache_attn in include/fa2_cache.h): the step of a decoding server.
//
// The query heads that share a key/value head and the query tokens of a sequence are the
// rows of one small matrix: row r is token r / G, head r % G of the group, so a cache byte
// is read once for all of them.
//
// Mathematics.  The tensor cores take the cache's codes as they are (kind::f8f6f4); what
// multiplies them is split into e4m3 terms:
//     q 2^-e = q0 + 2^-4 q1             (e: largest magnitude of the row in [128, 256))
// is exact for a bf16 q, because e4m3 holds half of bf16's eight bits (an element below
// 2^-14 of its row's largest is off by at most 2^-21 of that); and
//     p = p0 + 2^-4 p1 + 2^-8 p2        (p in [0, 256], first rounded to f16)
// is off by at most 2^-11 of p, or 2^-26 of the tile's largest.  Both products are taken
// transposed, so that the cache is the 128-row operand and the few query rows are columns:
//     S^T [128 keys, 2 R]  = K  [q0 | q1]^T
//     O^T [D, 3 R]         = V^T [p0 | p1 | p2]^T
// A thread owns a key of the tile (S) and a column d (O).  For key j with page exponents
// ek, ev
//     x_j = (S0 + 2^-4 S1) scale log2 e 2^(e + ek),     p_j = 2^(x_j + ev - m + 8)
// with m the least whole number above the tile's maximum of x + ev for the row; a tile's
// O^T is added to fp32 registers times 2^(m - M), M the largest m so far, and
// l += 2^-ev p likewise.  Every tile has a reference of its own, so the terms' small range
// never meets the spread of scores over a long context, and since the references are whole
// numbers the factors are exact.  l sums the weights as they are before their rounding: LSE
// needs that sum, and one of the rounded weights for O alone, in which the rounding of a key
// that dominates would cancel (2^-11 at most, under bf16's 2^-8), would cost R registers and
// the additions.
//
// What bounds it.  One token of a group of 8 does 16 operations a cache byte, the card
// could do 290: the bytes are the time, and no other unit may come near it.  The codes are
// not touched by the threads at all: TMA puts pages of 128 keys into a ring of
// shared-memory slots, one thread issues the products, and 128 threads do the softmax of
// R columns; the copies run ahead by the ring's depth.  Two or three CTAs share an SM, so
// that one's softmax runs under the other's products (D = 128, 16 rows, 131 MB of cache: 49
// us, 61 with one; D = 64, 8 rows: 41 with three, 43 with two).  Work is cut and merged as
// in fa2_cache_line.cuh.
// Measured (several inputs in turn, so that none is in L2): one token of 48 sequences of 64 to
// 8192 positions, 8 heads of 128, groups of 4: 407 MB in 70 us, 5.8 TB/s, 86 % of the
// measured copy rate; of two of 125000: 514 MB in 84.5 us, 6.1 TB/s; D = 256, 16 of 16000, 4
// heads, groups of 8: 525 MB in 87.6 us, 6.0 TB/s, and 8 of 8000, 8 heads: 262 MB in 48.9, 5.4.
// At D = 64 a tile holds half the bytes for the same softmax, and that bounds it: 16 sequences
// of 24000, 8 heads, groups of 8, 394 MB in 102 us, 3.9 TB/s, and of 6000 98 MB in 34, 2.9.  So
// does twice the softmax for 16 rows: D = 128, 16 of 4000, 132 MB in 42.6 us, 3.1 TB/s.  Short
// calls are latency: of 14 us for 34 MB in L2 (a window of 1024 in 16 sequences; 17 from
// memory), 2 go to the launch, 1.5 to laying out the line, 1 to q, 2 to merging parts.
#pragma once

#include <atomic>

#include "fa2_cache_line.cuh"
#include "fa2_cache_tile.cuh"

namespace fa2 {
namespace cache {

template <int D_, int R_>
struct StepCfg {
    static constexpr int D = D_;
    static constexpr int R = R_;                     // query rows of a unit
    static constexpr int TILE = 128;                 // keys
    static constexpr int UNIT_COST = 3, MIN_TILES = 1;   // see fa2_cache_line.cuh
    static constexpr int ALIGN = 128;                // whole pages: a tile begins at a multiple
    static constexpr int CTAS = D == 64 ? (R == 8 ? 3 : 2) : D == 128 ? 2 : 1;   // an SM
    static constexpr int WARP_LOAD = 4, WARP_MMA = 5;
    static constexpr int T = 32 * 6;

    static constexpr int ROW = D == 64 ? 64 : 128;   // bytes of a row in an operand panel: its swizzle span
    static constexpr int PANELS = D / ROW;
    static constexpr int PANEL = TILE * ROW;         // of a slot
    static constexpr int SLOT = TILE * D;            // keys or values of a tile
    static constexpr int SLOTS = D == 256 ? 5 : 6;
    static constexpr int NQ = 2 * R, Q_PANEL = NQ * ROW;            // rows [q0 | q1]
    static constexpr int NP = (3 * R + 15) / 16 * 16;               // rows [p0 | p1 | p2], 128 bytes each
    static constexpr int OFF_RING = 0, OFF_P = SLOTS * SLOT, OFF_Q = OFF_P + NP * 128, OFF_ROWS = OFF_Q + NQ * D;
    // per row: the maxima of the four warps (two tiles), factors of the last two tiles, scale
    // factor, first and last visible key
    static constexpr int OFF_MAX = OFF_ROWS, OFF_FRAME = OFF_MAX + 2 * R * 16, OFF_SCALE = OFF_FRAME + 2 * R * 8;
    static constexpr int OFF_LO = OFF_SCALE + R * 4, OFF_HI = OFF_LO + R * 4, OFF_L = OFF_HI + R * 4;   // (OFF_L: four sums)
    static constexpr int OFF_INV = OFF_L + R * 16, OFF_PLACE = OFF_INV + R * 4;   // 1 / sum; places in o and lse
    static constexpr int OFF_FLAGS = OFF_PLACE + R * 16, OFF_NAN = OFF_FLAGS + 32, OFF_INFO = OFF_NAN + 16;
    static constexpr int INFO_BYTES = TILE / CHUNK * 4, OFF_BAR = OFF_INFO + 4 * INFO_BYTES;   // (ring of four tiles)
    static constexpr int NUM_BAR = 2 * SLOTS + 7;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BAR * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;         // 1024: operand alignment

    static constexpr int TM_S = 0, TM_O = 2 * NQ, HALVES = D == 256 ? 2 : 1;   // O: NP columns for each 128 of d
    static constexpr int TM_USED = TM_O + HALVES * NP;
    static constexpr int TMEM_COLS = TM_USED <= 64 ? 64 : TM_USED <= 128 ? 128 : TM_USED <= 256 ? 256 : 512;

    static constexpr int BAR_FULL = 0, BAR_EMPTY = SLOTS, BAR_Q_FULL = 2 * SLOTS, BAR_Q_EMPTY = BAR_Q_FULL + 1,
                         BAR_S_FULL = BAR_Q_FULL + 2, BAR_P_FULL = BAR_Q_FULL + 4, BAR_O_DONE = BAR_Q_FULL + 5,
                         BAR_DRAIN = BAR_Q_FULL + 6;
    static_assert(SLOTS <= 6, "the ring of four tiles' scales");
    static_assert(R % 8 == 0 && R <= 16 && TM_USED <= 512 && CTAS * TMEM_COLS <= 512, "tensor memory holds CTAS of them");
    static_assert(CTAS * (SMEM_BYTES + 1024 + 512) <= 228 * 1024, "an SM holds CTAS of them");
    static_assert(OFF_P % 1024 == 0 && OFF_Q % 1024 == 0 && Q_PANEL % 512 == 0, "swizzle atoms");
};

// Error codes of waits that ran out (bits 8-11 the waiting role).
constexpr int STEP_ERR_SOFTMAX = 12 << 8, STEP_ERR_LOAD = 13 << 8, STEP_ERR_MMA = 14 << 8, STEP_ERR_DRAIN = 15 << 8;

#ifdef __CUDACC__

// Largest of a warp's values (NaN only if all are).
__device__ __forceinline__ float warp_max(float v)
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

template <class C>
__global__ void __launch_bounds__(C::T, C::CTAS)
    step_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const AttnArgs a,
                const Parts parts)
{
    using namespace ptx;
    constexpr int D = C::D, R = C::R, TILE = C::TILE, SLOTS = C::SLOTS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ LineShared sh_line;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool cut = parts.data != nullptr;
    const int cta = blockIdx.x;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *const smem = smem_raw + (base - smem_u32(smem_raw));
    auto bar = [&](int i) { return base + C::OFF_BAR + 8 * i; };
    volatile uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    // (while the lengths are on their way)
    if (warp == C::WARP_MMA) {
        tmem_alloc(base + C::OFF_MISC, C::TMEM_COLS);
        tmem_relinquish();
    } else if (tid == 32 * C::WARP_LOAD) {
        for (int i = 0; i < C::NUM_BAR; ++i)
            mbar_init(bar(i), i == C::BAR_Q_FULL || i == C::BAR_P_FULL ? 4 : 1);
        fence_mbar_init();
        tma_prefetch_desc(&k_map);
        tma_prefetch_desc(&v_map);
    }
    tc_fence_before();
    Range range;
    int first, end;
    Line<C> line;
    const bool any = find_range<C>(a, cut, sh_line, range, first, end, line);   // (barriers of the CTA in it)
    if (!any) {
        if (warp == C::WARP_MMA) {
            __syncwarp();
            tmem_dealloc(*tmem_slot, C::TMEM_COLS);
        }
        return;
    }
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // A wait that ran out is recorded and not waited for again: the role runs on to its end
    // without waiting (its outputs are undefined), so that barriers between warps still match.
    bool ok = true;
    auto warp_wait = [&](int i, uint32_t parity, int code) {
        if (ok)
            ok = wait_phase(bar(i), parity, a.err, code | i, a.wait_limit_ns);
    };
    auto warp_arrive = [&](int i) {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(i));
    };
    // the tiles of the unit `line` that lie in this CTA's range
    auto part_of = [&](int &tile0, int &tile1) {
        tile0 = cut && first > line.at ? first - line.at : 0;
        tile1 = cut && end < line.at + line.span.tiles ? end - line.at : line.span.tiles;
    };
    auto next_unit = [&]() { return line.next(a, end); };
    uint32_t *const sh_info = reinterpret_cast<uint32_t *>(smem + C::OFF_INFO);   // [4][8 groups of 16 keys]
    // tile g's keys are item 2 g of the ring, its values item 2 g + 1
    uint32_t it = 0, unit = 0;   // tiles and units before the present unit

    if (warp == C::WARP_LOAD) {
        // ============================================ pages -> ring
        const int pages = TILE >> a.c.page_shift;          // of a tile: one a lane
        const uint32_t page_bytes = static_cast<uint32_t>(D) << a.c.page_shift;
        const uint32_t offset = static_cast<uint32_t>(lane) * C::ROW << a.c.page_shift;   // in each panel
        uint32_t issued = 0;                               // items
#pragma unroll 1
        for (int i = a.naps; i > 0; --i)
            __nanosleep(500);
        do {
            int tile0, tile1;
            part_of(tile0, tile1);
            const int n = tile1 - tile0, h = line.h;
            const int from = (line.span.lo & ~(C::ALIGN - 1)) + tile0 * TILE;
            const int stop = line.span.hi < from + n * TILE ? line.span.hi : from + n * TILE;
            auto page_at = [&](int j) {                    // -1: none, or not seen
                const int pos = from + j * TILE + (lane << a.c.page_shift);
                const bool seen = j < n && lane < pages && pos < stop && pos + (1 << a.c.page_shift) > line.span.lo;
                return seen ? page_of(a.c, line.b, pos >> a.c.page_shift) : -1;
            };
            auto scales_of = [&](int page) -> uint32_t {
                if (page < 0)
                    return 0;
                const long long i = static_cast<long long>(page) * a.c.H + h;
                return a.c.k.scale[i] | static_cast<uint32_t>(a.c.v.scale[i]) << 8 | PAGE_BIT;
            };
            int id = page_at(0), id_next = page_at(1);     // pages two tiles ahead, scales one
            uint32_t sc = scales_of(id);
            for (int j = 0; j < n && ok; ++j) {
                const int id_after = page_at(j + 2);
                const uint32_t sc_next = scales_of(id_next);
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, id >= 0)) * page_bytes;
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    const uint32_t item = 2 * (it + j) + side, slot = item % SLOTS, full = bar(C::BAR_FULL + slot);
                    if (item >= SLOTS)
                        warp_wait(C::BAR_EMPTY + slot, (item / SLOTS - 1) & 1, STEP_ERR_LOAD);
                    if (!ok)
                        break;
                    if (lane == 0)
                        expect_tx(full, bytes);
                    __syncwarp();
                    if (id >= 0)
#pragma unroll
                        for (int p = 0; p < C::PANELS; ++p)
                            tma_load_4d(base + C::OFF_RING + slot * C::SLOT + p * C::PANEL + offset, side ? &v_map : &k_map,
                                        p * 128, 0, h, id, full);
                    // The keys' copies are under way while the scales arrive.  (Whose place the
                    // tile four back had: it has been through its softmax, for its values' slot
                    // came back before the last tile was loaded.)
                    if (side == 0 && lane < pages)
                        for (int k = 0; k < 1 << (a.c.page_shift - 4); ++k)
                            sh_info[((it + j) & 3) * (TILE / CHUNK) + (lane << (a.c.page_shift - 4)) + k] = sc;
                    warp_arrive(C::BAR_FULL + slot);
                    issued = item + 1;
                }
                id = id_next;
                id_next = id_after;
                sc = sc_next;
            }
            it += n;
        } while (ok && next_unit());
        // the copies in flight have landed before the CTA goes
        for (uint32_t item = issued > SLOTS ? issued - SLOTS : 0; item < issued; ++item) {
            const int i = C::BAR_FULL + item % SLOTS;
            wait_phase(bar(i), item / SLOTS & 1, a.err, STEP_ERR_DRAIN | i, a.drain_limit_ns);
        }
    } else if (warp == C::WARP_MMA) {
        // ============================================ one thread issues the products
        if (elect_one()) {
            const uint64_t desc_q = D == 64 ? sdesc_sw64(base + C::OFF_Q, 16, 512) : sdesc_sw128(base + C::OFF_Q, 16, 1024);
            const uint64_t desc_p = sdesc_sw128(base + C::OFF_P, 16, 1024);
            const uint64_t desc_k = D == 64 ? sdesc_sw64(base, 16, 512) : sdesc_sw128(base, 16, 1024);
            // V^T: d is the contiguous direction.  At D = 64 the 128 rows are the 64 columns
            // twice (stride 0), and lanes 64.. of O^T a copy that nobody reads.
            const uint64_t desc_v = D == 64 ? sdesc_sw64(base, 0, 512) : sdesc_sw128(base, 16, 1024);
            auto wait = [&](int i, uint32_t parity) {
                if (ok)
                    ok = lone_wait(bar(i), parity, a.err, STEP_ERR_MMA | i, a.wait_limit_ns);
            };
            auto wait_item = [&](uint32_t item) { wait(C::BAR_FULL + item % SLOTS, item / SLOTS & 1); };
            auto issue_s = [&](uint32_t g, bool last) {
                wait_item(2 * g);
                tc_fence_after();
                const uint32_t slot = 2 * g % SLOTS;
                const uint64_t dk = desc_k + (C::OFF_RING + slot * C::SLOT >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk) {
                    const int panel = kk * 32 / C::ROW, col = kk * 32 % C::ROW;
                    mma_ss<true>(tmem + C::TM_S + (g & 1) * C::NQ, dk + (panel * C::PANEL + col >> 4),
                                 desc_q + (panel * C::Q_PANEL + col >> 4), idesc_e4m3_f32(128, C::NQ, false, false), kk > 0);
                }
                mma_commit(bar(C::BAR_S_FULL + (g & 1)));
                mma_commit(bar(C::BAR_EMPTY + slot));
                if (last)
                    mma_commit(bar(C::BAR_Q_EMPTY));
            };
            auto issue_pv = [&](uint32_t g) {
                wait_item(2 * g + 1);
                wait(C::BAR_P_FULL, g & 1);
                tc_fence_after();
                const uint32_t slot = (2 * g + 1) % SLOTS;
                const uint64_t dv = desc_v + (C::OFF_RING + slot * C::SLOT >> 4);
#pragma unroll
                for (int half = 0; half < C::HALVES; ++half)
#pragma unroll
                    for (int kk = 0; kk < TILE / 32; ++kk)
                        mma_ss<true>(tmem + C::TM_O + half * C::NP, dv + (half * C::PANEL + kk * 32 * C::ROW >> 4),
                                     desc_p + (kk * 32 >> 4), idesc_e4m3_f32(128, C::NP, true, false), kk > 0);
                mma_commit(bar(C::BAR_O_DONE));
                mma_commit(bar(C::BAR_EMPTY + slot));
            };
            do {
                int tile0, tile1;
                part_of(tile0, tile1);
                const int n = tile1 - tile0;
                wait(C::BAR_Q_FULL, unit & 1);
                if (ok)
                    issue_s(it, n == 1);
                for (int j = 0; j < n && ok; ++j) {
                    // (its S buffer was read before the weights of the tile two back were ready)
                    if (j + 1 < n)
                        issue_s(it + j + 1, j + 2 == n);
                    if (ok)
                        issue_pv(it + j);
                }
                it += n;
                ++unit;
            } while (ok && next_unit());
            // nothing issued is still running when tensor memory is given back
            mma_commit(bar(C::BAR_DRAIN));
            lone_wait(bar(C::BAR_DRAIN), 0, a.err, STEP_ERR_DRAIN | C::BAR_DRAIN, a.drain_limit_ns);
        }
        __syncwarp();
    } else {
        // ============================================ softmax: thread = key of S^T, column d of O^T
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        const float scale_log2 = a.scale * 1.4426950408889634f;
        float *const sh_max = reinterpret_cast<float *>(smem + C::OFF_MAX);           // [2][R][4]
        float2 *const sh_frame = reinterpret_cast<float2 *>(smem + C::OFF_FRAME);     // [2][R]
        float *const sh_scale = reinterpret_cast<float *>(smem + C::OFF_SCALE);       // [R]
        int *const sh_lo = reinterpret_cast<int *>(smem + C::OFF_LO), *const sh_hi = reinterpret_cast<int *>(smem + C::OFF_HI);
        float *const sh_l = reinterpret_cast<float *>(smem + C::OFF_L);               // [R][4]
        float *const sh_inv = reinterpret_cast<float *>(smem + C::OFF_INV);           // [R]
        longlong2 *const sh_place = reinterpret_cast<longlong2 *>(smem + C::OFF_PLACE);   // [R]; -1: not a row
        volatile uint32_t *const sh_flags = reinterpret_cast<uint32_t *>(smem + C::OFF_FLAGS);   // [2][4]
        volatile uint32_t *const sh_nan = reinterpret_cast<uint32_t *>(smem + C::OFF_NAN);       // [4]
        auto sync = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };            // the four softmax warps
        constexpr float NONE = -3.402823466e38f;   // reference of nothing: no finite score lies below it
        const bool owns_d = D > 64 || tid < 64;

        do {
            int tile0, tile1;
            part_of(tile0, tile1);
            const int n = tile1 - tile0, b = line.b, h = line.h, rb = line.rb;
            const Seq s = line.s;
            const Span span = line.span;
            const int from = (span.lo & ~(C::ALIGN - 1)) + tile0 * TILE;
            const int stop = span.hi < from + n * TILE ? span.hi : from + n * TILE;
            const int rows = s.n * a.G, live = rows - rb * R;   // rows of the block (four at a time below)
            int all_lo, all_hi;
            line.seen_by_all(a, all_lo, all_hi);

            // ---- Q as two e4m3 terms; TPR threads a row
            if (unit > 0)
                warp_wait(C::BAR_Q_EMPTY, (unit - 1) & 1, STEP_ERR_SOFTMAX);
            {
                constexpr int TPR = 128 / R, E = D / TPR;   // threads a row, elements a thread
                const int r = tid / TPR, d0 = tid % TPR * E;
                const int rr = rb * R + r, tok = rr / a.G, hq = h * a.G + rr % a.G;
                const bool is_row = rr < rows;
                const uint16_t *q = static_cast<const uint16_t *>(a.q) + b * a.q_sb + hq * a.q_sh + tok * a.q_sl + d0;
                uint2 w[E / 4];
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < E / 4; ++k) {
                    w[k] = is_row ? __ldg(reinterpret_cast<const uint2 *>(q) + k) : make_uint2(0, 0);
                    const uint32_t m0 = max(w[k].x & 0x7fffu, w[k].x >> 16 & 0x7fffu), m1 = max(w[k].y & 0x7fffu, w[k].y >> 16 & 0x7fffu);
                    top = max(top, max(m0, m1));
                }
#pragma unroll
                for (int d = 1; d < TPR; d <<= 1)
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                int e = static_cast<int>(top >> 7) - 127 - 7;
                e = e < -126 ? -126 : e;   // 2^126 is as far as fp32 goes (zero and subnormal rows)
                // a row with an infinity or NaN has no finite scores: make it NaN
                const float f = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : pow2i(-e);
#pragma unroll
                for (int k = 0; k < E / 4; ++k) {
                    uint32_t x01 = pack_f16x2(__uint_as_float(w[k].x << 16) * f, __uint_as_float(w[k].x & 0xffff0000u) * f);
                    uint32_t x23 = pack_f16x2(__uint_as_float(w[k].y << 16) * f, __uint_as_float(w[k].y & 0xffff0000u) * f);
                    const int d = d0 + 4 * k, panel = d / C::ROW, col = d % C::ROW;
#pragma unroll
                    for (int term = 0; term < 2; ++term) {
                        const uint32_t lo = take_term<16>(x01), hi = take_term<16>(x23);
                        const int row = term * R + r, x = C::ROW == 64 ? row >> 1 & 3 : row & 7;
                        *reinterpret_cast<uint32_t *>(smem + C::OFF_Q + panel * C::Q_PANEL + row * C::ROW +
                                                      (((col >> 4) ^ x) << 4) + (col & 15)) = lo | hi << 16;
                    }
                }
                if (tid % TPR == 0) {
                    const int pos = s.kv - s.n + tok;
                    const long long lo = static_cast<long long>(pos) - a.window;
                    sh_scale[r] = scale_log2 * pow2i(e);
                    sh_hi[r] = !is_row ? 0 : a.causal ? pos + 1 : s.kv;
                    sh_lo[r] = a.window >= 0 && lo > 0 ? static_cast<int>(lo) : 0;
                    sh_place[r] = make_longlong2(is_row ? b * a.o_sb + hq * a.o_sh + tok * a.o_sl : -1,
                                                 (static_cast<long long>(b) * a.Hq + hq) * a.Lq + tok);
                }
                fence_proxy_async_shared();
                warp_arrive(C::BAR_Q_FULL);
            }
            const int first_cta = cut ? range.owner(line.at) : cta;
            const int last_cta = cut ? range.owner(line.at + span.tiles - 1) : cta;
            const bool alone = first_cta == last_cta;
            float *const part =
                cut ? parts.data + (2 * static_cast<size_t>(cta) + (cta == first_cta ? 1 : 0)) * Parts::slot_floats(R, D) : nullptr;
            sync();   // the rows' scales and limits are there

            float acc[C::HALVES][R], l[R], psum[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                acc[0][r] = acc[C::HALVES - 1][r] = 0.f;
                l[r] = psum[r] = 0.f;
            }
            uint32_t nan_rows[C::HALVES] = {};   // rows whose O at this d a visible NaN value makes NaN
            // The row's reference (threads below R): a float, for scores may be any; a difference of two
            // is whole, or far past what a factor can be.
            float M = NONE;

            // O^T of the tile before `g` into the registers, in the row's new frame
            auto add_tile = [&](uint32_t g) {
                warp_wait(C::BAR_O_DONE, (g - 1) & 1, STEP_ERR_SOFTMAX);
                tc_fence_after();
                const float2 *frame = sh_frame + ((g - 1) & 1) * R;
#pragma unroll
                for (int r0 = 0; r0 < R; r0 += 4) {
                    if (r0 >= live)
                        break;
#pragma unroll
                    for (int half = 0; half < C::HALVES; ++half) {
                        uint32_t t0[4], t1[4], t2[4];
                        const uint32_t addr = tmem + lanes + C::TM_O + half * C::NP + r0;
                        tmem_ld(addr, t0);
                        tmem_ld(addr + R, t1);
                        tmem_ld(addr + 2 * R, t2);
                        tmem_wait_ld();
                        tmem_pin(t0);
                        tmem_pin(t1);
                        tmem_pin(t2);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int r = r0 + k;
                            const float2 f = frame[r];   // old frame -> new, tile -> new
                            const float o = fmaf(__uint_as_float(t2[k]), 1.f / 256.f,
                                                 fmaf(__uint_as_float(t1[k]), 1.f / 16.f, __uint_as_float(t0[k])));
                            acc[half][r] = fmaf(o, f.y, acc[half][r] * f.x);
                            if (half == 0)
                                l[r] = fmaf(psum[r], f.y, l[r] * f.x);
                        }
                    }
                }
                tc_fence_before();
            };

            for (int j = 0; j < n; ++j) {
                const uint32_t g = it + j, par = g & 1;
                const int pos = from + j * TILE + tid;
                warp_wait(C::BAR_S_FULL + par, g >> 1 & 1, STEP_ERR_SOFTMAX);
                tc_fence_after();
                const uint32_t sc = sh_info[(g & 3) * (TILE / CHUNK) + (tid >> 4)];
                const int ek = static_cast<int>(sc & 255) - 127;
                const bool there = sc != 0 && pos >= span.lo && pos < stop, nan_scale = there && (sc >> 8 & 255) == 255;
                const int ev = there && !nan_scale ? static_cast<int>(sc >> 8 & 255) - 127 : 0;
                const float kf = ek == 128 ? __uint_as_float(0x7fc00000u) : pow2i(ek);
                const bool whole = there && !nan_scale && pos >= all_lo && pos < all_hi;   // every row sees the key
                float x[R];               // x + ev
#pragma unroll
                for (int r0 = 0; r0 < R; r0 += 4) {
                    if (r0 >= live)
                        break;
                    uint32_t s0[4], s1[4];
                    tmem_ld(tmem + lanes + C::TM_S + par * C::NQ + r0, s0);
                    tmem_ld(tmem + lanes + C::TM_S + par * C::NQ + R + r0, s1);
                    tmem_wait_ld();
                    tmem_pin(s0);
                    tmem_pin(s1);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[r0 + k] = fmaf(fmaf(__uint_as_float(s1[k]), 1.f / 16.f, __uint_as_float(s0[k])), sh_scale[r0 + k] * kf,
                                         static_cast<float>(ev));
                    if (!whole)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            x[r0 + k] = there && pos >= sh_lo[r0 + k] && pos < sh_hi[r0 + k] ? x[r0 + k] : -INFINITY;
                    // the rows' maxima over the warp's keys
                    float mine = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float m = warp_max(x[r0 + k]);
                        mine = lane == k ? m : mine;
                    }
                    if (lane < 4)
                        sh_max[(par * R + r0 + lane) * 4 + warp] = mine;
                }
                tc_fence_before();
                {
                    const bool some = __any_sync(0xffffffffu, !whole);
                    if (lane == 0)
                        sh_flags[par * 4 + warp] = some;
                }
                sync();
                // the tile's references, above the maxima; a row's frame is moved by its own thread
                auto reference = [&](int r) {
                    const float4 m4 = *reinterpret_cast<const float4 *>(sh_max + (par * R + r) * 4);
                    return fmaxf(ceilf(fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w))), NONE);
                };
                if (tid < R && tid < live) {
                    auto factor = [](float down) { return pow2i(static_cast<int>(fmaxf(down, -200.f))); };   // (0 from -150)
                    const float mt = reference(tid), now = fmaxf(mt, M);
                    sh_frame[par * R + tid] = make_float2(factor(M - now), factor(mt - now));
                    M = now;
                }
                // weights
                uint32_t p[3][R / 2];
                float psum_new[R];
                const float lf = pow2i(-ev);
#pragma unroll
                for (int r0 = 0; r0 < R; r0 += 4) {
                    if (r0 >= live)
                        break;
#pragma unroll
                    for (int r = r0; r < r0 + 4; r += 2) {
                        const float y0 = ex2_approx(x[r] - reference(r) + 8.f), y1 = ex2_approx(x[r + 1] - reference(r + 1) + 8.f);
                        psum_new[r] = y0 * lf;
                        psum_new[r + 1] = y1 * lf;
                        uint32_t y = pack_f16x2(y0, y1);
#pragma unroll
                        for (int term = 0; term < 3; ++term)
                            p[term][r / 2] = take_term<16>(y);
                    }
                }
                // Keys that not every row sees: what lies in their slots' place in shared memory
                // may be anything, and NaN times a weight of 0 is NaN.
                if (sh_flags[par * 4] | sh_flags[par * 4 + 1] | sh_flags[par * 4 + 2] | sh_flags[par * 4 + 3]) {
                    const uint32_t item = 2 * g + 1;
                    warp_wait(C::BAR_FULL + item % SLOTS, item / SLOTS & 1, STEP_ERR_SOFTMAX);
                    uint8_t *const tile = smem + C::OFF_RING + item % SLOTS * C::SLOT;
                    auto at = [&](int key, int d) -> uint8_t * {   // d a multiple of 16, or any
                        const int panel = d / C::ROW, col = d % C::ROW, x = C::ROW == 64 ? key >> 1 & 3 : key & 7;
                        return tile + panel * C::PANEL + key * C::ROW + (((col >> 4) ^ x) << 4) + (col & 15);
                    };
                    bool nan = nan_scale;
                    for (int d = 0; d < D; d += 16) {
                        uint4 *w = reinterpret_cast<uint4 *>(at(tid, d));
                        if (!there)
                            *w = make_uint4(0, 0, 0, 0);
                        else
                            nan |= ((w->x ^ without_nan(w->x)) | (w->y ^ without_nan(w->y)) | (w->z ^ without_nan(w->z)) |
                                    (w->w ^ without_nan(w->w))) != 0;
                    }
                    const uint32_t votes = __ballot_sync(0xffffffffu, nan);
                    const uint32_t scale_votes = __ballot_sync(0xffffffffu, nan_scale);
                    if (lane == 0) {
                        sh_nan[warp] = votes;
                        sh_l[warp] = __uint_as_float(scale_votes);
                    }
                    sync();
                    if (sh_nan[0] | sh_nan[1] | sh_nan[2] | sh_nan[3]) {
#pragma unroll 1
                        for (int key = 0; key < TILE; ++key) {
                            if (!(sh_nan[key >> 5] >> (key & 31) & 1))
                                continue;
                            const bool all = __float_as_uint(sh_l[key >> 5]) >> (key & 31) & 1;
                            const int kp = from + j * TILE + key;
                            uint32_t see = 0;
                            for (int r = 0; r < R; ++r)
                                see |= (kp >= sh_lo[r] && kp < sh_hi[r] ? 1u : 0u) << r;
#pragma unroll
                            for (int half = 0; half < C::HALVES; ++half)
                                if (owns_d && (all || (*at(key, half * 128 + tid) & 0x7f) == 0x7f))
                                    nan_rows[half] |= see;
                        }
                        sync();
                        if (nan)
                            for (int d = 0; d < D; d += 16) {
                                uint4 *w = reinterpret_cast<uint4 *>(at(tid, d));
                                *w = make_uint4(without_nan(w->x), without_nan(w->y), without_nan(w->z), without_nan(w->w));
                            }
                    }
                }
                if (j > 0)
                    add_tile(g);   // (and its product no longer reads the weights' place)
#pragma unroll
                for (int r0 = 0; r0 < R; r0 += 4) {
                    if (r0 >= live)
                        break;
#pragma unroll
                    for (int r = r0; r < r0 + 4; ++r) {
                        psum[r] = psum_new[r];
#pragma unroll
                        for (int term = 0; term < 3; ++term) {
                            const int row = term * R + r;
                            smem[C::OFF_P + row * 128 + (((tid >> 4) ^ (row & 7)) << 4) + (tid & 15)] =
                                static_cast<uint8_t>(p[term][r / 2] >> (r & 1) * 8);
                        }
                    }
                }
                fence_proxy_async_shared();
                warp_arrive(C::BAR_P_FULL);
            }
            it += n;
            sync();            // the last frame is there
            add_tile(it);

            // ---- O and LSE of the unit's rows, or of this part of them
#pragma unroll
            for (int r0 = 0; r0 < R; r0 += 4) {
                if (r0 >= live)
                    break;
                float mine = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float v = l[r0 + k];
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1)
                        v += __shfl_xor_sync(0xffffffffu, v, d);
                    mine = lane == k ? v : mine;
                }
                if (lane < 4)
                    sh_l[(r0 + lane) * 4 + warp] = mine;
            }
            sync();
            float2 lse2 = make_float2(-INFINITY, 0.f);   // (threads below R)
            if (tid < R) {
                const float4 l4 = *reinterpret_cast<const float4 *>(sh_l + tid * 4);
                const float sum = tid < live ? (l4.x + l4.y) + (l4.z + l4.w) : 0.f;
                sh_inv[tid] = sum == 0.f ? 0.f : __fdividef(1.f, sum);
                if (sum != 0.f)
                    lse2 = two_floats(M, lg2_approx(sum) - 8.f);
            }
            uint16_t *const o = static_cast<uint16_t *>(a.o);
            auto write_lse = [&](int r, float v) {
                if (r < live)
                    a.lse[sh_place[r].y] = v * 0.69314718055994531f;
            };
            sync();
            if (tid < R) {
                if (alone)
                    write_lse(tid, lse2.x);
                else
                    reinterpret_cast<float2 *>(part + R * D)[tid] = lse2;
            }
#pragma unroll
            for (int r0 = 0; r0 < R; r0 += 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = r0 + k;
                    if (r >= live || !owns_d)
                        break;
                    const float inv = sh_inv[r];
#pragma unroll
                    for (int half = 0; half < C::HALVES; ++half) {
                        const float v = nan_rows[half] >> r & 1 ? __uint_as_float(0x7fc00000u) : acc[half][r] * inv;
                        const int d = half * 128 + tid;
                        if (alone)
                            o[sh_place[r].x + d] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
                        else
                            part[r * D + d] = v;
                    }
                }
            }
            if (!alone) {
                // the CTA whose part is the last to arrive merges them
                volatile int *const last = reinterpret_cast<int *>(smem + C::OFF_MISC + 4);
                __threadfence();
                sync();
                if (tid == 0) {
                    int *const counter = parts.counters + 2 * first_cta;
                    *last = atomicAdd(counter, 1) == last_cta - first_cta;
                    if (*last)
                        *counter = 0;
                }
                sync();
                if (*last) {
                    __threadfence();
                    // N quadruples a thread, so that one pass takes the block (two at R D = 4096)
                    constexpr int N = R * D >= 2048 ? 4 : R * D / 512, TPR = D / 4 / N;
                    for (int r = tid / TPR; r < (live < R ? live : R); r += 128 / TPR) {
                        float4 v[N];
                        auto column = [&](int k) { return (tid % TPR + k * TPR) * 4; };
                        const float merged = merge_row<C, N, 4>(parts, first_cta, last_cta, r, [&](int k) { return r * D + column(k); }, v);
#pragma unroll
                        for (int k = 0; k < N; ++k)
                            *reinterpret_cast<uint2 *>(o + sh_place[r].x + column(k)) =
                                make_uint2(pack_bf16x2(v[k].x, v[k].y), pack_bf16x2(v[k].z, v[k].w));
                        if (tid % TPR == 0)
                            write_lse(r, merged);
                    }
                }
            }
            ++unit;
            sync();   // the rows' places are free again
        } while (next_unit());
    }

    tc_fence_before();
    __syncthreads();
    if (warp == C::WARP_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

template <class C>
fa2_status launch_step(const AttnArgs &a)
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
        if (cudaFuncSetAttribute(step_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess) {
            (void)cudaGetLastError();
            return FA2_ERR_CUDA;
        }
        configured.fetch_or(bit);
    }
    step_kernel<C><<<grid, C::T, C::SMEM_BYTES, a.stream>>>(k_map, v_map, a, parts);
    return cudaGetLastError() == cudaSuccess ? FA2_OK : FA2_ERR_CUDA;
}
#endif

}  // namespace cache
}  // namespace fa2
