// fa2_paged_chunk.cuh -- attention of many query rows over the paged 16-bit cache
// (fa2_paged_attn in include/fa2_paged.h): blocks of up to 256 rows on the 5th-generation
// tensor cores.
//
// Mathematics.  As in fa2_paged_step.cuh, rows are the tokens of a sequence times the query
// heads that share a key/value head.  With c = scale log2 e and M a score of the row, the largest
// so far or up to 8 / c below it,
//     p_j = 2^(S_j c - M c + LIFT),   P = p in the cache's type,   O += P V,   l += p,   l' += P
// O and l are brought to a larger M only when a tile's scores pass it by more than 8 in the
// exponent.  O is divided by l', the sum of the weights that the product saw, so that a weight's
// rounding cancels where one key dominates (fp16, and bf16 at D = 256, where P is two terms: by l);
// LSE and a part's share in a row come from l.  The
// reference is the float F = M c - LIFT, whatever it was rounded by, and 2^(S_j c - F) one
// multiply-add.  Where |F| passes 2^25 its rounding could leave the range of a weight: there the
// scores are replaced by S_j - M first, where they are, and the reference is M c - LIFT itself.
//
// What bounds it.  4 D operations a (row, key) pair: the tensor pipe, and beside it the
// exponentials.  Work has warps of its own,
//     4 warps a row tile  softmax: a thread a row, its 128 scores of a tile in registers
//     1 warp              issues the products: one 128-row tile's run under the other's softmax
//     2 warps             pages into a ring of shared-memory slots by TMA, keys and values
//     1 warp              the next unit's queries, under the end of the present one, and values
//                         that not every row sees (below)
// on one CTA an SM.  The weights go to tensor memory, where the second product reads them, in
// two halves, so that it begins under the second half's exponentials.  Work is cut and merged as
// in fa2_paged_line.cuh.  A unit of 128 rows or fewer (D < 256) is a twin: its two row tiles are
// the same rows with every other tile of keys each, put together at its end.
//
// Measured (in a graph, in bursts of some milliseconds at the full clock, 2070 MHz).  2048 tokens of a
// prompt over 16384 keys, theirs included, 32 and 8 heads of 128, causal (515 GFLOP): 333 to 343 us,
// 1.50 to 1.55 PFLOP/s, 0.79 to 0.81 of the measured matrix rate; for seconds, at the 1935 MHz that the
// power cap leaves, 359 us, and 361 as calls from Python: the same cycles, 694 to 699 thousand.
// The loop over tiles shifts by 3 % with any change of its code.  The same with heads of 64
// (as many exponentials for half the products) 282 us; 16 and 4 heads of 256 478 us, fp16 384;
// pages of 16 keys 347.  No single unit is the bound: in timing copies, without the exponentials 334 us for
// 360, with half the bytes of K and V 341 for 354.
// Five drafted tokens of 24 contexts of up to 4096 keys, 16 and 2 heads of 64 (26 MB), 20.5 us:
// a launch, the lengths, one or two units of half-filled tiles a CTA, and the merge.
//
// A weight of 0 times an infinity or NaN is NaN.  In a tile in which some row does not see some
// key, one warp makes zeros of the values that no row sees, and of the infinities and NaN among
// those that only some rows see; the rows that see one of these make their O at its column NaN at
// the end.
#pragma once

#include <atomic>
#include <type_traits>

#include "fa2_paged.cuh"
#include "fa2_paged_line.cuh"
#include "fa2_paged_merge.cuh"

namespace fa2 {
namespace paged {

template <int D_, bool F16_>
struct ChunkCfg {
    static constexpr int D = D_;
    static constexpr bool F16 = F16_;
    static constexpr int NQ = D == 256 ? 1 : 2;      // 128-row tiles of a unit
    static constexpr int R = 128 * NQ;               // its query rows
    static constexpr int TILE = 128;                 // keys
    // see fa2_paged_line.cuh
    // (A tile of one row tile takes somewhat more than half the time of a tile of two.  COST 24 to 44
    // and LEAST 16 to 32 differ by 3 % at most.)
    static constexpr int GRAIN_SHIFT = 7, COST = 32, LEAST = 24;
    __host__ __device__ static constexpr int weight_shift(int rows, int) { return NQ == 2 && rows <= 128 ? 2 : 3; }
    static constexpr int CTAS = 1;                   // an SM
    static constexpr int WARP_MMA = 4 * NQ, WARP_LOAD = WARP_MMA + 1, WARP_SCAN = WARP_MMA + 2, WARP_V = WARP_MMA + 3;
    static constexpr int T = 32 * (WARP_MMA + 4);
    // With three warpgroups the launch leaves 168 registers a thread; the softmax rises.
    static constexpr bool REG_SPLIT = NQ == 2;
    static constexpr int REG_SOFTMAX = 200, REG_CTRL = 104;
    static_assert(2 * REG_SOFTMAX + REG_CTRL <= 3 * 168, "the split draws on the launch's registers");
    // Whether l' is summed: a bf16 weight is off by 2^-8, as O itself, an fp16 one by 2^-11, a
    // quarter of which on average shows in O (and adding fp16 to fp32 takes twice the issue slots
    // of bf16: six ragged prompts' chunks at D = 64 66 us with it, 59 without).
    static constexpr bool SEEN = !F16 && D < 256;
    // bf16 weights at D = 256 are two terms, as in the dense pass: with one, where two or three keys stand
    // out alike, 50 of 8.2 M values were off by more than 1e-2 (2 x 8 heads, 2000 rows of 3000 keys, every 64th
    // of them eight times as large), some of 2 to 3, which no rounding of O explains; with two 41, all of 4 or
    // more, whose own rounding it is.  It costs one more product: the prompt chunk at D = 256 478 us, 388 with
    // one (fp16, which has one, 384).
    static constexpr bool TWO = !F16 && D == 256;
    static constexpr float LIFT = Weight<F16>::LIFT;

    // A tile's keys, and its values, are PARTS slots of the ring, of up to 128 columns each, in
    // panels of 64 columns (128 bytes a row, the swizzle's span).
    static constexpr int PARTS = D == 256 ? 2 : 1, DP = D / PARTS, PANELS = DP / 64;
    static constexpr int PANEL = TILE * 128, SLOT = PANELS * PANEL;
    static constexpr int SLOTS = D == 64 ? 8 : 4, VT = SLOTS / (2 * PARTS);   // VT: tiles whose values it holds
    static constexpr int Q_PANEL = 128 * 128, Q_TILE = D / 64 * Q_PANEL;
    static constexpr int NS = D == 256 ? 2 : 1;      // S buffers a row tile
    // The weights lie over the scores where tensor memory has no room beside them; else the next
    // scores are computed while they are made.
    static constexpr bool P_APART = D == 64;
    static constexpr int TM_S = 0, TM_O = NQ * NS * TILE, TM_P = P_APART ? TM_O + NQ * D : TM_S, P_STEP = P_APART ? TILE / 2 : TILE;
    static constexpr int TMEM_COLS = 512;
    static_assert(TM_O + NQ * D + (P_APART ? NQ * P_STEP : 0) <= TMEM_COLS, "tensor memory holds it");
    static constexpr int P_LOW = TILE / 2;           // the second term's columns behind the first's
    static_assert(!TWO || !P_APART, "both terms lie over the scores");

    static constexpr int OFF_Q = 0, OFF_RING = NQ * Q_TILE, MARK_WORDS = D / 32;
    static constexpr int OFF_MARK = OFF_RING + SLOTS * SLOT;         // values of O that are NaN, by row
    static constexpr int OFF_SUM = OFF_MARK + R * MARK_WORDS * 4;    // M, l, l' of a row, by row tile
    // Rings of eight tiles (the loading warps are at most six ahead of a tile's softmax): page bits,
    // keys with an infinity or NaN in their values.
    static constexpr int OFF_OUT = OFF_SUM + R * 16;                 // of each softmax warp: 32 rows by 32 columns of O
    static constexpr int RING = 8, OFF_SEES = OFF_OUT + R * 64, OFF_ODD = OFF_SEES + R * 8,   // (OFF_SEES: keys a row sees)
                         OFF_INFO = OFF_ODD + RING * 16;
    static constexpr int OFF_BAR = OFF_INFO + 2 * RING * 4;   // (OFF_INFO: of keys, of values)
    static_assert(VT + 1 < RING, "the rings hold the tiles under way");
    // Barriers of scanned tiles, in turn.  A softmax warp waits for the scan of some tiles only, and a
    // parity tells a phase from the one before only: when a tile's scores are there, the product of two
    // tiles before has been issued, behind its scan, so two will do.
    static constexpr int NC = VT < 2 ? 2 : VT;
    // (the first ones: one for each row tile, or S buffer)
    static constexpr int BAR_Q_FULL = 0, BAR_Q_EMPTY = 2, BAR_S_FULL = 4, BAR_S_EMPTY = 6, BAR_PA = 8, BAR_P = 10, BAR_O_DONE = 12,
                         BAR_DRAIN = 14, BAR_CLEAN = 15, BAR_FULL = BAR_CLEAN + NC, BAR_EMPTY = BAR_FULL + SLOTS,
                         NUM_BAR = BAR_EMPTY + SLOTS;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BAR * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;          // 1024: operand alignment
    static_assert(SMEM_BYTES + 1024 + 1024 <= 228 * 1024, "an SM holds it");
};

// References past which a row's scores are taken by differences: a float's last place is 4 there.
constexpr float LARGE = 1 << 25;
// How far a tile's scores may pass the reference, in the exponent, before O and l are brought to a
// larger one.
constexpr float SLACK = 8.f;
constexpr uint32_t WHOLE = 1u << 31;   // of a tile: every row sees every key

// Error codes of waits that ran out (bits 8-11 the waiting role).
constexpr int CHUNK_ERR_SOFTMAX = 8 << 8, CHUNK_ERR_SCAN = 9 << 8, CHUNK_ERR_MMA = 10 << 8, CHUNK_ERR_LOAD = 11 << 8,
              CHUNK_ERR_DRAIN = 7 << 8, CHUNK_ERR_Q = 6 << 8;

#ifdef __CUDACC__

// 16 bytes from global to shared memory, under way until waited for; zeros if not `there`.
__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits for all but the last N groups of this thread's copies.
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A row's reference as a float, and what of M c - LIFT it leaves out.
template <class C>
__device__ __forceinline__ float reference(float M, float c)
{
    return __fsub_rn(__fmul_rn(M, c), C::LIFT);
}
template <class C>
__device__ __forceinline__ float left_out(float M, float c)
{
    const float x = __fmul_rn(M, c), y = __fsub_rn(x, C::LIFT);
    const float lift = __fsub_rn(x, y);   // what of LIFT went into y; what of x: y + lift
    return fmaf(M, c, -x) + (__fsub_rn(x, __fadd_rn(y, lift)) + __fsub_rn(lift, C::LIFT));
}
// 2^(from - to): what is relative to one reference, brought to another.
template <class C>
__device__ __forceinline__ float to_frame(float from, float to, float c)
{
    auto rest = [&](float M) { return fabsf(reference<C>(M, c)) > LARGE ? left_out<C>(M, c) : 0.f; };
    return from == -INFINITY ? 0.f : ptx::ex2_approx((reference<C>(from, c) - reference<C>(to, c)) + (rest(from) - rest(to)));
}

// Scores of a tile that the row does not see (columns outside [above, below), or without a page)
// become -infinity, where they are.  (This and the others below run for few tiles, and stand apart
// from the loop over tiles, whose registers and instructions they are not to share.)  Of most tiles
// that any row does not see whole, a warp's 32 rows do see most columns alike: a look at 32 columns'
// bits first (all columns, compared one by one: 1.6 to 1.9 us a tile).
template <class C>
__device__ __noinline__ void mask_scores(uint32_t s_addr, int above, int below, uint32_t pages, int page_shift)
{
#pragma unroll 1
    for (int k = 0; k < C::TILE; k += 32) {
        auto first = [](int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; };   // n bits
        const bool page0 = pages >> (k >> page_shift) & 1, page1 = pages >> (k + 16 >> page_shift) & 1;
        const uint32_t sees = first(below - k) & ~first(above - k) & ((page0 ? 0xffffu : 0u) | (page1 ? 0xffff0000u : 0u));
        if (__all_sync(0xffffffffu, sees == ~0u))
            continue;
        uint32_t x[32];
        ptx::tmem_ld32(s_addr + k, x);
        ptx::tmem_ld_wait(x);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            x[e] = sees >> e & 1 ? x[e] : 0xff800000u;
        ptx::tmem_st32(s_addr + k, x);
    }
    ptx::tmem_st_wait();
}

// N columns of tensor memory (O) times `by`.
template <int N>
__device__ __noinline__ void scale_columns(uint32_t addr, float by)
{
#pragma unroll 1
    for (int k = 0; k < N; k += 32) {
        uint32_t x[32];
        ptx::tmem_ld32(addr + k, x);
        ptx::tmem_ld_wait(x);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            x[e] = __float_as_uint(__uint_as_float(x[e]) * by);
        ptx::tmem_st32(addr + k, x);
    }
    ptx::tmem_st_wait();
}

// N columns of tensor memory (scores) less `sub`.
template <int N>
__device__ __noinline__ void shift_columns(uint32_t addr, float sub)
{
#pragma unroll 1
    for (int k = 0; k < N; k += 32) {
        uint32_t x[32];
        ptx::tmem_ld32(addr + k, x);
        ptx::tmem_ld_wait(x);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            x[e] = __float_as_uint(__uint_as_float(x[e]) - sub);
        ptx::tmem_st32(addr + k, x);
    }
    ptx::tmem_st_wait();
}

// Marks the values of O that an infinity or NaN among the values of the keys [k0, k1) of a tile,
// those with a bit in odd[4], makes NaN.
template <class C>
__device__ __noinline__ void mark_odd(const AttnArgs &a, const volatile uint32_t *odd, int b, int h, int pos0, int k0, int k1,
                                      uint32_t *mark)
{
#pragma unroll 1
    for (int k = k0; k < k1; ++k) {
        if (!(odd[k >> 5] >> (k & 31) & 1))
            continue;
        const int pos = pos0 + k, id = cache::page_of(a.c, b, pos >> a.c.page_shift);
        if (id < 0)   // (only behind a wait that ran out, where the bits may be anything)
            continue;
        const uint32_t *v = reinterpret_cast<const uint32_t *>(a.c.v.codes + id * a.c.v.s_page + h * a.c.v.s_head +
                                                               (pos & ((1 << a.c.page_shift) - 1)) * a.c.v.s_slot);
#pragma unroll 1
        for (int w = 0; w < C::D / 2; ++w) {
            const uint32_t x = v[w];
            if (odd_lo<C::F16>(x) || odd_hi<C::F16>(x))
                mark[(w >> 4) * C::R] |= ((odd_lo<C::F16>(x) ? 1u : 0u) | (odd_hi<C::F16>(x) ? 2u : 0u)) << (w & 15) * 2;
        }
    }
}

template <class C>
__global__ void __launch_bounds__(C::T, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                 const __grid_constant__ AttnArgs a, const cache::Parts parts)
{
    using namespace ptx;
    using cache::Range;
    constexpr int D = C::D, R = C::R, TILE = C::TILE, SLOTS = C::SLOTS, PARTS = C::PARTS, NS = C::NS;
    constexpr bool F16 = C::F16;
    extern __shared__ uint8_t smem_raw[];
    __shared__ cache::LineShared sh_line;
    // Each warp's place on the line: it changes with the unit only, and would cost the roles
    // registers in their loops over tiles.
    __shared__ struct {
        Range range;
        int first, end, any;
        Line<C> line[C::T / 32];
    } sh;

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
        for (int i = 0; i < C::NUM_BAR; ++i) {
            const bool rows = i / 2 == C::BAR_S_EMPTY / 2 || i / 2 == C::BAR_PA / 2 || i / 2 == C::BAR_P / 2;
            mbar_init(bar(i), rows ? 4 : 1);
        }
        fence_mbar_init();
        tma_prefetch_desc(&k_map);
        tma_prefetch_desc(&v_map);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Line<C> &line = sh.line[warp];

    const uint64_t limit = a.wait_limit_ns;
    auto warp_wait = [&](int i, uint32_t parity, int code) -> bool {
        return cache::wait_phase(bar(i), parity, a.err, code | i, limit);
    };
    auto warp_arrive = [&](int i) {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(i));
    };
    // the unit's keys [from, stop) in this CTA's range, and the tiles they make
    auto part_of = [&](int &from, int &stop) { return line.piece(a, cut, sh.first, sh.end, from, stop); };
    // of a unit's tiles from `from`, those whose keys every row sees, as far as positions go: [w0, w1)
    auto whole_of = [&](int from, int &w0, int &w1) {
        int lo, hi;
        line.seen_by_all(a, lo, hi);
        w0 = lo > from ? (lo - from + TILE - 1) / TILE : 0;
        w1 = hi > from ? (hi - from) / TILE : 0;
    };
    auto next_unit = [&]() -> bool {     // by a whole warp
        __syncwarp();
        bool more = false;
        if (lane == 0)
            more = sh.line[warp].next(a, sh.end);
        __syncwarp();                    // (a shuffle orders no memory)
        return __shfl_sync(0xffffffffu, more, 0);
    };
    volatile uint32_t *const sh_info = reinterpret_cast<uint32_t *>(smem + C::OFF_INFO);   // bit i: page i is there
    volatile uint32_t *const sh_odd = reinterpret_cast<uint32_t *>(smem + C::OFF_ODD);     // [RING][4]
    uint32_t it = 0;               // tiles before the present unit's first
    // A unit of no more than 128 rows: the row tiles are the same rows, one with the even
    // tiles of keys, one with the odd ones, and are put together at the end.
    auto is_twin = [&] { return C::NQ > 1 && line.s.n * a.G - line.rb * R <= 128; };

    if (warp >= C::WARP_MMA) {
        if constexpr (C::REG_SPLIT)
            setmaxnreg_dec<C::REG_CTRL>();
        // These four warps lay out the line, for the others too.
        bool any;
        {
            auto sync = [] { asm volatile("bar.sync 4, 128;" ::: "memory"); };
            Range range;
            int first, end;
            Line<C> mine;
            any = paged::find_range<C, 128>(a, cut, sh_line, range, first, end, mine, tid - 32 * C::WARP_MMA, sync);
            if (lane == 0) {
                for (int w = warp; w >= 0; w -= 4)
                    sh.line[w] = mine;
                if (warp == C::WARP_MMA) {
                    sh.range = range;
                    sh.first = first;
                    sh.end = end;
                    sh.any = any;
                }
            }
            sync();
            asm volatile("bar.arrive 5, %0;" ::"n"(C::T) : "memory");
        }
        if (!any) {
        } else if (warp == C::WARP_MMA) {
            // ======================================== one thread issues the products
            // (the whole loop in one lane: groups of products issued from a branch that the
            // warp's other lanes skip take twice the time of the products)
            if (elect_one()) {
                const uint64_t desc_q = sdesc_sw128(base + C::OFF_Q, 16, 1024), desc_k = sdesc_sw128(base + C::OFF_RING, 16, 1024),
                               desc_v = sdesc_sw128(base + C::OFF_RING, C::PANEL, 1024);
                bool ok = true;
                auto wait = [&](int i, uint32_t parity) {
                    if (ok)
                        ok = lone_wait(bar(i), parity, a.err, CHUNK_ERR_MMA | i, limit);
                };
                // of each row tile: tiles of keys, and loads of Q, before the present unit
                uint32_t done[C::NQ] = {}, loads[C::NQ] = {};
                // S = Q K^T of row tile q (rows q_at of Q) and tile g of keys, its tile d, the first and the last
                // to read this tile of keys, the last to read Q
                auto issue_s = [&](int q, int q_at, uint32_t g, uint32_t d, bool first_k, bool last_k, bool last_q) {
                    const uint32_t b = NS == 2 ? d & 1 : 0;
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        const uint32_t item = 2 * PARTS * g + part, slot = item % SLOTS;
                        if (first_k) {
                            wait(C::BAR_FULL + slot, item / SLOTS & 1);
                            if (!ok)
                                return;
                            tc_fence_after();
                        }
                        const uint64_t dk = desc_k + (slot * C::SLOT >> 4),
                                       dq = desc_q + (q_at * C::Q_TILE + part * C::PANELS * C::Q_PANEL >> 4);
#pragma unroll
                        for (int kk = 0; kk < C::PANELS * 4; ++kk)
                            mma_ss(tmem + C::TM_S + (q * NS + b) * TILE, dq + ((kk >> 2) * C::Q_PANEL + (kk & 3) * 32 >> 4),
                                   dk + ((kk >> 2) * C::PANEL + (kk & 3) * 32 >> 4), idesc(F16, 128, TILE, false, false),
                                   part > 0 || kk > 0);
                        if (part == PARTS - 1)
                            mma_commit(bar(C::BAR_S_FULL + q * NS + b));
                        if (last_k)
                            mma_commit(bar(C::BAR_EMPTY + slot));
                    }
                    if (last_q)
                        mma_commit(bar(C::BAR_Q_EMPTY + q_at));
                };
                auto issue_pv = [&](int q, uint32_t g, uint32_t d, bool start, bool last_v) {   // O += P V
                    const uint32_t b = NS == 2 ? d & 1 : 0, p = tmem + C::TM_P + (q * NS + b) * C::P_STEP;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        wait((half ? C::BAR_P : C::BAR_PA) + q * NS + b, d / NS & 1);
                        if (!ok)
                            return;
                        tc_fence_after();
#pragma unroll
                        for (int part = 0; part < PARTS; ++part) {
                            const uint32_t item = 2 * PARTS * g + PARTS + part, slot = item % SLOTS;
                            const uint64_t dv = desc_v + (slot * C::SLOT >> 4);
#pragma unroll
                            for (int kk = half * 4; kk < half * 4 + 4; ++kk)
#pragma unroll
                                for (int term = 0; term < (C::TWO ? 2 : 1); ++term)
                                    mma_ts(tmem + C::TM_O + q * D + part * C::DP, p + term * C::P_LOW + kk * 8,
                                           dv + (kk * 16 * 128 >> 4), idesc(F16, 128, C::DP, false, true),
                                           !start || kk > 0 || term > 0);
                            if (half && last_v)
                                mma_commit(bar(C::BAR_EMPTY + slot));
                        }
                    }
                    mma_commit(bar(C::BAR_O_DONE + q));
                };
                // (For the scan of every tile, whether it had anything to do or not: else the scanning warp,
                // late, could find a slot filled twice, and take the one tile for the other.)
                auto wait_v = [&](uint32_t g) {
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        const uint32_t item = 2 * PARTS * g + PARTS + part;
                        wait(C::BAR_FULL + item % SLOTS, item / SLOTS & 1);
                    }
                    wait(C::BAR_CLEAN + g % C::NC, g / C::NC & 1);
                };
                // One unit.  The first tiles' scores; then for each tile and row tile the product with the
                // values, and the scores of the tile NS after (twins: two after).  (A unit's first product
                // overwrites O: the warps whose weights it waits for have read out the one before.)
                auto unit = [&](auto twins, int n) {
                    constexpr bool twin = decltype(twins)::value;
                    constexpr int every = twin ? 2 : 1, ahead = twin ? 2 : NS;
#pragma unroll
                    for (int b = 0; b < NS; ++b)
#pragma unroll
                        for (int q = 0; q < C::NQ; ++q) {
                            if (b == 0 && (q == 0 || !twin))
                                wait(C::BAR_Q_FULL + q, loads[q] & 1);
                            const int j = twin ? q : b;
                            if (ok && j < n) {
                                tc_fence_after();
                                issue_s(q, twin ? 0 : q, it + j, done[q] + b, twin || q == 0, twin || q == C::NQ - 1, j == n - 1);
                            }
                        }
                    for (int j = 0; j < n && ok; ++j) {
                        wait_v(it + j);
#pragma unroll
                        for (int q = 0; q < C::NQ; ++q)
                            if (ok && (!twin || q == (j & 1))) {
                                const uint32_t d = done[q] + (twin ? j >> 1 : j);
                                auto next_s = [&] {
                                    if (ok && j + ahead < n)
                                        issue_s(q, twin ? 0 : q, it + j + ahead, d + (twin ? 1 : NS), twin || q == 0,
                                                twin || q == C::NQ - 1, j + ahead == n - 1);
                                };
                                if (C::P_APART) {    // (its scores are in registers before the weights are made)
                                    if (j + ahead < n)
                                        wait(C::BAR_S_EMPTY + q, d & 1);
                                    tc_fence_after();
                                    next_s();
                                }
                                if (ok)
                                    issue_pv(q, it + j, d, j < every, twin || q == C::NQ - 1);
                                if (!C::P_APART)
                                    next_s();
                            }
                    }
#pragma unroll
                    for (int q = 0; q < C::NQ; ++q) {
                        done[q] += twin ? (n + 1 - q) >> 1 : n;
                        loads[q] += q == 0 || !twin;
                    }
                };
                bool more;
                do {
                    int from, stop;
                    const int n = part_of(from, stop);
                    if (C::NQ > 1 && is_twin())
                        unit(std::bool_constant<C::NQ != 1>{}, n);
                    else
                        unit(std::false_type{}, n);
                    it += n;
                    more = ok && sh.line[C::WARP_MMA].next(a, sh.end);
                } while (more);
                // nothing issued is still running when tensor memory is given back
                mma_commit(bar(C::BAR_DRAIN));
                lone_wait(bar(C::BAR_DRAIN), 0, a.err, CHUNK_ERR_DRAIN | C::BAR_DRAIN, a.drain_limit_ns);
            }
            __syncwarp();
        } else if (warp == C::WARP_LOAD || warp == C::WARP_V) {
            // ======================================== pages -> ring: keys' by one warp, values' by another
            // (one warp for both: 570 us instead of 388 for the prompt chunk at D = 256, there with one term a
            // weight, 391 instead of 346 over pages of 16 at D = 128)
            const bool values = warp == C::WARP_V;
            const CUtensorMap *const map = values ? &v_map : &k_map;
            volatile uint32_t *const info = sh_info + (values ? C::RING : 0);
            const int box_shift = a.c.page_shift;              // rows of a box: a page
            const int boxes_shift = 7 - box_shift;             // boxes of a tile
            const uint32_t box_bytes = static_cast<uint32_t>(C::PANELS) * 128 << box_shift;   // of a slot
            const int in_tile = lane & ((1 << boxes_shift) - 1);
            const uint32_t offset = static_cast<uint32_t>(in_tile) * 128 << box_shift;        // in each panel
            const int batch_tiles = 32 >> boxes_shift;
            uint32_t issued = 0;                               // items
            bool ok = true;
#pragma unroll 1
            for (int i = a.naps; i > 0; --i)
                __nanosleep(500);
            do {
                int from, stop;
                const int n = part_of(from, stop), h = line.h;
                int whole0, whole1;
                whole_of(from, whole0, whole1);
                // A lane has one of 32 boxes, those of the next 4 to 32 tiles: the table's
                // entries come a batch ahead.
                auto pages = [&](int tile) {                   // -1: none, or not seen
                    if (tile >= n)
                        return -1;
                    const int pos = from + tile * TILE + (lane << box_shift);
                    return pos < stop && pos + (1 << box_shift) > line.span.lo
                               ? cache::page_of(a.c, line.b, pos >> a.c.page_shift)
                               : -1;
                };
                int id = pages(0), id_next = pages(batch_tiles);
                for (int j = 0; j < n && ok; ++j) {
                    const int jj = j & (batch_tiles - 1);
                    if (jj == 0 && j > 0) {
                        id = id_next;
                        id_next = pages(j + batch_tiles);
                    }
                    const bool mine = lane >> boxes_shift == jj;
                    const uint32_t g = it + j, all = (1u << (1 << boxes_shift)) - 1;
                    const uint32_t there = __ballot_sync(0xffffffffu, id >= 0) >> (jj << boxes_shift) & all;
                    const uint32_t bytes = __popc(there) * box_bytes;
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) {
                        const uint32_t item = 2 * PARTS * g + (values ? PARTS : 0) + k, slot = item % SLOTS;
                        const uint32_t full = bar(C::BAR_FULL + slot);
                        if (item >= SLOTS && !(ok = warp_wait(C::BAR_EMPTY + slot, (item / SLOTS - 1) & 1, CHUNK_ERR_LOAD)))
                            break;
                        // values without a page are zeros (their weights are, and what lies there may be NaN)
                        if (values && there != all) {
                            for (int row = lane; row < TILE; row += 32)
                                if (!(there >> (row >> box_shift) & 1))
                                    for (int x = 0; x < C::PANELS * 8; ++x)
                                        st_shared_v4(base + C::OFF_RING + slot * C::SLOT + x / 8 * C::PANEL + row * 128 +
                                                         x % 8 * 16, 0, 0, 0, 0);
                            fence_proxy_async_shared();
                            __syncwarp();
                        }
                        if (lane == 0) {
                            if (k == 0)
                                info[g % C::RING] = there | (there == all && j >= whole0 && j < whole1 ? WHOLE : 0u);
                            mbar_arrive_expect_tx(full, bytes);
                        }
                        __syncwarp();
                        if (mine && id >= 0)
#pragma unroll
                            for (int p = 0; p < C::PANELS; ++p)
                                tma_load_4d(base + C::OFF_RING + slot * C::SLOT + p * C::PANEL + offset, map,
                                            (k * C::PANELS + p) * 64, 0, h, id, full);
                        __syncwarp();
                        issued = item + 1;
                    }
                }
                it += n;
            } while (ok && next_unit());
            // the copies in flight have landed before the CTA goes
            for (uint32_t item = issued > SLOTS ? issued - SLOTS : 0; item < issued; ++item) {
                if ((item / PARTS & 1) != (values ? 1u : 0u))   // (the other warp's)
                    continue;
                const int i = C::BAR_FULL + item % SLOTS;
                cache::wait_phase(bar(i), item / SLOTS & 1, a.err, CHUNK_ERR_DRAIN | i, a.drain_limit_ns);
            }
        } else {
            // ======================================== queries; values that not every row sees
            bool ok = true;
#pragma unroll 1
            for (int i = 2 * a.naps; i > 0; --i)   // (later than the loads)
                __nanosleep(500);
            uint32_t loads[C::NQ] = {};
            do {
                const bool twin = is_twin();
#pragma unroll
                for (int q = 0; q < C::NQ; ++q) {
                    if (q > 0 && twin)
                        break;
                    if (ok && loads[q] > 0)
                        ok = warp_wait(C::BAR_Q_EMPTY + q, (loads[q] - 1) & 1, CHUNK_ERR_Q);
                    if (!ok)
                        break;
                    // a row by D / 8 lanes, so that they read whole lines; no row: zeros
                    constexpr int LPR = D / 8, RPI = 32 / LPR;
                    const uint16_t *const from = static_cast<const uint16_t *>(a.q) + line.b * a.q_sb;
                    const int chunk = lane % LPR;
                    const uint32_t to = base + C::OFF_Q + q * C::Q_TILE + chunk / 8 * C::Q_PANEL;
#pragma unroll 1
                    for (int i = 0; i < 128; i += 32) {
                        const int rr = line.rb * R + q * 128 + i + lane;
                        const long long mine = rr < line.s.n * a.G ? (line.h * a.G + rr % a.G) * a.q_sh + rr / a.G * a.q_sl : -1;
#pragma unroll 8
                        for (int k = 0; k < 32; k += RPI) {
                            const long long at = __shfl_sync(0xffffffffu, mine, k + lane / LPR);
                            const int row = i + k + lane / LPR;
                            copy16(to + row * 128 + ((chunk % 8 ^ (row & 7)) << 4), from + (at < 0 ? 0 : at) + chunk * 8, at >= 0);
                        }
                    }
                    copies_commit();
                    ++loads[q];
                }
                // (the first row tile's may be there before the second's)
                if (ok && C::NQ > 1 && !twin) {
                    copies_wait<1>();
                    fence_proxy_async_shared();
                    warp_arrive(C::BAR_Q_FULL);
                }
                copies_wait<0>();
                fence_proxy_async_shared();
                if (ok)
                    warp_arrive(C::BAR_Q_FULL + (C::NQ > 1 && !twin ? 1 : 0));
                int from, stop;
                const int n = part_of(from, stop);
                int whole0, whole1, all_lo, all_hi;
                whole_of(from, whole0, whole1);
                line.seen_by_all(a, all_lo, all_hi);
                for (int j = 0; j < n && ok; ++j) {
                    const uint32_t g = it + j;
                    uint32_t slot[PARTS];
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        const uint32_t item = 2 * PARTS * g + PARTS + part;
                        slot[part] = item % SLOTS;
                        if (ok)
                            ok = warp_wait(C::BAR_FULL + slot[part], item / SLOTS & 1, CHUNK_ERR_SCAN);
                    }
                    if (!ok)
                        break;
                    if (j < whole0 || j >= whole1) {
                        const uint32_t info = sh_info[C::RING + g % C::RING];
#pragma unroll 1
                        for (int i = 0; i < 4; ++i) {
                            const int key = i * 32 + lane, pos = from + j * TILE + key;
                            const bool seen = (info >> (key >> a.c.page_shift) & 1) && pos >= line.span.lo && pos < stop;
                            // (what every row sees is theirs as it is)
                            const bool some = seen && !(pos >= all_lo && pos < all_hi);
                            auto at = [&](int i) {   // eight values
                                const int part = i / (C::DP / 8), d = i % (C::DP / 8) * 8;
                                return reinterpret_cast<uint4 *>(smem + C::OFF_RING + slot[part] * C::SLOT + d / 64 * C::PANEL +
                                                                 key * 128 + ((d % 64 / 8 ^ (key & 7)) << 4));
                            };
                            if (!seen)
#pragma unroll
                                for (int i = 0; i < D / 8; ++i)
                                    *at(i) = make_uint4(0, 0, 0, 0);
                            const bool odd = some && any_odd<F16, D / 8>(at);
                            if (odd)
#pragma unroll
                                for (int i = 0; i < D / 8; ++i)
                                    *at(i) = finite4<F16>(*at(i));
                            const uint32_t votes = __ballot_sync(0xffffffffu, odd);
                            if (lane == 0)
                                sh_odd[g % C::RING * 4 + i] = votes;
                        }
                        fence_proxy_async_shared();
                    }
                    warp_arrive(C::BAR_CLEAN + g % C::NC);
                }
                it += n;
            } while (ok && next_unit());
        }
    } else {
        // ============================================ softmax: a thread a row
        if constexpr (C::REG_SPLIT)
            setmaxnreg_inc<C::REG_SOFTMAX>();
        const int rt = warp >> 2, row = tid & 127;             // row tile, row in it
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float c = a.scale * 1.4426950408889634f;
        const uint32_t o_addr = tmem + lanes + C::TM_O + rt * D;
        // the row tile's warps; all of them
        auto tile_sync = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + rt) : "memory"); };
        auto all_sync = [] { asm volatile("bar.sync 3, %0;" ::"n"(128 * C::NQ) : "memory"); };
        // A wait that ran out is recorded and not waited for again: the role runs on to its end
        // without waiting (its outputs are undefined), so that barriers between warps still match.
        bool ok = false;
        auto wait = [&](int i, uint32_t parity) {
            if (ok)
                ok = warp_wait(i, parity, CHUNK_ERR_SOFTMAX);
        };
        // The loop over tiles is some 15 KB of instructions, whose first way to the SM takes 4 us.  So while
        // the line is laid out and the first tiles are on their way the warps go through it once for
        // nothing: without waiting (ok) or arriving, reading what lies in tensor memory and writing
        // where nothing is yet.
        bool dry = true;
        int arriving = 32;
        auto arrive = [&](int i) {
            __syncwarp();
            if (lane == arriving)
                mbar_arrive(bar(i));
        };
        uint32_t n_done = 0;                                   // of this row tile: tiles of keys
        while (true) {
            int from = 0, stop = 0, n = 1 + rt;
            bool twin = rt != 0;
            if (!dry) {
                n = part_of(from, stop);
                twin = is_twin();
            }
            const int every = twin ? 2 : 1, j0 = twin ? rt : 0;   // this row tile's tiles of keys
            const int row_at = twin ? row : rt * 128 + row;       // its row in the unit
            // What only a unit's beginning and end, and tiles that a row does not see whole, ask for is
            // kept out of the registers of the loop over tiles: the row's token and head are taken
            // again from its number, the keys that it sees lie in shared memory.
            struct Row {
                int tok, hq;
                bool live;
            };
            auto this_row = [&] {
                int rr = line.rb * R + row_at;
                asm volatile("" : "+r"(rr));
                return Row{rr / a.G, line.h * a.G + rr % a.G, rr < line.s.n * a.G};
            };
            int2 *const sees = reinterpret_cast<int2 *>(smem + C::OFF_SEES) + rt * 128 + row;
            if (!dry) {
                const Row r = this_row();
                const int pos = line.s.kv - line.s.n + r.tok;
                const long long x = static_cast<long long>(pos) - a.window;
                *sees = make_int2(a.window >= 0 && x > 0 ? static_cast<int>(x) : 0, !r.live ? 0 : a.causal ? pos + 1 : line.s.kv);
            }
            float M = -INFINITY, l = 0.f, l_seen = 0.f;          // l_seen: of the weights as the product sees them
            float add = 0.f;                                     // less the reference
            bool large = false;                                  // |reference| > LARGE in a row of the warp
            // values of O that a visible infinity or NaN makes NaN: word w at [w * R]
            uint32_t *const mark = reinterpret_cast<uint32_t *>(smem + C::OFF_MARK) + rt * 128 + row;
#pragma unroll
            for (int w = 0; w < C::MARK_WORDS; ++w)
                mark[w * R] = 0;

            int whole0 = 0, whole1 = 0;
            if (!dry)
                whole_of(from, whole0, whole1);
            uint32_t d = n_done;
            for (int j = j0; j < n; j += every, ++d) {
                const uint32_t g = it + j, b = NS == 2 ? d & 1 : 0;
                const bool fresh = j < every, last = j + every >= n;   // the first of them, the last
                wait(C::BAR_S_FULL + rt * NS + b, d / NS & 1);
                tc_fence_after();
                const uint32_t s_addr = tmem + lanes + C::TM_S + (rt * NS + b) * TILE;
                const uint32_t p_addr = C::P_APART ? tmem + lanes + C::TM_P + rt * C::P_STEP : dry ? o_addr : s_addr;
                // The loop over tiles is sensitive to what else it holds.  So a tile in which a row does not
                // see a key has its scores masked where they are, before they are read, and large scores are
                // replaced by their differences where they are, and read again.  (Both in registers:
                // 371 us for the prompt chunk at D = 128, 318 at D = 64; masks so, large ones by a loop
                // of their own: 359 and 348; so 356 and 297.)
                {
                    const uint32_t info = dry ? +WHOLE : sh_info[g % C::RING];
                    if (!(info & WHOLE)) {
                        const int pos0 = from + j * TILE, above = sees->x - pos0, below = sees->y - pos0;
                        mask_scores<C>(s_addr, above, below, info, a.c.page_shift);
                        if (j < whole0 || j >= whole1) {
                            wait(C::BAR_CLEAN + g % C::NC, g / C::NC & 1);
                            const volatile uint32_t *const odd = sh_odd + g % C::RING * 4;
                            if (odd[0] | odd[1] | odd[2] | odd[3])
                                mark_odd<C>(a, odd, line.b, line.h, pos0, above > 0 ? above : 0, below < TILE ? below : TILE, mark);
                        }
                    }
                }
                float s[TILE];
                float alpha = 1.f;
                bool grow = false, moved = false;
                while (true) {
                    uint32_t r[4][32];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        tmem_ld32(s_addr + 32 * q, r[q]);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        tmem_ld_wait(r[q]);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            s[32 * q + e] = __uint_as_float(r[q][e]);
                    if (moved)
                        break;
                    // the tile's largest score: four independent chains of 3-input maxima
                    float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
#pragma unroll
                    for (int k = 4; k < TILE; k += 8) {
                        mx0 = max3(mx0, s[k], s[k + 1]);
                        mx1 = max3(mx1, s[k + 2], s[k + 3]);
                        if (k + 4 < TILE) {
                            mx2 = max3(mx2, s[k + 4], s[k + 5]);
                            mx3 = max3(mx3, s[k + 6], s[k + 7]);
                        }
                    }
                    const float mx = fmaxf(max3(mx0, mx1, mx2), mx3);
                    const bool raise = !fresh && (mx - M) * c > SLACK;
                    grow = __any_sync(0xffffffffu, raise);
                    if (fresh || grow) {
                        if (raise)
                            alpha = to_frame<C>(M, mx, c);
                        M = fresh || raise ? mx : M;
                        // (a row may see nothing so far: any finite reference gives it weights of 0)
                        add = M == -INFINITY ? 0.f : -reference<C>(M, c);
                        large = __any_sync(0xffffffffu, fabsf(add) > LARGE && !dry);
                    }
                    if (!large)
                        break;
                    moved = true;
                    shift_columns<TILE>(s_addr, fabsf(add) > LARGE ? M : 0.f);
                }
                // O is brought to a larger reference (only in warps in which a row's grew) once the tile
                // before's product has landed, and weights apart go where that tile's were.  A parity tells
                // a phase from the one before only: a tile's scores were issued after the product of the
                // one NS before, or two before (weights apart), so this wait is for the phase in
                // flight or the last one; and the last tile waits in any case, so that the end's wait
                // is as well.
                bool waited = fresh;
                auto wait_product = [&] {
                    if (!waited) {
                        wait(C::BAR_O_DONE + rt, (d - 1) & 1);
                        waited = true;
                        tc_fence_after();
                    }
                };
                if (C::P_APART || grow)
                    wait_product();
                if (grow)
                    scale_columns<D>(o_addr, alpha);
                if (C::P_APART) {
                    tc_fence_before();
                    arrive(C::BAR_S_EMPTY + rt);
                }
                float seen[2] = {};
                uint64_t sum[2] = {};            // packed (0.f, 0.f)
                const float plus = large && fabsf(add) > LARGE ? C::LIFT : add;
                const uint64_t c2 = f32x2(c, c), add2 = f32x2(plus, plus);
                auto weights = [&](auto half) {
                    constexpr int H = decltype(half)::value;
                    uint32_t p[32], low[C::TWO ? 32 : 1];
#pragma unroll
                    for (int k = 0; k < 64; k += 4) {
                        const float *const x = s + H * 64 + k;
                        float x0, x1, x2, x3;
                        unpack_f32x2(fma_f32x2(f32x2(x[0], x[1]), c2, add2), x0, x1);
                        unpack_f32x2(fma_f32x2(f32x2(x[2], x[3]), c2, add2), x2, x3);
                        const float p0 = ex2_approx(x0), p1 = ex2_approx(x1), p2 = ex2_approx(x2), p3 = ex2_approx(x3);
                        sum[0] = add_f32x2(sum[0], f32x2(p0, p1));
                        sum[1] = add_f32x2(sum[1], f32x2(p2, p3));
                        p[k / 2] = pack2<F16>(p0, p1);
                        p[k / 2 + 1] = pack2<F16>(p2, p3);
                        if constexpr (C::SEEN) {
                            seen[0] = add_bf16x2_to_f32(seen[0], p[k / 2]);
                            seen[1] = add_bf16x2_to_f32(seen[1], p[k / 2 + 1]);
                        }
                        if constexpr (C::TWO) {
                            float z0, z1, z2, z3;
                            unpack2<F16>(p[k / 2], z0, z1);
                            unpack2<F16>(p[k / 2 + 1], z2, z3);
                            low[k / 2] = pack2<F16>(p0 - z0, p1 - z1);
                            low[k / 2 + 1] = pack2<F16>(p2 - z2, p3 - z3);
                        }
                    }
                    tmem_st32(p_addr + H * 32, p);
                    if constexpr (C::TWO)
                        tmem_st32(p_addr + C::P_LOW + H * 32, low);
                };
                weights(std::integral_constant<int, 0>{});
                tmem_st_wait();
                tc_fence_before();
                arrive(C::BAR_PA + rt * NS + b);
                weights(std::integral_constant<int, 1>{});
                float a0, a1, a2, a3;
                unpack_f32x2(sum[0], a0, a1);
                unpack_f32x2(sum[1], a2, a3);
                l = fmaf(l, alpha, (a0 + a1) + (a2 + a3));
                l_seen = C::SEEN ? fmaf(l_seen, alpha, seen[0] + seen[1]) : l;
                if (last)
                    wait_product();
                tmem_st_wait();
                tc_fence_before();
                arrive(C::BAR_P + rt * NS + b);
            }
            if (dry) {
                tmem_st_wait();
                asm volatile("bar.sync 5, %0;" ::"n"(C::T) : "memory");   // the line is laid out
                if (!sh.any)
                    break;
                dry = false;
                ok = true;
                arriving = 0;
                continue;
            }

            // ---- O out of tensor memory: the unit's rows, or this part of them
            it += n;
            const int mine = twin ? (n + 1 - rt) >> 1 : n;
            n_done += mine;
            if (mine > 0)
                wait(C::BAR_O_DONE + rt, (n_done - 1) & 1);
            // Twins: both tiles' references and sums; each tile's warps then take half of the columns.
            float f0 = 1.f, f1 = 0.f;
            if (twin) {
                float4 *const sums = reinterpret_cast<float4 *>(smem + C::OFF_SUM) + row;
                sums[rt * 128] = make_float4(M, l, l_seen, 0.f);
                tc_fence_before();
                all_sync();
                const float4 x = sums[0], y = sums[128];
                M = fmaxf(x.x, y.x);
                f0 = to_frame<C>(x.x, M, c);
                f1 = to_frame<C>(y.x, M, c);
                l = x.y * f0 + y.y * f1;
                l_seen = x.z * f0 + y.z * f1;
            }
            tc_fence_after();
            const int first_cta = cut ? sh.range.owner(line.at) : cta;
            const int last_cta = cut ? sh.range.owner(line.last()) : cta;
            const bool alone = first_cta == last_cta;
            const float inv = l_seen == 0.f ? 0.f : 1.f / l_seen;
            // log2 of the weights' sum, relative to M c itself
            const float y = l == 0.f ? -INFINITY
                                     : lg2_approx(l * (1.f / Weight<F16>::UNIT)) -
                                           (fabsf(reference<C>(M, c)) > LARGE ? 0.f : left_out<C>(M, c));
            const Row at = this_row();
            uint16_t *const o = static_cast<uint16_t *>(a.o) + line.b * a.o_sb;
            const long long o_place = at.live ? at.hq * a.o_sh + at.tok * a.o_sl : -1;
            float *const part = cut ? parts.data + (2 * static_cast<size_t>(cta) + (cta == first_cta ? 1 : 0)) *
                                                       cache::Parts::slot_floats(R, D)
                                    : nullptr;
            // a part's quadruple u of columns: neighbouring threads' rows lie next to each other
            auto place = [&](int u) { return (u * R + row_at) * 4; };
            const int chunk0 = twin ? rt : 0, chunks = twin ? 2 : 1;   // of 32 columns: the first, every
#pragma unroll 1
            for (int cc = chunk0; cc < D / 32; cc += chunks) {
                uint32_t r[32];
                tmem_ld32((twin ? o_addr - rt * D : o_addr) + 32 * cc, r);
                tmem_ld_wait(r);
                uint32_t marked = mark[cc * R];
                if (twin) {
                    marked |= mark[cc * R + (rt ? -128 : 128)];
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        r[k] = __float_as_uint(__uint_as_float(r[k]) * f0);
                    if (n > 1) {
                        uint32_t r1[32];
                        tmem_ld32(o_addr + (1 - rt) * D + 32 * cc, r1);
                        tmem_ld_wait(r1);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            r[k] = __float_as_uint(fmaf(__uint_as_float(r1[k]), f1, __uint_as_float(r[k])));
                    }
                }
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    r[k] = __float_as_uint(__uint_as_float(r[k]) * inv);
                if (marked)
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        r[k] = (marked >> k & 1) ? 0x7fc00000u : r[k];
                if (alone) {
                    // through shared memory, so that a row's 64 bytes leave together
                    const uint32_t out = base + C::OFF_OUT + warp * 2048;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        st_shared_v4(out + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4),
                                     pack2<F16>(__uint_as_float(r[8 * k]), __uint_as_float(r[8 * k + 1])),
                                     pack2<F16>(__uint_as_float(r[8 * k + 2]), __uint_as_float(r[8 * k + 3])),
                                     pack2<F16>(__uint_as_float(r[8 * k + 4]), __uint_as_float(r[8 * k + 5])),
                                     pack2<F16>(__uint_as_float(r[8 * k + 6]), __uint_as_float(r[8 * k + 7])));
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int to = k * 8 + (lane >> 2);
                        const long long place = __shfl_sync(0xffffffffu, o_place, to);
                        uint4 x;
                        ld_shared_v4(out + to * 64 + (((lane & 3) ^ (to >> 1 & 3)) << 4), x.x, x.y, x.z, x.w);
                        if (place >= 0)
                            *reinterpret_cast<uint4 *>(o + place + cc * 32 + (lane & 3) * 8) = x;
                    }
                    __syncwarp();
                } else {
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        *reinterpret_cast<uint4 *>(part + place(cc * 8 + k / 4)) = make_uint4(r[k], r[k + 1], r[k + 2], r[k + 3]);
                }
            }
            tc_fence_before();
            auto write_lse = [&](float v) {
                a.lse[(static_cast<long long>(line.b) * a.Hq + at.hq) * a.Lq + at.tok] = v * 0.69314718055994531f;
            };
            if (alone) {
                if (chunk0 == 0 && at.live)
                    write_lse(y == -INFINITY ? y : log2_sum(M, c, y));
            } else {
                if (chunk0 == 0)
                    reinterpret_cast<float2 *>(part + R * D)[row_at] = make_float2(y == -INFINITY ? NONE : M, y);
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
                if (row == 0 && rt == tile) {
                    int *const counter = parts.counters + 2 * first_cta + tile;
                    *last = atomicAdd(counter, 1) == last_cta - first_cta;
                    if (*last)
                        *counter = 0;
                }
                sync();
                if (*last) {
                    __threadfence();
#pragma unroll 1
                    for (int cc = chunk0; cc < D / 32; cc += chunks) {
                        float4 v[8];
                        const auto offset = [&](int k) { return place(cc * 8 + k); };
                        const float merged = paged::merge_row<C, 8, 2>(parts, c, first_cta, last_cta, row_at, offset, v);
                        if (at.live) {
#pragma unroll
                            for (int k = 0; k < 8; k += 2)
                                *reinterpret_cast<uint4 *>(o + o_place + cc * 32 + k * 4) =
                                    make_uint4(pack2<F16>(v[k].x, v[k].y), pack2<F16>(v[k].z, v[k].w),
                                               pack2<F16>(v[k + 1].x, v[k + 1].y), pack2<F16>(v[k + 1].z, v[k + 1].w));
                            if (cc == 0)
                                write_lse(merged);
                        }
                    }
                }
            }
            // the marks and O are read
            if (twin)
                all_sync();
            if (!next_unit())
                break;
        }
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
    cache::Parts parts;
    if (!cache::parts_of<C>(a, parts))
        return FA2_ERR_INVALID_ARG;
    const int grid = paged::line_grid<C>(a, parts.data != nullptr);
    if (grid == 0)
        return FA2_ERR_UNSUPPORTED;
    const cache::EncodeTiled encode = cache::encode_tiled();
    CUtensorMap k_map, v_map;
    const int rows = 1 << a.c.page_shift;
    if (!encode || !page_map(encode, &k_map, a.c.k, a.c, C::D, rows) || !page_map(encode, &v_map, a.c.v, a.c, C::D, rows))
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

}  // namespace paged
}  // namespace fa2
