// fa2_paged_step.cuh -- attention of a few query rows over the paged 16-bit cache
// (fa2_paged_attn in include/fa2_paged.h): the step of a decoding server.
//
// The query heads that share a key/value head and the query tokens of a sequence are the
// rows of one small matrix: row r is token r / G, head r % G of the group, so a cache byte
// is read once for all of them.
//
// Mathematics.  Both products are taken transposed, so that the cache, as it lies in its
// pages, is the 128-row operand of the tensor cores and the few query rows are columns:
//     S^T [128 keys, R] = K q^T
//     O^T [D, 2 R]      = V^T [p0 | p1]^T
// A thread owns a key of the tile (S) and a column d (O).  With c = scale log2 e and M a score of
// the row, the largest so far or up to SLACK / c below it,
//     p_j = 2^((S_j - M) c + LIFT),   p0 = p rounded to the cache's type, p1 = p - p0 rounded
// and O and l += p are fp32 in registers, brought to a larger M only when a tile's scores pass it by
// more than SLACK in the exponent, which every thread sees of its own key: most tiles need no
// maximum.  Two terms cost no time (the columns are few) and hold a weight to 2^-16 (bf16) or 2^-22
// (fp16): with one, O would be off by as much again as its own rounding.  M is a score as the
// product gave it, and every exponent a difference of scores times c, so scores may be of any
// size.
//
// What bounds it.  One token of a group of 8 does 8 operations a cache byte, the card could
// do 280: the bytes are the time, and no other unit may come near it.  The cache is not
// touched by the threads at all: TMA puts pages into a ring of shared-memory slots of 128
// keys, one thread issues the products, and 128 threads do the softmax of R columns; the
// copies run ahead by the ring's depth.  Work is cut and merged as in fa2_paged_line.cuh.  Up
// to 16 rows two CTAs share an SM and hide each other's beginnings and ends; 17 to 32 take two
// groups of four softmax warps, half of the rows each, in one CTA with twice the ring.
//
// Measured (in a graph; calls from Python, one after the other, take 2 us more).  One token of 40
// sequences of up to 10000 keys, 32 and 8 heads of 128: 824 MB in
// 126 us, 6.5 TB/s, 0.96 of the measured copy rate; two of up to 131072 keys 946 MB in 141 us, 0.99;
// 16 of 6000 keys with heads of 64 197 MB in 39 us (their tiles are half as many bytes for the same
// softmax); 8 of 8000 with heads of 256 525 MB in 86 us.  One short context is 8.2 to 8.6 us: a
// launch, ways to memory one after the other (lengths, table, page), a first tile and a merge.
#pragma once

#include <atomic>

#include "fa2_paged.cuh"
#include "fa2_paged_line.cuh"
#include "fa2_paged_merge.cuh"

namespace fa2 {
namespace paged {

template <int D_, int R_, bool F16_>
struct StepCfg {
    static constexpr int D = D_;
    static constexpr int R = R_;                     // query rows of a unit
    static constexpr bool F16 = F16_;
    static constexpr int TILE = 128;                 // keys
    // see fa2_paged_line.cuh
    // (COST: 24 sequences of 2000 keys, 24 rows of D = 64, 17.2 us with 12 and 16, 19.2 with 5 and 8; all
    // else is within 4 % of each other.  Grains of 128 keys: within 2 %.)
    static constexpr int GRAIN_SHIFT = 6, COST = 12, LEAST = 4;
    __host__ __device__ static constexpr int weight_shift(int, int grain_shift) { return grain_shift - 5; }   // a place: 32 keys
    // More than 16 rows are shared by two groups of four softmax warps, each with all keys of a tile and
    // half of the rows; one CTA an SM then.
    static constexpr int NW = R > 16 ? 2 : 1, RW = R / NW;
    static constexpr int CTAS = D == 256 || NW == 2 ? 1 : 2;    // an SM
    static constexpr int SOFTMAX = 128 * NW, WARP_LOAD = 4 * NW, WARP_MMA = WARP_LOAD + 1;   // SOFTMAX: threads
    static constexpr int T = NW == 2 ? SOFTMAX + 128 : SOFTMAX + 64;
    // With three warpgroups (two idle warps in the last) the launch leaves 168 registers a thread; the
    // softmax rises.
    static constexpr bool REG_SPLIT = NW == 2;
    static constexpr int REG_SOFTMAX = 216, REG_CTRL = 72;
    static_assert(2 * REG_SOFTMAX + REG_CTRL <= 3 * 168, "the split draws on the launch's registers");
    static constexpr float LIFT = Weight<F16>::LIFT, SLACK = 8.f;

    // A tile's keys, and its values, are PARTS slots of the ring, of up to 128 columns each, in
    // panels of 64 columns (128 bytes a row, the swizzle's span).
    static constexpr int PARTS = D == 256 ? 2 : 1, PANELS = D / PARTS / 64;
    static constexpr int PANEL = TILE * 128, SLOT = PANELS * PANEL;
    static constexpr int SLOTS = D == 256 ? 6 : (D == 128 ? 3 : 6) * NW;
    static constexpr int NQ = R < 16 ? 16 : R, Q_PANEL = NQ * 128;  // rows of q (the product wants 16)
    // Weights lie as a thread has them, a key's [p0 | p1] in a row of 64 or 128 bytes (the swizzle's span),
    // 64 columns a panel: four 16-byte stores for 16 rows where keys along a row would take 32 of two.
    static constexpr int NP = 2 * R, P_ROW = NP < 64 ? 64 : 128, P_PANEL = TILE * P_ROW, P_PANELS = NP < 64 ? 1 : NP / 64;
    static constexpr int OFF_RING = 0, OFF_P = SLOTS * SLOT, OFF_Q = OFF_P + P_PANELS * P_PANEL,
                         OFF_ROWS = OFF_Q + D / 64 * Q_PANEL;
    // per row: the maxima of four warps, the reference, a factor, first and last visible key
    static constexpr int OFF_MAX = OFF_ROWS, OFF_REF = OFF_MAX + R * 16, OFF_FACTOR = OFF_REF + R * 4, OFF_LO = OFF_FACTOR + R * 4;
    static constexpr int OFF_HI = OFF_LO + R * 4, OFF_L = OFF_HI + R * 4;   // (OFF_L: four sums)
    static constexpr int OFF_PLACE = OFF_L + R * 16;   // places in o and lse
    static constexpr int OFF_FLAGS = OFF_PLACE + R * 16, OFF_ODD = OFF_FLAGS + 32 * NW, OFF_INFO = OFF_ODD + 16 * NW;
    static constexpr int RING = 8;                                  // of tiles: pages that are there (OFF_INFO)
    static constexpr int OFF_BAR = OFF_INFO + RING * 4;
    static constexpr int NUM_BAR = 2 * SLOTS + 8;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BAR * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;         // 1024: operand alignment

    static constexpr int TM_S = 0, TM_O = 2 * NQ;                   // O: NP columns for each part
    static constexpr int TM_USED = TM_O + PARTS * NP;
    static constexpr int TMEM_COLS = TM_USED <= 64 ? 64 : TM_USED <= 128 ? 128 : TM_USED <= 256 ? 256 : 512;

    static constexpr int BAR_FULL = 0, BAR_EMPTY = SLOTS, BAR_Q_FULL = 2 * SLOTS, BAR_Q_EMPTY = BAR_Q_FULL + 1,
                         BAR_S_FULL = BAR_Q_FULL + 2, BAR_P_FULL = BAR_Q_FULL + 4, BAR_O_DONE = BAR_Q_FULL + 5,
                         BAR_DRAIN = BAR_Q_FULL + 6, BAR_ODD = BAR_Q_FULL + 7;   // (BAR_ODD: read by the second group)
    static_assert(SLOTS >= 3 * PARTS && SLOTS <= (2 * RING - 2) * PARTS, "a tile ahead; the ring of tiles' pages");
    static_assert(RW % 8 == 0 && RW <= 32 && TM_USED <= 512 && CTAS * TMEM_COLS <= 512, "tensor memory holds CTAS of them");
    static_assert(CTAS * (SMEM_BYTES + 1024 + 512) <= 228 * 1024, "an SM holds CTAS of them");
    static_assert(OFF_P % 1024 == 0 && OFF_Q % 1024 == 0, "swizzle atoms");
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
                const cache::Parts parts)
{
    using namespace ptx;
    using cache::Range;
    using cache::Seq;
    using cache::tmem_ld;
    using cache::tmem_pin;
    using cache::tmem_wait_ld;
    constexpr int D = C::D, R = C::R, RW = C::RW, TILE = C::TILE, SLOTS = C::SLOTS, PARTS = C::PARTS;
    constexpr bool F16 = C::F16;
    extern __shared__ uint8_t smem_raw[];
    __shared__ cache::LineShared sh_line;
    // Each warp's place on the line: it changes with the unit only, and would cost the roles
    // registers in their loops over tiles.
    struct Place {
        Range range;
        int first, end;
        Line<C> line;
    };
    __shared__ Place sh_places[C::T / 32];

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
            mbar_init(bar(i), i == C::BAR_Q_FULL || i == C::BAR_P_FULL ? 4 * C::NW : i == C::BAR_ODD ? 4 : 1);
        fence_mbar_init();
        tma_prefetch_desc(&k_map);
        tma_prefetch_desc(&v_map);
    }
    tc_fence_before();
    bool any;
    {
        Place mine;
        any = paged::find_range<C, C::T>(a, cut, sh_line, mine.range, mine.first, mine.end, mine.line, tid,
                                         [] { __syncthreads(); });
        if (any && lane == 0)
            sh_places[warp] = mine;
        __syncwarp();
    }
    if (!any) {
        if (warp == C::WARP_MMA) {
            __syncwarp();
            tmem_dealloc(*tmem_slot, C::TMEM_COLS);
        }
        return;
    }
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Place &place = sh_places[warp];
    const Line<C> &line = place.line;

    // A wait that ran out is recorded and not waited for again: the role runs on to its end
    // without waiting (its outputs are undefined), so that barriers between warps still match.
    bool ok = true;
    auto warp_wait = [&](int i, uint32_t parity, int code) {
        if (ok)
            ok = cache::wait_phase(bar(i), parity, a.err, code | i, a.wait_limit_ns);
    };
    auto warp_arrive = [&](int i) {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(i));
    };
    // the unit's keys [from, stop) in this CTA's range, and the tiles they make
    auto part_of = [&](int &from, int &stop) { return line.piece(a, cut, place.first, place.end, from, stop); };
    auto next_unit = [&]() -> bool {     // by a whole warp
        __syncwarp();
        bool more = false;
        if (lane == 0)
            more = sh_places[warp].line.next(a, place.end);
        __syncwarp();                    // (a shuffle orders no memory)
        return __shfl_sync(0xffffffffu, more, 0);
    };
    volatile uint32_t *const sh_info = reinterpret_cast<uint32_t *>(smem + C::OFF_INFO);   // [RING]: bit i: page i is there
    // tile g's keys are items 2 g PARTS .. of the ring, its values the PARTS after them
    uint32_t it = 0, unit = 0;   // tiles and units before the present unit

    if (warp >= C::WARP_LOAD) {
        if constexpr (C::REG_SPLIT)
            setmaxnreg_dec<C::REG_CTRL>();
        if (warp == C::WARP_LOAD) {
            // ============================================ pages -> ring
            const int pages = TILE >> a.c.page_shift;          // of a tile: one a lane
            const uint32_t page_bytes = static_cast<uint32_t>(C::PANELS) * 128 << a.c.page_shift;   // of a slot
            const uint32_t offset = static_cast<uint32_t>(lane) * 128 << a.c.page_shift;             // in each panel
            uint32_t issued = 0;                               // items
    #pragma unroll 1
            for (int i = a.naps; i > 0; --i)
                __nanosleep(500);
            do {
                int from, stop;
                const int n = part_of(from, stop), h = line.h;
                auto page_at = [&](int j) {                    // -1: none, or not seen
                    const int pos = from + j * TILE + (lane << a.c.page_shift);
                    const bool seen = j < n && lane < pages && pos < stop && pos + (1 << a.c.page_shift) > line.span.lo;
                    return seen ? cache::page_of(a.c, line.b, pos >> a.c.page_shift) : -1;
                };
                int id = page_at(0), id_next = page_at(1);     // two tiles ahead
                for (int j = 0; j < n && ok; ++j) {
                    const int id_after = page_at(j + 2);
                    const uint32_t there = __ballot_sync(0xffffffffu, id >= 0);
                    const uint32_t bytes = __popc(there) * page_bytes;
    #pragma unroll
                    for (int k = 0; k < 2 * PARTS; ++k) {
                        const uint32_t item = 2 * PARTS * (it + j) + k, slot = item % SLOTS, full = bar(C::BAR_FULL + slot);
                        if (item >= SLOTS)
                            warp_wait(C::BAR_EMPTY + slot, (item / SLOTS - 1) & 1, STEP_ERR_LOAD);
                        if (!ok)
                            break;
                        // (Whose place the tile RING back had: it has been through its softmax, for a
                        // slot of its values came back before this.)
                        if (lane == 0) {
                            if (k == 0)
                                sh_info[(it + j) % C::RING] = there;
                            cache::expect_tx(full, bytes);
                        }
                        __syncwarp();
                        if (id >= 0)
    #pragma unroll
                            for (int p = 0; p < C::PANELS; ++p)
                                tma_load_4d(base + C::OFF_RING + slot * C::SLOT + p * C::PANEL + offset,
                                            k >= PARTS ? &v_map : &k_map, (k % PARTS * C::PANELS + p) * 64, 0, h, id, full);
                        warp_arrive(C::BAR_FULL + slot);
                        issued = item + 1;
                    }
                    id = id_next;
                    id_next = id_after;
                }
                it += n;
            } while (ok && next_unit());
            // the copies in flight have landed before the CTA goes
            for (uint32_t item = issued > SLOTS ? issued - SLOTS : 0; item < issued; ++item) {
                const int i = C::BAR_FULL + item % SLOTS;
                cache::wait_phase(bar(i), item / SLOTS & 1, a.err, STEP_ERR_DRAIN | i, a.drain_limit_ns);
            }
        } else if (warp == C::WARP_MMA) {
            // ============================================ one thread issues the products
            if (elect_one()) {
                const uint64_t desc_q = sdesc_sw128(base + C::OFF_Q, 16, 1024), desc_k = sdesc_sw128(base, 16, 1024);
                const uint64_t desc_p = C::P_ROW == 64 ? cache::sdesc_sw64(base + C::OFF_P, 0, 512)
                                                       : sdesc_sw128(base + C::OFF_P, C::P_PANEL, 1024);
                // V^T: d is the contiguous direction.  At D = 64 the 128 rows are the 64 columns
                // twice (stride 0), and lanes 64.. of O^T a copy that nobody reads.
                const uint64_t desc_v = sdesc_sw128(base, D == 64 ? 0 : C::PANEL, 1024);
                auto wait = [&](int i, uint32_t parity) {
                    if (ok)
                        ok = lone_wait(bar(i), parity, a.err, STEP_ERR_MMA | i, a.wait_limit_ns);
                };
                auto wait_item = [&](uint32_t item) { wait(C::BAR_FULL + item % SLOTS, item / SLOTS & 1); };
                auto issue_s = [&](uint32_t g, bool last) {
    #pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        const uint32_t item = 2 * PARTS * g + part, slot = item % SLOTS;
                        wait_item(item);
                        if (!ok)
                            return;
                        tc_fence_after();
                        const uint64_t dk = desc_k + (C::OFF_RING + slot * C::SLOT >> 4);
    #pragma unroll
                        for (int kk = 0; kk < C::PANELS * 4; ++kk)
                            mma_ss(tmem + C::TM_S + (g & 1) * C::NQ, dk + ((kk >> 2) * C::PANEL + (kk & 3) * 32 >> 4),
                                   desc_q + ((part * C::PANELS + (kk >> 2)) * C::Q_PANEL + (kk & 3) * 32 >> 4),
                                   idesc(F16, 128, C::NQ, false, false), part > 0 || kk > 0);
                        if (part == PARTS - 1)
                            mma_commit(bar(C::BAR_S_FULL + (g & 1)));
                        mma_commit(bar(C::BAR_EMPTY + slot));
                    }
                    if (last)
                        mma_commit(bar(C::BAR_Q_EMPTY));
                };
                auto issue_pv = [&](uint32_t g) {
                    wait(C::BAR_P_FULL, g & 1);
    #pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        const uint32_t item = 2 * PARTS * g + PARTS + part, slot = item % SLOTS;
                        wait_item(item);
                        if (!ok)
                            return;
                        tc_fence_after();
                        const uint64_t dv = desc_v + (C::OFF_RING + slot * C::SLOT >> 4);
    #pragma unroll
                        for (int kk = 0; kk < TILE / 16; ++kk)
                            mma_ss(tmem + C::TM_O + part * C::NP, dv + (kk * 16 * 128 >> 4),
                                   desc_p + (kk * 16 * C::P_ROW >> 4), idesc(F16, 128, C::NP, true, true), kk > 0);
                        if (part == PARTS - 1)
                            mma_commit(bar(C::BAR_O_DONE));
                        mma_commit(bar(C::BAR_EMPTY + slot));
                    }
                };
                do {
                    int from, stop;
                    const int n = part_of(from, stop);
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
                } while (ok && sh_places[C::WARP_MMA].line.next(a, place.end));
                // nothing issued is still running when tensor memory is given back
                mma_commit(bar(C::BAR_DRAIN));
                lone_wait(bar(C::BAR_DRAIN), 0, a.err, STEP_ERR_DRAIN | C::BAR_DRAIN, a.drain_limit_ns);
            }
            __syncwarp();
        }
    } else {
        if constexpr (C::REG_SPLIT)
            setmaxnreg_inc<C::REG_SOFTMAX>();
        // ============================================ softmax: thread = key of S^T, column d of O^T
        // rows row0 .. of the block are this thread's; with their number within that, r below
        const int group = warp >> 2, key = tid & 127, row0 = group * RW;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float c = a.scale * 1.4426950408889634f;
        auto floats = [&](int offset) { return reinterpret_cast<float *>(smem + offset); };
        auto ints = [&](int offset) { return reinterpret_cast<int *>(smem + offset); };
        float *const sh_max = floats(C::OFF_MAX) + row0 * 4, *const sh_l = floats(C::OFF_L) + row0 * 4;      // [R][4]
        float *const sh_ref = floats(C::OFF_REF) + row0, *const sh_factor = floats(C::OFF_FACTOR) + row0;    // [R]
        int *const sh_lo = ints(C::OFF_LO) + row0, *const sh_hi = ints(C::OFF_HI) + row0;                    // [R]
        longlong2 *const sh_place = reinterpret_cast<longlong2 *>(smem + C::OFF_PLACE);         // [R], of all rows
        volatile uint32_t *const sh_flags = reinterpret_cast<uint32_t *>(smem + C::OFF_FLAGS) + group * 8;   // [2][4]
        volatile uint32_t *const sh_odd = reinterpret_cast<uint32_t *>(smem + C::OFF_ODD) + group * 4;       // [4]
        // the group's four warps; all of them
        auto sync = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); };
        auto sync_all = [] { asm volatile("bar.sync 3, %0;" ::"n"(C::SOFTMAX) : "memory"); };
        const bool owns_d = D > 64 || key < 64;
        uint32_t odd_tiles = 0;   // tiles with an infinity or NaN that not every row sees, before this one
        // N consecutive columns of tensor memory; valid after the wait
        auto columns = [](uint32_t addr, auto &to) {
            constexpr int N = sizeof(to) / 4;
            if constexpr (N == 32) {
                tmem_ld32(addr, to);
            } else if constexpr (N == 16) {
                tmem_ld(addr, to);
            } else {
                static_assert(N == 8, "8, 16 or 32");
                tmem_ld(addr, *reinterpret_cast<uint32_t(*)[4]>(to));
                tmem_ld(addr + 4, *reinterpret_cast<uint32_t(*)[4]>(to + 4));
            }
        };

        do {
            int from, stop;
            const int n = part_of(from, stop), b = line.b, h = line.h, rb = line.rb;
            const Seq s = line.s;
            const Span span = line.span;
            const int rows = s.n * a.G, live = rows - rb * R - row0;   // of this group's rows
            int all_lo, all_hi;
            line.seen_by_all(a, all_lo, all_hi);

            // ---- q; TPR threads a row
            if (unit > 0)
                warp_wait(C::BAR_Q_EMPTY, (unit - 1) & 1, STEP_ERR_SOFTMAX);
            {
                constexpr int TPR = C::SOFTMAX / R, E = D / TPR;   // threads a row, numbers a thread
                const int r = tid / TPR, d0 = tid % TPR * E;
                const int rr = rb * R + r, tok = rr / a.G, hq = h * a.G + rr % a.G;
                const bool is_row = rr < rows;
                const uint16_t *q = static_cast<const uint16_t *>(a.q) + b * a.q_sb + hq * a.q_sh + tok * a.q_sl + d0;
                uint2 w[E / 4];
#pragma unroll
                for (int k = 0; k < E / 4; ++k)
                    w[k] = is_row ? __ldg(reinterpret_cast<const uint2 *>(q) + k) : make_uint2(0, 0);
#pragma unroll
                for (int k = 0; k < E / 4; ++k) {
                    const int d = d0 + 4 * k, col = d % 64 * 2;
                    *reinterpret_cast<uint2 *>(smem + C::OFF_Q + d / 64 * C::Q_PANEL + r * 128 + (((col >> 4) ^ (r & 7)) << 4) +
                                               (col & 15)) = w[k];
                }
                if (tid % TPR == 0) {
                    const int pos = s.kv - s.n + tok;
                    const long long lo = static_cast<long long>(pos) - a.window;
                    sh_ref[r - row0] = is_row ? NONE : 0.f;
                    sh_hi[r - row0] = !is_row ? 0 : a.causal ? pos + 1 : s.kv;
                    sh_lo[r - row0] = a.window >= 0 && lo > 0 ? static_cast<int>(lo) : 0;
                    sh_place[r] = make_longlong2(is_row ? b * a.o_sb + hq * a.o_sh + tok * a.o_sl : -1,
                                                 (static_cast<long long>(b) * a.Hq + hq) * a.Lq + tok);
                }
                fence_proxy_async_shared();
                warp_arrive(C::BAR_Q_FULL);
            }
            const int first_cta = cut ? place.range.owner(line.at) : cta;
            const int last_cta = cut ? place.range.owner(line.last()) : cta;
            const bool alone = first_cta == last_cta;
            float *const part = cut ? parts.data + (2 * static_cast<size_t>(cta) + (cta == first_cta ? 1 : 0)) *
                                                       cache::Parts::slot_floats(R, D)
                                    : nullptr;
            sync();   // the rows' limits are there

            float acc[PARTS][RW], l[RW];
#pragma unroll
            for (int r = 0; r < RW; ++r)
                acc[0][r] = acc[PARTS - 1][r] = l[r] = 0.f;
            uint32_t odd_rows[PARTS] = {};   // rows whose O at this d a visible infinity or NaN makes NaN

            // O^T of the tile before `g` into the registers
            auto add_tile = [&](uint32_t g) {
                warp_wait(C::BAR_O_DONE, (g - 1) & 1, STEP_ERR_SOFTMAX);
                tc_fence_after();
                constexpr int BATCH = RW < 16 ? RW : 16;   // rows whose loads are under way together
#pragma unroll
                for (int half = 0; half < PARTS; ++half)
#pragma unroll
                    for (int r0 = 0; r0 < RW; r0 += BATCH) {
                        uint32_t t0[BATCH], t1[BATCH];
                        const uint32_t addr = tmem + lanes + C::TM_O + half * C::NP + row0 + r0;
                        columns(addr, t0);
                        columns(addr + R, t1);
                        tmem_wait_ld();
                        tmem_pin(t0);
                        tmem_pin(t1);
#pragma unroll
                        for (int k = 0; k < BATCH; ++k)
                            acc[half][r0 + k] += __uint_as_float(t0[k]) + __uint_as_float(t1[k]);
                    }
                tc_fence_before();
            };

            for (int j = 0; j < n; ++j) {
                const uint32_t g = it + j, par = g & 1;
                const int pos = from + j * TILE + key;
                warp_wait(C::BAR_S_FULL + par, g >> 1 & 1, STEP_ERR_SOFTMAX);
                tc_fence_after();
                const bool there = (sh_info[g % C::RING] >> (key >> a.c.page_shift) & 1) && pos >= span.lo && pos < stop;
                const bool whole = there && pos >= all_lo && pos < all_hi;   // every row sees the key
                // (All rows, live or not, in straight runs: with a branch after every four of them a tile of
                // 8 rows took 1900 cycles, one of 64 rows 4800.)
                float x[RW];                  // scores, less the row's reference
                const bool some = __any_sync(0xffffffffu, there && !whole);   // a key that some rows see and some do not
                auto scores = [&] {           // -infinity where the row does not see the key
                    uint32_t s0[RW];
                    columns(tmem + lanes + C::TM_S + par * C::NQ + row0, s0);
                    tmem_wait_ld();
                    tmem_pin(s0);
#pragma unroll
                    for (int r = 0; r < RW; ++r)
                        x[r] = there ? __uint_as_float(s0[r]) : -INFINITY;
                    if (some)
#pragma unroll
                        for (int r = 0; r < RW; ++r)
                            x[r] = pos >= sh_lo[r] && pos < sh_hi[r] ? x[r] : -INFINITY;
                };
                auto maxima = [&] {           // of the warp's keys, by row
#pragma unroll
                    for (int r0 = 0; r0 < RW; r0 += 4) {
                        float mine = -INFINITY;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float m = warp_max(x[r0 + k]);
                            mine = lane == k ? m : mine;
                        }
                        if (lane < 4)
                            sh_max[(r0 + lane) * 4 + (warp & 3)] = mine;
                    }
                };
                const bool fresh = j == 0;
                bool high = false;            // a score too far above its reference (NONE until a row sees a key)
                scores();
                if (fresh) {
                    maxima();
                } else {
                    float over = -INFINITY;
#pragma unroll
                    for (int r = 0; r < RW; r += 4) {
                        const float4 ref = *reinterpret_cast<const float4 *>(sh_ref + r);
                        x[r] -= ref.x, x[r + 1] -= ref.y, x[r + 2] -= ref.z, x[r + 3] -= ref.w;
                        over = fmaxf(over, fmaxf(fmaxf(x[r], x[r + 1]), fmaxf(x[r + 2], x[r + 3])));
                    }
                    high = over * c > C::SLACK || over > 1e38f;
                }
                {
                    // bit 0: a key that no row sees; bit 1: one that some rows see; bit 2: high
                    const uint32_t f = (some ? 2u : 0u) | __reduce_or_sync(0xffffffffu, (there ? 0u : 1u) | (high ? 4u : 0u));
                    if (lane == 0)
                        sh_flags[par * 4 + (warp & 3)] = f;
                }
                sync();
                uint32_t f0, f1, f2, f3;
                ld_shared_v4(base + C::OFF_FLAGS + group * 32 + par * 16, f0, f1, f2, f3);
                const uint32_t flags = f0 | f1 | f2 | f3;
                bool added = fresh;
                if (fresh || (flags & 4)) {
                    // the rows' references become the largest scores so far, O and l go with them
                    if (!fresh) {
                        add_tile(g);
                        added = true;
                        scores();
                        maxima();
                        sync();
                    }
                    if (key < RW) {
                        const float4 m4 = *reinterpret_cast<const float4 *>(sh_max + key * 4);
                        const float before = sh_ref[key], now = fmaxf(fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w)), before);
                        sh_factor[key] = ex2_approx((before - now) * c);
                        sh_ref[key] = now;
                    }
                    sync();
#pragma unroll
                    for (int r = 0; r < RW; ++r) {
                        x[r] -= sh_ref[r];
                        if (!fresh) {
                            const float f = sh_factor[r];
                            l[r] *= f;
#pragma unroll
                            for (int half = 0; half < PARTS; ++half)
                                acc[half][r] *= f;
                        }
                    }
                }
                tc_fence_before();
                // weights
                uint32_t p[2][RW / 2];
#pragma unroll
                for (int r = 0; r < RW; r += 2) {
                    const float y0 = ex2_approx(fmaf(x[r], c, C::LIFT)), y1 = ex2_approx(fmaf(x[r + 1], c, C::LIFT));
                    l[r] += y0;
                    l[r + 1] += y1;
                    p[0][r / 2] = pack2<F16>(y0, y1);
                    float z0, z1;
                    unpack2<F16>(p[0][r / 2], z0, z1);
                    p[1][r / 2] = pack2<F16>(y0 - z0, y1 - z1);
                }
                // Keys that not every row sees: what lies in their slots' place in shared memory
                // may be anything, and NaN times a weight of 0 is NaN.
                if (flags & 3) {
                    uint32_t item[PARTS];
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        item[part] = 2 * PARTS * g + PARTS + part;
                        warp_wait(C::BAR_FULL + item[part] % SLOTS, item[part] / SLOTS & 1, STEP_ERR_SOFTMAX);
                    }
                    auto at = [&](int k, int d) -> uint8_t * {
                        const int col = d % 64 * 2, panel = d / 64;
                        return smem + C::OFF_RING + item[panel / C::PANELS] % SLOTS * C::SLOT + panel % C::PANELS * C::PANEL +
                               k * 128 + (((col >> 4) ^ (k & 7)) << 4) + (col & 15);
                    };
                    if (!there && group == 0)
#pragma unroll
                        for (int d = 0; d < D; d += 8)
                            *reinterpret_cast<uint4 *>(at(key, d)) = make_uint4(0, 0, 0, 0);
                    if (flags & 2) {
                        const bool odd = there && !whole && any_odd<F16, D / 8>([&](int i) { return at(key, 8 * i); });
                        const uint32_t votes = __ballot_sync(0xffffffffu, odd);
                        if (lane == 0)
                            sh_odd[warp & 3] = votes;
                        sync();
                        if (sh_odd[0] | sh_odd[1] | sh_odd[2] | sh_odd[3]) {   // (the same in both groups)
#pragma unroll 1
                            for (int k = 0; k < TILE; ++k) {
                                if (!(sh_odd[k >> 5] >> (k & 31) & 1))
                                    continue;
                                const int kp = from + j * TILE + k;
                                uint32_t see = 0;
                                for (int r = 0; r < RW; ++r)
                                    see |= (kp >= sh_lo[r] && kp < sh_hi[r] ? 1u : 0u) << r;
#pragma unroll
                                for (int half = 0; half < PARTS; ++half)
                                    if (owns_d && odd_lo<F16>(*reinterpret_cast<const uint16_t *>(at(k, half * 128 + key))))
                                        odd_rows[half] |= see;
                            }
                            // (Not a barrier of both groups: behind a wait that ran out one may come here and the
                            // other not.)
                            sync();
                            if (C::NW == 2 && group == 1)
                                warp_arrive(C::BAR_ODD);
                            if (C::NW == 2 && group == 0)
                                warp_wait(C::BAR_ODD, odd_tiles++ & 1, STEP_ERR_SOFTMAX);
                            if (odd && group == 0)
                                for (int d = 0; d < D; d += 8) {
                                    uint4 *w = reinterpret_cast<uint4 *>(at(key, d));
                                    *w = finite4<F16>(*w);
                                }
                        }
                    }
                }
                if (!added)
                    add_tile(g);   // (and its product no longer reads the weights' place)
#pragma unroll
                for (int r0 = 0; r0 < RW; r0 += 8) {
#pragma unroll
                    for (int term = 0; term < 2; ++term) {
                        const int col = (term * R + row0 + r0) * 2, in_row = col % C::P_ROW >> 4;   // bytes; 16-byte column
                        const int swizzle = C::P_ROW == 64 ? key >> 1 & 3 : key & 7;
                        st_shared_v4(base + C::OFF_P + col / C::P_ROW * C::P_PANEL + key * C::P_ROW + ((in_row ^ swizzle) << 4),
                                     p[term][r0 / 2], p[term][r0 / 2 + 1], p[term][r0 / 2 + 2], p[term][r0 / 2 + 3]);
                    }
                }
                fence_proxy_async_shared();
                warp_arrive(C::BAR_P_FULL);
            }
            it += n;
            // ---- a warp's sums, four rows at a time: lanes that differ in bit 4, then 3, take rows of their own
#pragma unroll
            for (int r0 = 0; r0 < RW; r0 += 4) {
                const bool b4 = lane & 16, b3 = lane & 8;
                float x0 = b4 ? l[r0 + 2] : l[r0], x1 = b4 ? l[r0 + 3] : l[r0 + 1];
                x0 += __shfl_xor_sync(0xffffffffu, b4 ? l[r0] : l[r0 + 2], 16);
                x1 += __shfl_xor_sync(0xffffffffu, b4 ? l[r0 + 1] : l[r0 + 3], 16);
                float x = b3 ? x1 : x0;
                x += __shfl_xor_sync(0xffffffffu, b3 ? x0 : x1, 8);
#pragma unroll
                for (int d = 4; d > 0; d >>= 1)
                    x += __shfl_xor_sync(0xffffffffu, x, d);
                if ((lane & 7) == 0)
                    sh_l[(r0 + (lane >> 4) * 2 + (lane >> 3 & 1)) * 4 + (warp & 3)] = x;
            }
            add_tile(it);      // (the last product, under the sums)
            sync();
            // ---- O and LSE of the unit's rows, or of this part of them
            auto sum_of = [&](int r) {
                const float4 l4 = *reinterpret_cast<const float4 *>(sh_l + r * 4);
                return r < live ? (l4.x + l4.y) + (l4.z + l4.w) : 0.f;
            };
            float y = -INFINITY;   // log2 of the weights' sum (a group's threads below RW)
            if (key < RW) {
                const float sum = sum_of(key);
                if (sum != 0.f)
                    y = lg2_approx(sum * (1.f / Weight<F16>::UNIT));
            }
            const float M = sh_ref[key < RW ? key : 0];
            uint16_t *const o = static_cast<uint16_t *>(a.o);
            auto write_lse = [&](int row, float v) {
                if (sh_place[row].x >= 0)
                    a.lse[sh_place[row].y] = v * 0.69314718055994531f;
            };
            if (key < RW) {
                if (alone)
                    write_lse(row0 + key, y == -INFINITY ? y : log2_sum(M, c, y));
                else
                    reinterpret_cast<float2 *>(part + R * D)[row0 + key] = make_float2(M, y);
            }
#pragma unroll
            for (int r0 = 0; r0 < RW; r0 += 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = r0 + k;
                    if (r >= live || !owns_d)
                        break;
                    const float sum = sum_of(r), inv = sum == 0.f ? 0.f : __fdividef(1.f, sum);
#pragma unroll
                    for (int half = 0; half < PARTS; ++half) {
                        const float v = odd_rows[half] >> r & 1 ? __uint_as_float(0x7fc00000u) : acc[half][r] * inv;
                        const int d = half * 128 + key;
                        if (alone)
                            o[sh_place[row0 + r].x + d] = static_cast<uint16_t>(pack2<F16>(v, 0.f));
                        else
                            part[(row0 + r) * D + d] = v;
                    }
                }
            }
            if (!alone) {
                // the CTA whose part is the last to arrive merges them
                volatile int *const last = reinterpret_cast<int *>(smem + C::OFF_MISC + 4);
                __threadfence();
                sync_all();
                if (tid == 0) {
                    int *const counter = parts.counters + 2 * first_cta;
                    *last = atomicAdd(counter, 1) == last_cta - first_cta;
                    if (*last)
                        *counter = 0;
                }
                sync_all();
                if (*last) {
                    __threadfence();
                    // N quadruples a thread, so that one pass takes the block (two where RW D is 4096)
                    constexpr int N = RW * D >= 2048 ? 4 : RW * D / 512, TPR = D / 4 / N;
                    const int all = rows - rb * R < R ? rows - rb * R : R;
                    for (int r = tid / TPR; r < all; r += C::SOFTMAX / TPR) {
                        float4 v[N];
                        auto column = [&](int k) { return (tid % TPR + k * TPR) * 4; };
                        const auto offset = [&](int k) { return r * D + column(k); };
                        const float merged = paged::merge_row<C, N, N <= 2 ? 8 : 4>(parts, c, first_cta, last_cta, r, offset, v);
#pragma unroll
                        for (int k = 0; k < N; ++k)
                            *reinterpret_cast<uint2 *>(o + sh_place[r].x + column(k)) =
                                make_uint2(pack2<F16>(v[k].x, v[k].y), pack2<F16>(v[k].z, v[k].w));
                        if (tid % TPR == 0)
                            write_lse(r, merged);
                    }
                }
            }
            ++unit;
            sync_all();   // the rows' places are free again
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

}  // namespace paged
}  // namespace fa2
