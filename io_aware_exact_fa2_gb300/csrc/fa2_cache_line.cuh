// fa2_cache_line.cuh -- how fa2_cache_attn's kernels share out their work: the key tiles
// of all sequences, heads and blocks of query rows as one line, cut into equal ranges.
//
// A unit is a block of C::R query rows of one (sequence, key/value head); it spans the
// tiles of C::TILE keys that any of its rows sees.  Units lie on the line in the order
// sequence, row block, head: the heads of a row block are alike, so a place on the line is
// found among the row blocks, which the threads of a CTA share out.
// A unit is C::UNIT_COST tiles longer on the line than it is, for what it costs to begin and
// end one; a range that holds only of those has nothing to do with the unit.  No range is
// shorter than C::MIN_TILES, for more of them than that only add parts to merge.  Measured
// (cost / least: us): ragged chunks of prompts, by rows, 2/2: 63.1, 3/2: 61.6, 4/3: 57.7,
// 5/3: 58.5, 7/4: 58.9; ragged steps, by columns, 1/1: 75, 2/1: 71, 3/1: 69; one short
// sequence, 3/1: 9.3, 3/2: 10.1, 3/4: 11.9.
// Lengths are device data, so every CTA lays out the line for itself.
#pragma once

#include "fa2_cache.cuh"
#include "sm103_ptx.cuh"

namespace fa2 {
namespace cache {

constexpr int CHUNK = 16;                 // keys of the smallest piece; divides every page size
// Query rows of a key/value head (Lq G) up to which they are columns of the products, in a
// block of 8 or 16 (fa2_cache_step.cuh); more are rows, up to 256 a block
// (fa2_cache_chunk.cuh).  Measured, in us: 16 sequences of 4000 positions, 8 heads of 128:
// columns 49 for 16 rows, 80 for 32 (two blocks), 137 for 64; rows 61 for any of them.
// 24 of 2000, 2 heads of 64: 21, 27, 39 against 27; 8 of 2000, 8 heads of 256: 33, 47, 76
// against 49.  (Two short sequences stay ahead as columns: 18 against 25 for 32 and 64 rows.
// How long they are the host does not know.)  A block of 8 rather than 16 for up to 8 rows:
// 41 against 45 at 16 sequences of 6000, 8 heads of 64; alike or 2 us ahead elsewhere.
constexpr long long kStepRows = 16;

// Parts of cut units: for each CTA two slots (its range's first unit, its last one) of
// R rows: O fp32, R D of them in the kernel's own order, then the log2-sum-exp2 [R], each as
// two floats (two_floats).
struct Parts {
    int *counters;      // [grid][2]: of the units that begin in a range and go on, arrived parts
    float *data;
    __host__ __device__ static constexpr size_t slot_floats(int R, int D) { return static_cast<size_t>(R) * (D + 2); }
    // (the same for every configuration: calls of different ones may take the same workspace
    // in turn, and none's data may lie where another's counters do)
    static constexpr int MAX_CTAS = 4;   // an SM
    __host__ __device__ static constexpr size_t counter_bytes(int num_sms)
    {
        return (static_cast<size_t>(num_sms) * MAX_CTAS * 2 * sizeof(int) + 255) & ~static_cast<size_t>(255);
    }
};

// Bytes of workspace for units of R rows of D.
template <class C>
size_t attn_workspace(int num_sms)
{
    static_assert(C::CTAS <= Parts::MAX_CTAS, "a counter pair a CTA");
    return Parts::counter_bytes(num_sms) +
           static_cast<size_t>(num_sms) * C::CTAS * 2 * Parts::slot_floats(C::R, C::D) * sizeof(float);
}

// The workspace as parts (none: null pointers); false if it is too small.
template <class C>
bool parts_of(const AttnArgs &a, Parts &parts)
{
    parts = Parts{nullptr, nullptr};
    if (!a.workspace)
        return true;
    if (a.workspace_bytes < attn_workspace<C>(a.num_sms))
        return false;
    parts.counters = static_cast<int *>(a.workspace);
    parts.data = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + Parts::counter_bytes(a.num_sms));
    return true;
}

// Places on the line: an int counts them, with room for what is added to a place.
constexpr int MAX_LINE = 1 << 30;

// CTAs to launch: no more than the longest sequences could make ranges for; 0 if the line
// could be longer than that.
template <class C>
int line_grid(const AttnArgs &a, bool cut)
{
    const long long most = a.num_sms * C::CTAS;
    const long long blocks = (static_cast<long long>(a.Lq) * a.G + C::R - 1) / C::R;
    const long long length = ((static_cast<long long>(a.c.max_pages) << a.c.page_shift) + C::TILE - 1) / C::TILE + 1 + C::UNIT_COST;
    const long long units = static_cast<long long>(a.c.B) * a.c.H * blocks;   // (B H, blocks < 2^31)
    if (units > MAX_LINE || units * length > MAX_LINE)
        return 0;
    const long long grid = cut ? (units * length + C::MIN_TILES - 1) / C::MIN_TILES : units;
    return static_cast<int>(grid > most ? most : grid);
}

#ifdef __CUDACC__

// Keys that a block of query rows sees at all: [lo, hi), and the tiles they span.
struct Span {
    int lo, hi, tiles;
};

struct Seq {
    int kv, n;      // positions held, query rows of them
};

__device__ __forceinline__ Seq sequence(const AttnArgs &a, int b)
{
    Seq s;
    const long long cap = static_cast<long long>(a.c.max_pages) << a.c.page_shift;
    const int kv = a.kv_lens[b];
    s.kv = kv < 0 ? 0 : kv > cap ? static_cast<int>(cap) : kv;
    const int n = a.q_lens ? a.q_lens[b] : a.Lq;
    s.n = n < 0 ? 0 : n > a.Lq ? a.Lq : n;
    return s;
}

template <class C>
__device__ __forceinline__ Span span_of(const AttnArgs &a, const Seq &s, int rb)
{
    const int rows = s.n * a.G;
    const int r1 = (rb + 1) * C::R < rows ? (rb + 1) * C::R : rows;
    const int i0 = rb ? rb * C::R / a.G : 0, i1 = r1 == rows ? s.n - 1 : (r1 - 1) / a.G;
    Span p;
    p.hi = a.causal ? s.kv - s.n + i1 + 1 : s.kv;
    p.hi = p.hi < 0 ? 0 : p.hi;
    p.lo = 0;
    if (a.window >= 0) {
        const long long lo = static_cast<long long>(s.kv) - s.n + i0 - a.window;
        p.lo = lo > 0 ? static_cast<int>(lo) : 0;
    }
    const int from = p.lo & ~(C::ALIGN - 1);
    p.tiles = p.hi > from ? (p.hi - from + C::TILE - 1) / C::TILE : 0;
    p.tiles = p.tiles > 0 ? p.tiles : 1;   // a unit that sees nothing still writes its rows
    return p;
}

template <class C>
__device__ __forceinline__ int row_blocks(const AttnArgs &a, const Seq &s)
{
    return (s.n * a.G + C::R - 1) / C::R;
}

// The line cut into `grid` ranges, the first `more` of them of size + 1 tiles.
struct Range {
    int grid, size, more;
    Range() = default;
    __device__ Range(int total, int ranges) : grid(ranges), size(total / ranges), more(total - total / ranges * ranges) {}
    __device__ int begin(int c) const { return c * size + (c < more ? c : more); }
    // the range that tile x lies in
    __device__ int owner(int x) const
    {
        const int y = x - more * (size + 1);
        return y < 0 ? x / (size + 1) : more + y / size;
    }
};

// A unit's place on the line.
template <class C>
struct Line {
    int at;            // its first tile
    int b, h, rb;
    Seq s;
    Span span;

    // The following unit; false if it begins at `end` or later, or nowhere.  (It is not looked for
    // there: behind the last one of a padded batch each sequence would be read first.  8 sequences
    // of 4000 in a batch of 1024: 18 us, 83 when they were.)
    __device__ __forceinline__ bool next(const AttnArgs &a, int end)
    {
        at += span.tiles + C::UNIT_COST;
        if (at >= end)
            return false;
        if (++h < a.c.H)
            return true;
        h = 0;
        if (++rb == row_blocks<C>(a, s)) {
            rb = 0;
            do {
                if (++b == a.c.B)
                    return false;
                s = sequence(a, b);
            } while (s.n == 0);
        }
        span = span_of<C>(a, s, rb);
        return true;
    }
    // keys that every row of the block sees: [lo, hi)
    __device__ __forceinline__ void seen_by_all(const AttnArgs &a, int &lo, int &hi) const
    {
        const int rows = s.n * a.G;
        const int r1 = (rb + 1) * C::R < rows ? (rb + 1) * C::R : rows;
        const int i0 = rb ? rb * C::R / a.G : 0, i1 = r1 == rows ? s.n - 1 : (r1 - 1) / a.G;
        hi = a.causal ? s.kv - s.n + i0 + 1 : s.kv;
        const long long from = static_cast<long long>(s.kv) - s.n + i1 - a.window;
        lo = a.window >= 0 && from > 0 ? static_cast<int>(from) : 0;
    }
};

struct LineShared {
    int scan[32], at, b, rb, kv, n;
};

// Lays out the line and finds this CTA's range of it, [first, end), and the unit it
// begins with; all C::T threads call it.  False: nothing to do.  Uncut (cut false), a
// unit belongs whole to the range that its first tile lies in.
template <class C>
__device__ __forceinline__ bool find_range(const AttnArgs &a, bool cut, LineShared &sh, Range &range, int &first, int &end,
                                           Line<C> &line)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // A thread takes a run of the row blocks (as many a sequence as Lq can have), and the
    // one whose run holds the first tile finds its unit.
    const int blocks = (a.Lq * a.G + C::R - 1) / C::R, items = a.c.B * blocks;
    const int per = items <= C::T ? 1 : (items + C::T - 1) / C::T;
    const int i0 = tid * per, i1 = i0 + per < items ? i0 + per : items;
    const int b0 = blocks == 1 ? i0 : i0 / blocks, rb0 = i0 - b0 * blocks;
    Seq s{0, 0};
    int length = 0;                     // of the block's units on the line, all heads'
    auto item = [&](int b, int rb, bool read) {
        if (read)
            s = sequence(a, b);
        length = rb * C::R < s.n * a.G ? (span_of<C>(a, s, rb).tiles + C::UNIT_COST) * a.c.H : 0;
    };
    int mine = 0;
    {
        int b = b0, rb = rb0;
        for (int i = i0; i < i1; ++i) {
            item(b, rb, i == i0 || rb == 0);
            mine += length;
            if (++rb == blocks) {
                rb = 0;
                ++b;
            }
        }
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, d);
        upto += lane >= d ? x : 0;
    }
    if (lane == 31)
        sh.scan[warp] = upto;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < C::T / 32; ++w) {
        before += w < warp ? sh.scan[w] : 0;
        total += sh.scan[w];
    }
    before += upto - mine;
    if (total == 0)
        return false;
    const int most = cut ? (total + C::MIN_TILES - 1) / C::MIN_TILES : total;
    range = Range(total, most < static_cast<int>(gridDim.x) ? most : static_cast<int>(gridDim.x));
    const int cta = blockIdx.x;
    if (cta >= range.grid)
        return false;
    first = range.begin(cta);
    end = range.begin(cta + 1);
    if (first >= before && first < before + mine) {
        int b = b0, rb = rb0, at = before;
        if (per > 1) {
            item(b, rb, true);
            while (first >= at + length) {
                at += length;
                if (++rb == blocks) {
                    rb = 0;
                    ++b;
                }
                item(b, rb, rb == 0);
            }
        }
        sh.at = at;
        sh.b = b;
        sh.rb = rb;
        sh.kv = s.kv;
        sh.n = s.n;
    }
    __syncthreads();
    line.b = sh.b;
    line.rb = sh.rb;
    line.s = Seq{sh.kv, sh.n};
    line.span = span_of<C>(a, line.s, line.rb);
    const int unit = line.span.tiles + C::UNIT_COST;
    line.h = (first - sh.at) / unit;
    line.at = sh.at + line.h * unit;
    // (the range may begin in a unit's extra length: then with the next unit)
    if ((line.at + line.span.tiles <= first || (!cut && line.at < first)) && !line.next(a, end))
        return false;
    return line.at < end;
}

// m + t as two floats that hold more of it than one.  A part counts by a power of its
// log2-sum-exp2, so where scores are large, 10^5 say, the last place of one float, 2^-7, would
// be half a percent of its weight.
__device__ __forceinline__ float2 two_floats(float m, float t)
{
    const float sum = m + t;
    return make_float2(sum, t - (sum - m));
}

// Merges what ranges c0 .. c1 computed of N quadruples of one row of a unit, always in that
// order: place(k) is quadruple k's offset in a slot.  Returns the row's log2-sum-exp2.  (One
// pass, W parts at a time: the loads of a thread's quadruples are under way together, where
// a pass for the maximum and one a quadruple waited for one load after the other.  Ragged
// prompts merged in 13 us that way.  W = 4 where registers allow it: two contexts over all SMs
// 84.2 us, by two parts 85.7.)
template <class C, int N, int W, class P>
__device__ __forceinline__ float merge_row(const Parts &parts, int c0, int c1, int row, P place, float4 (&v)[N])
{
    const size_t slot_floats = Parts::slot_floats(C::R, C::D);
    auto slot = [&](int c) { return parts.data + (2 * static_cast<size_t>(c) + (c == c0 ? 1 : 0)) * slot_floats; };
    float top = -INFINITY, l = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k)
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int c = c0; c <= c1; c += W) {
        float2 lse[W];
        float4 x[W][N];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const bool there = c + i <= c1;
            const float *const s = slot(c + i);
            lse[i] = there ? __ldcg(reinterpret_cast<const float2 *>(s + C::R * C::D) + row) : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int k = 0; k < N; ++k)
                x[i][k] = there ? __ldcg(reinterpret_cast<const float4 *>(s + place(k))) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float before = top;
#pragma unroll
        for (int i = 0; i < W; ++i)
            top = fmaxf(top, lse[i].x);
        const float ref = top == -INFINITY ? 0.f : top, f = ptx::ex2_approx(before - ref);
        l *= f;
#pragma unroll
        for (int k = 0; k < N; ++k)
            v[k].x *= f, v[k].y *= f, v[k].z *= f, v[k].w *= f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float g = ptx::ex2_approx(lse[i].x - ref + lse[i].y);
            l += g;
#pragma unroll
            for (int k = 0; k < N; ++k)
                v[k].x += x[i][k].x * g, v[k].y += x[i][k].y * g, v[k].z += x[i][k].z * g, v[k].w += x[i][k].w * g;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int k = 0; k < N; ++k)
        v[k].x *= inv, v[k].y *= inv, v[k].z *= inv, v[k].w *= inv;
    return l == 0.f ? -INFINITY : top + ptx::lg2_approx(l);
}
#endif

}  // namespace cache
}  // namespace fa2
