// fa2_paged_line.cuh -- how fa2_paged_attn's kernels share out their work: as in
// fa2_cache_line.cuh the keys of all sequences, heads and blocks of query rows lie on one line,
// cut into equal ranges, one a CTA; but here they are cut at grains, which may be shorter than a
// tile, and a grain takes as many places on the line as it costs.
//
// A grain is a page of keys, or C::GRAIN of smaller ones.  A unit (a block of C::R query rows of
// one sequence and key/value head) is the places of the grains that any of its rows sees,
// 2^C::weight_shift each, and C::COST more, for what it takes to begin and end one.  A grain belongs to the
// range that its first place lies in; a range that holds only a unit's last places has nothing
// to do with it.  No range is shorter than C::LEAST places (but a line that is), at least what a
// grain takes: so each range that ends inside a unit's grains, or between two that do, holds the
// first place of one of them.
//
// Of fa2_cache_line.cuh the sequences' lengths (Seq, sequence, row_blocks), the cut into ranges (Range),
// the workspace (Parts) and LineShared are taken as they are.  Span, Line, line_grid and find_range stand
// in both files, there in tiles, here in places and grains: what is mended in one is to be looked at
// in the other.
#pragma once

#include "fa2_cache_line.cuh"

namespace fa2 {
namespace paged {

template <class C>
__host__ __device__ constexpr int grain_shift(const cache::AttnArgs &a)
{
    return a.c.page_shift > C::GRAIN_SHIFT ? a.c.page_shift : C::GRAIN_SHIFT;
}

// CTAs to launch: no more than the longest sequences could make ranges for; 0 if the line
// could be longer than an int counts, with room for what is added to a place.
template <class C>
int line_grid(const cache::AttnArgs &a, bool cut)
{
    const long long most = a.num_sms * C::CTAS;
    const long long blocks = (static_cast<long long>(a.Lq) * a.G + C::R - 1) / C::R;
    const long long grains = (static_cast<long long>(a.c.max_pages) << a.c.page_shift >> grain_shift<C>(a)) + 2;
    const long long length = (grains << C::weight_shift(C::R, grain_shift<C>(a))) + C::COST;
    const long long units = static_cast<long long>(a.c.B) * a.c.H * blocks;   // (B H, blocks < 2^31)
    if (units > cache::MAX_LINE || units * length > cache::MAX_LINE)
        return 0;
    const long long grid = cut ? units * length / C::LEAST + 1 : units;
    return static_cast<int>(grid > most ? most : grid);
}

#ifdef __CUDACC__

// Keys that a block of query rows sees at all: [lo, hi), and the grains they span.
struct Span {
    int lo, hi, grains;
};

// The first and last token of a block of rows.  (A step has one block: no division is waited for.)
template <class C>
__device__ __forceinline__ void tokens_of(const cache::AttnArgs &a, const cache::Seq &s, int rb, int &i0, int &i1)
{
    const int rows = s.n * a.G;
    i0 = 0;
    i1 = s.n - 1;
    if (rows > C::R) {
        i0 = rb * C::R / a.G;
        if ((rb + 1) * C::R < rows)
            i1 = ((rb + 1) * C::R - 1) / a.G;
    }
}

template <class C>
__device__ __forceinline__ Span span_of(const cache::AttnArgs &a, const cache::Seq &s, int rb)
{
    int i0, i1;
    tokens_of<C>(a, s, rb, i0, i1);
    Span p;
    p.hi = a.causal ? s.kv - s.n + i1 + 1 : s.kv;
    p.hi = p.hi < 0 ? 0 : p.hi;
    p.lo = 0;
    if (a.window >= 0) {
        const long long lo = static_cast<long long>(s.kv) - s.n + i0 - a.window;
        p.lo = lo > 0 ? static_cast<int>(lo) : 0;
    }
    const int shift = grain_shift<C>(a);
    p.grains = p.hi > p.lo ? ((p.hi - 1) >> shift) - (p.lo >> shift) + 1 : 1;   // a unit that sees nothing still writes its rows
    return p;
}

// A unit's place on the line.
template <class C>
struct Line {
    int at;            // its first place
    int weight_shift;  // places of each of its grains: 2^this
    int b, h, rb;
    cache::Seq s;
    Span span;

    __device__ __forceinline__ int length() const { return (span.grains << weight_shift) + C::COST; }
    // its first grain that begins at place x or later
    __device__ __forceinline__ int grain_at(int x) const
    {
        const int t = x <= at ? 0 : (x - at + (1 << weight_shift) - 1) >> weight_shift;
        return t < span.grains ? t : span.grains;
    }
    // the place of its last grain
    __device__ __forceinline__ int last() const { return at + ((span.grains - 1) << weight_shift); }
    // The keys of the unit in [from, stop) that lie in the range [first, end), and the tiles they
    // make (uncut: all).
    __device__ __forceinline__ int piece(const cache::AttnArgs &a, bool cut, int first, int end, int &from, int &stop) const
    {
        const int shift = grain_shift<C>(a);
        const int g0 = cut ? grain_at(first) : 0, g1 = cut ? grain_at(end) : span.grains;
        from = ((span.lo >> shift) + g0) << shift;
        const int keys = (g1 - g0) << shift;
        stop = span.hi - from < keys ? span.hi : from + keys;
        return (keys + C::TILE - 1) / C::TILE;
    }
    __device__ __forceinline__ void lay(const cache::AttnArgs &a)
    {
        span = paged::span_of<C>(a, s, rb);
        weight_shift = C::weight_shift(s.n * a.G - rb * C::R, grain_shift<C>(a));
    }
    // The following unit; false if it begins at `end` or later, or nowhere.
    __device__ __forceinline__ bool next(const cache::AttnArgs &a, int end)
    {
        at += length();
        if (at >= end)
            return false;
        if (++h < a.c.H)
            return true;
        h = 0;
        if (++rb == cache::row_blocks<C>(a, s)) {
            rb = 0;
            do {
                if (++b == a.c.B)
                    return false;
                s = cache::sequence(a, b);
            } while (s.n == 0);
        }
        lay(a);
        return true;
    }
    // keys that every row of the block sees: [lo, hi)
    __device__ __forceinline__ void seen_by_all(const cache::AttnArgs &a, int &lo, int &hi) const
    {
        int i0, i1;
        tokens_of<C>(a, s, rb, i0, i1);
        hi = a.causal ? s.kv - s.n + i0 + 1 : s.kv;
        const long long from = static_cast<long long>(s.kv) - s.n + i1 - a.window;
        lo = a.window >= 0 && from > 0 ? static_cast<int>(from) : 0;
    }
};

// Lays out the line and finds this CTA's range of it, [first, end), and the unit it
// begins with; T threads call it, numbered `tid`, whom `sync` makes wait for one another.  False:
// nothing to do.  Uncut (cut false), a unit belongs whole to the range that its first place lies in.
template <class C, int T, class S>
__device__ __forceinline__ bool find_range(const cache::AttnArgs &a, bool cut, cache::LineShared &sh, cache::Range &range,
                                           int &first, int &end, Line<C> &line, int tid, S sync)
{
    const int warp = tid >> 5, lane = tid & 31;
    // A thread takes a run of the row blocks (as many a sequence as Lq can have), and the
    // one whose run holds the first place finds its unit.
    const int blocks = (a.Lq * a.G + C::R - 1) / C::R, items = a.c.B * blocks;
    const int per = items <= T ? 1 : (items + T - 1) / T;
    const int i0 = tid * per, i1 = i0 + per < items ? i0 + per : items;
    const int b0 = blocks == 1 ? i0 : i0 / blocks, rb0 = i0 - b0 * blocks;
    cache::Seq s{0, 0};
    int length = 0;                     // of the block's units on the line, all heads'
    auto item = [&](int b, int rb, bool read) {
        if (read)
            s = cache::sequence(a, b);
        const int rows = s.n * a.G - rb * C::R;
        const int shift = C::weight_shift(rows, grain_shift<C>(a));
        length = rows > 0 ? ((paged::span_of<C>(a, s, rb).grains << shift) + C::COST) * a.c.H : 0;
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
    sync();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) {
        before += w < warp ? sh.scan[w] : 0;
        total += sh.scan[w];
    }
    before += upto - mine;
    if (total == 0)
        return false;
    const int most = !cut ? total : total < C::LEAST ? 1 : total / C::LEAST;
    range = cache::Range(total, most < static_cast<int>(gridDim.x) ? most : static_cast<int>(gridDim.x));
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
    sync();
    line.b = sh.b;
    line.rb = sh.rb;
    line.s = cache::Seq{sh.kv, sh.n};
    line.lay(a);
    line.h = (first - sh.at) / line.length();
    line.at = sh.at + line.h * line.length();
    // (the range may begin behind a unit's last grain: then with the next unit)
    if ((line.grain_at(first) == line.span.grains || (!cut && line.at < first)) && !line.next(a, end))
        return false;
    return line.at < end;
}
#endif

}  // namespace paged
}  // namespace fa2
