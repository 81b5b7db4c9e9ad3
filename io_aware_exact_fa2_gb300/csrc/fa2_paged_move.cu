// fa2_paged_move.cu -- fa2_rope and fa2_paged_append: 16-bit rows turned by their positions on
// the way from one place to another.  Both only move bytes (4 a number: 2 in, 2 out; three
// operations a turned number), so they are one kernel over rows of up to three kinds (append:
// keys, values and queries in one launch).
//
// A thread has the same 16 numbers, eight pairs, of the same token in up to HEADS heads: two
// 16-byte pieces a head, and one load of cos and sin for them all (64 bytes, which would be as
// much as a head's own traffic).  Pairs (j, R + j) are eight numbers at 8 c and eight at R + 8 c,
// so no pair is split between threads, and rows may be turned in place.
//
// Measured (several inputs in turn, so that none is in L2; in a graph, and as calls one after the
// other): queries and keys of a training batch, 4 x 8192 tokens, 32 and 8 heads of 128, 675 MB in 101 us
// (103), 6.7 TB/s; eight prompts of up to 4096 tokens appended, 607 MB in 89 to 92 us (94), 6.6 to 6.8
// TB/s: 97 to 100 % of the measured copy rate (calls: 97 and 95).  Short calls are a launch and three
// ways to memory, counts, page and rows: 2.6 to 2.8 us (4.1) for 3 x 333 tokens.
#include <climits>

#include "fa2_paged.cuh"
#include "sm103_ptx.cuh"

namespace fa2 {
namespace paged {

namespace {

constexpr int THREADS = 128;
constexpr int BATCH = 4;      // heads whose loads are under way together
// Heads of one kind a block, so many share a load of cos and sin, and fewer where there would be
// fewer than BLOCKS blocks an SM: one token of 128 sequences, 48 heads of 128 in all, 3.4 us,
// 4.7 with 8.  (More a block or less, in large calls: 8 prompts' append 89.0 us, 95 with 16, 97 with 4;
// 16 instead of 4 blocks an SM: a gradient of 3 x 501 tokens 8.8 us for 7.0.)
constexpr int HEADS = 8, BLOCKS = 4;

// (x, y) by (c, s): (x c - y s, x s + y c)
__device__ __forceinline__ void turn(float &x, float &y, float c, float s)
{
    const float z = fmaf(x, c, -y * s);
    y = fmaf(x, s, y * c);
    x = z;
}

// Eight pairs in two pieces: word k of `a` and of `b` hold pairs 2 k and 2 k + 1, or
// (interleaved) each word of a, then of b, is a pair.
template <bool F16>
__device__ __forceinline__ void turn8(uint4 &a, uint4 &b, const float (&c)[8], const float (&s)[8], bool interleaved)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (interleaved) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float x, y;
            unpack2<F16>(w[k], x, y);
            turn(x, y, c[k], s[k]);
            w[k] = pack2<F16>(x, y);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float x0, x1, y0, y1;
            unpack2<F16>(w[k], x0, x1);
            unpack2<F16>(w[k + 4], y0, y1);
            turn(x0, y0, c[2 * k], s[2 * k]);
            turn(x1, y1, c[2 * k + 1], s[2 * k + 1]);
            w[k] = pack2<F16>(x0, x1);
            w[k + 4] = pack2<F16>(y0, y1);
        }
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
}

template <bool F16>
__global__ void __launch_bounds__(THREADS) move_kernel(const MoveArgs a, const int groups, const int heads, const int lpr_shift)
{
    // block -> (tokens, group of heads), the latter fastest: a token's table rows are shared
    const unsigned tokens_at = blockIdx.x / groups;
    int group = blockIdx.x - tokens_at * groups, kind = 0;
    for (; kind < 2; ++kind) {
        const int n = (a.rows[kind].heads + heads - 1) / heads;
        if (group < n)
            break;
        group -= n;
    }
    const Rows &rows = a.rows[kind];
    const int chunk = threadIdx.x & ((1 << lpr_shift) - 1);
    const unsigned token = (tokens_at << (7 - lpr_shift)) + (threadIdx.x >> lpr_shift);
    if (token >= static_cast<unsigned>(a.B) * static_cast<unsigned>(a.L))
        return;
    const int b = token / static_cast<unsigned>(a.L), i = token - static_cast<unsigned>(b) * a.L;
    // (asked for together: each is a way to memory)
    const int n = a.counts ? a.counts[b] : a.L, start = a.starts ? a.starts[b] : 0;
    if (i >= n)
        return;
    const long long pos = start + static_cast<long long>(i);

    // the two pieces
    const bool turned = rows.rotated && chunk * 8 < a.r.R, neighbours = !turned || a.r.interleaved;
    const int at0 = neighbours ? chunk * 16 : chunk * 8, at1 = neighbours ? at0 + 8 : a.r.R + at0;
    const int h0 = group * heads, h1 = h0 + heads < rows.heads ? h0 + heads : rows.heads;
    const uint16_t *const x = rows.x + b * rows.sb + i * rows.sl;
    uint4 u[BATCH], w[BATCH];
    auto load = [&](int h) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (h + k < h1) {
                const uint16_t *from = x + (h + k) * rows.sh;
                u[k] = *reinterpret_cast<const uint4 *>(from + at0);
                w[k] = *reinterpret_cast<const uint4 *>(from + at1);
            }
    };
    // the pairs' cos and sin
    float c[8], s[8];
    if (turned) {
        const long long p = pos < 0 ? 0 : pos < a.r.positions ? pos : a.r.positions - 1;
        const float4 *cs = reinterpret_cast<const float4 *>(a.r.cos + p * a.r.R + chunk * 8);
        const float4 *sn = reinterpret_cast<const float4 *>(a.r.sin + p * a.r.R + chunk * 8);
        const float4 c0 = __ldg(cs), c1 = __ldg(cs + 1), s0 = __ldg(sn), s1 = __ldg(sn + 1);
        const float sense = a.r.inverse ? -1.f : 1.f;
        c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
        s[0] = s0.x * sense, s[1] = s0.y * sense, s[2] = s0.z * sense, s[3] = s0.w * sense;
        s[4] = s1.x * sense, s[5] = s1.y * sense, s[6] = s1.z * sense, s[7] = s1.w * sense;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            c[k] = s[k] = 0.f;
    }
    uint16_t *out = rows.out;
    long long out_head = rows.out_sh;
    if (out) {
        out += b * rows.out_sb + i * rows.out_sl;
    } else {
        const View &v = a.c;
        if (pos < 0 || pos >= static_cast<long long>(v.max_pages) << v.page_shift)
            return;
        const int id = cache::page_of(v, b, static_cast<int>(pos >> v.page_shift));
        if (id < 0)
            return;
        const Half &half = rows.side ? v.v : v.k;
        const int slot = static_cast<int>(pos) & ((1 << v.page_shift) - 1);
        out = reinterpret_cast<uint16_t *>(half.codes + id * half.s_page + slot * half.s_slot);
        out_head = half.s_head / 2;
    }
    load(h0);
#pragma unroll 1
    for (int h = h0;;) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (h + k < h1) {
                if (turned)
                    turn8<F16>(u[k], w[k], c, s, a.r.interleaved);
                uint16_t *to = out + (h + k) * out_head;
                *reinterpret_cast<uint4 *>(to + at0) = u[k];
                *reinterpret_cast<uint4 *>(to + at1) = w[k];
            }
        h += BATCH;
        if (h >= h1)
            break;
        load(h);
    }
}

int lpr_shift_of(int D) { return D == 64 ? 2 : D == 128 ? 3 : 4; }   // threads a row, 16 numbers each

long long groups_of(const MoveArgs &a, int heads)
{
    long long n = 0;
    for (int k = 0; k < a.kinds; ++k)
        n += (static_cast<long long>(a.rows[k].heads) + heads - 1) / heads;
    return n;
}

// Blocks of tokens.
long long tokens_of(const MoveArgs &a)
{
    const int per = THREADS >> lpr_shift_of(a.D);
    return (static_cast<long long>(a.B) * a.L + per - 1) / per;   // (below 2^62)
}

}  // namespace

long long move_blocks(const MoveArgs &a)
{
    if (static_cast<long long>(a.B) * a.L > INT_MAX || groups_of(a, HEADS) > INT_MAX / tokens_of(a))
        return 1ll << 40;
    return tokens_of(a) * groups_of(a, HEADS);
}

fa2_status launch_move(const MoveArgs &a, bool f16, int num_sms, cudaStream_t stream)
{
    const long long tokens = tokens_of(a), wanted = static_cast<long long>(BLOCKS) * num_sms;
    int heads = HEADS;
    while (heads > 1 && tokens * groups_of(a, heads) < wanted)
        heads /= 2;
    const int blocks = static_cast<int>(tokens * groups_of(a, heads)), groups = static_cast<int>(groups_of(a, heads));
    if (f16)
        move_kernel<true><<<blocks, THREADS, 0, stream>>>(a, groups, heads, lpr_shift_of(a.D));
    else
        move_kernel<false><<<blocks, THREADS, 0, stream>>>(a, groups, heads, lpr_shift_of(a.D));
    return cudaGetLastError() == cudaSuccess ? FA2_OK : FA2_ERR_CUDA;
}

}  // namespace paged
}  // namespace fa2
