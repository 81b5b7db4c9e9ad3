// fa2_cache_move.cu -- fa2_cache_write and fa2_cache_read: bf16 rows into and out of
// the paged e4m3 cache.  Both only move bytes (3 per value: 2 bf16, 1 code); a code
// and its scale determine the value exactly, so nothing here rounds but the one
// conversion to e4m3.  Measured (three inputs in turn): eight prompts of up to 8192 rows, 8
// heads of 128, 302 MB in 48 us, 6.3 TB/s; four contexts of 16384, 16 heads of 128, 805 MB
// out in 124.5 us, 6.5 TB/s: 93 and 95 % of the measured copy rate.  One row a sequence (128
// of them, part of a page each) and short prefixes are launches: 2.7 and 2.9 us.
#include <climits>

#include "fa2_cache.cuh"
#include "sm103_ptx.cuh"

namespace fa2 {
namespace cache {

namespace {

// Sixteen bf16 of a row, as eight packed words.
struct Row16 {
    uint32_t w[8];
};

__device__ __forceinline__ void load16(Row16 &r, const uint16_t *p)
{
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p)), b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
    r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
}

// Largest magnitudes of two packed bf16 (a NaN only where there is nothing else).
__device__ __forceinline__ uint32_t packed_max(uint32_t m, uint32_t w)
{
    asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w & 0x7fff7fffu));
    return m;
}

// Largest finite magnitude among two packed bf16, as bf16 bits (magnitudes of bf16
// order as their bits do).
__device__ __forceinline__ uint32_t finite_max(uint32_t m, uint32_t w)
{
    const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
    m = lo < 0x7f80u && lo > m ? lo : m;
    return hi < 0x7f80u && hi > m ? hi : m;
}

// Least e >= kMinExponent with a <= 448 * 2^e, at most kMaxExponent; a given as bf16
// bits.  448 = 1.75 * 2^8, so with a = f * 2^E (1 <= f < 2) it is E - 8, and one more
// where f > 1.75 (fraction bits above 0x60).  Zeros and subnormals come out below the
// least exponent.
__device__ __forceinline__ int least_exponent(uint32_t a)
{
    const int e = static_cast<int>(a >> 7) - 127 - 8 + ((a & 0x7fu) > 0x60u ? 1 : 0);
    return e < kMinExponent ? kMinExponent : e > kMaxExponent ? kMaxExponent : e;
}

// x * inv; with INF, infinities as NaN: the saturating conversion below would make them 448.
template <bool INF>
__device__ __forceinline__ float scaled(float x, float inv)
{
    return INF ? fmaf(x, inv, x * 0.f) : x * inv;
}

template <bool INF>
__device__ __forceinline__ uint32_t quantise4(uint32_t a, uint32_t b, float inv)
{
    return ptx::pack_e4m3x4(scaled<INF>(__uint_as_float(a << 16), inv), scaled<INF>(__uint_as_float(a & 0xffff0000u), inv),
                            scaled<INF>(__uint_as_float(b << 16), inv), scaled<INF>(__uint_as_float(b & 0xffff0000u), inv));
}

template <bool INF>
__device__ __forceinline__ uint4 quantise16(const Row16 &r, float inv)
{
    return make_uint4(quantise4<INF>(r.w[0], r.w[1], inv), quantise4<INF>(r.w[2], r.w[3], inv),
                      quantise4<INF>(r.w[4], r.w[5], inv), quantise4<INF>(r.w[6], r.w[7], inv));
}

// Four codes brought from one scale to a larger one (f = 2^(before - after)).
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f)
{
    float a, b, c, d;
    unpack_f16x2(e4m3x2_to_f16x2(w), a, b);
    unpack_f16x2(e4m3x2_hi_to_f16x2(w), c, d);
    return ptx::pack_e4m3x4(a * f, b * f, c * f, d * f);
}

// One block quantises one page's new rows of one head, keys or values: the page's
// scale needs the largest magnitude of them all, so they are read once into registers
// (NP rows a thread, 16 values of each), reduced, and written out as codes.  (The arithmetic
// shows: with a magnitude compared and a code converted at a time 302 MB took 16 % more.)
template <int T, int NP>
__global__ void __launch_bounds__(T) write_kernel(const MoveArgs a, const int touched, const int lpr_shift)
{
    const View &c = a.c;
    // block -> (sequence, touched page, head, keys or values), the last fastest: blocks
    // that run together read neighbouring heads' rows
    unsigned idx = blockIdx.x;
    const int side = idx & 1;
    idx >>= 1;
    const int h = idx % c.H;
    idx /= c.H;
    const int j = idx % touched, b = idx / touched;

    const long long start = a.starts[b];
    int n = a.counts ? a.counts[b] : a.L;
    n = n < 0 ? 0 : n > a.L ? a.L : n;
    const long long cap = static_cast<long long>(c.max_pages) << c.page_shift;
    const long long lo = start > 0 ? start : 0, hi = start + n < cap ? start + n : cap;
    const long long page = (lo >> c.page_shift) + j;
    const long long p0 = page << c.page_shift;
    if (p0 >= hi || lo >= hi)
        return;
    const int page_size = 1 << c.page_shift;
    const int s0 = lo > p0 ? static_cast<int>(lo - p0) : 0;                       // first slot written
    const int s1 = hi - p0 < page_size ? static_cast<int>(hi - p0) : page_size;   // end of those written
    const int id = page_of(c, b, static_cast<int>(page));
    if (id < 0)
        return;

    const Half &half = side ? c.v : c.k;
    const int lpr = 1 << lpr_shift;                     // threads a row, 16 values each
    const int col = (threadIdx.x & (lpr - 1)) * 16, row0 = threadIdx.x >> lpr_shift, step = T >> lpr_shift;
    const uint16_t *x = static_cast<const uint16_t *>(a.x[side]) + b * a.sb[side] + h * a.sh[side] + col;
    uint8_t *codes = half.codes + id * half.s_page + h * half.s_head + col;
    uint8_t *scale = half.scale + static_cast<long long>(id) * c.H + h;

    Row16 r[NP];
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int s = s0 + row0 + k * step;
        if (s < s1)
            load16(r[k], x + (p0 + s - start) * a.sl[side]);
    }
    const int before = s0 > 0 ? static_cast<int>(*scale) - 127 : INT_MIN;
    // The arithmetic counts here: the plain maximum, and only where it is no finite number
    // (an infinity among them, or nothing but NaN) that of the finite ones.
    uint32_t pair = 0;
#pragma unroll
    for (int k = 0; k < NP; ++k)
        if (s0 + row0 + k * step < s1)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                pair = packed_max(pair, r[k].w[i]);
    m = max(pair & 0xffffu, pair >> 16);
    const bool odd = m >= 0x7f80u;
    if (odd) {
        m = 0;
#pragma unroll
        for (int k = 0; k < NP; ++k)
            if (s0 + row0 + k * step < s1)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    m = finite_max(m, r[k].w[i]);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (T > 32) {
        __shared__ uint32_t part[T / 32];
        if ((threadIdx.x & 31) == 0)
            part[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < T / 32; ++w)
            m = part[w] > m ? part[w] : m;
    }
    int e = least_exponent(m);
    e = before > e ? before : e;
    const float inv = pow2i(-e);
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int s = s0 + row0 + k * step;
        if (s < s1) {
            *reinterpret_cast<uint4 *>(codes + s * half.s_slot) = odd ? quantise16<true>(r[k], inv) : quantise16<false>(r[k], inv);
        }
    }
    if (s0 > 0 && e > before) {
        const float f = pow2i(before - e);
        for (int s = row0; s < s0; s += step) {
            uint4 *p = reinterpret_cast<uint4 *>(codes + s * half.s_slot);
            uint4 w = *p;
            w.x = rescale4(w.x, f);
            w.y = rescale4(w.y, f);
            w.z = rescale4(w.z, f);
            w.w = rescale4(w.w, f);
            *p = w;
        }
    }
    if (T == 32)
        __syncwarp();   // (wider blocks: the reduction's barrier) every thread has read the scale
    if (threadIdx.x == 0)
        *scale = static_cast<uint8_t>(e + 127);
}

template <int T, int NP>
fa2_status run_write(const MoveArgs &a, long long blocks, int touched, int lpr_shift, cudaStream_t stream)
{
    write_kernel<T, NP><<<static_cast<unsigned>(blocks), T, 0, stream>>>(a, touched, lpr_shift);
    return cudaGetLastError() == cudaSuccess ? FA2_OK : FA2_ERR_CUDA;
}

constexpr int READ_T = 256;      // threads a block
constexpr int READ_ROWS = 2;     // rows a thread (of 805 MB: 1 row 128 us, 2 122, 4 138, 8 171)

// A block copies READ_ROWS * 16 / D * READ_T rows of one head, keys or values.
__global__ void __launch_bounds__(READ_T) read_kernel(const MoveArgs a, const int chunks, const int lpr_shift)
{
    const View &c = a.c;
    unsigned idx = blockIdx.x;
    const int chunk = idx % chunks;
    idx /= chunks;
    const int side = idx & 1;
    idx >>= 1;
    const int h = idx % c.H, b = idx / c.H;
    const int lpr = 1 << lpr_shift, col = (threadIdx.x & (lpr - 1)) * 16, step = READ_T >> lpr_shift;
    const int row0 = chunk * step * READ_ROWS + (threadIdx.x >> lpr_shift);
    int n = a.counts ? a.counts[b] : a.L;
    n = n > a.L ? a.L : n;
    if (row0 >= n)
        return;
    const long long start = a.starts[b];
    const Half &half = side ? c.v : c.k;
    const long long cap = static_cast<long long>(c.max_pages) << c.page_shift;

    uint4 w[READ_ROWS];
    float f[READ_ROWS];
#pragma unroll
    for (int k = 0; k < READ_ROWS; ++k) {
        const int i = row0 + k * step;
        const long long p = start + i;
        w[k] = make_uint4(0, 0, 0, 0);
        f[k] = 0.f;
        if (i < n && p >= 0 && p < cap) {
            const int id = page_of(c, b, static_cast<int>(p >> c.page_shift));
            if (id >= 0) {
                const int slot = static_cast<int>(p) & ((1 << c.page_shift) - 1);
                w[k] = __ldg(reinterpret_cast<const uint4 *>(half.codes + id * half.s_page + h * half.s_head +
                                                             slot * half.s_slot + col));
                f[k] = e8m0(half.scale[static_cast<long long>(id) * c.H + h]);
            }
        }
    }
    uint16_t *x = static_cast<uint16_t *>(a.x[side]) + b * a.sb[side] + h * a.sh[side] + col;
#pragma unroll
    for (int k = 0; k < READ_ROWS; ++k) {
        const int i = row0 + k * step;
        if (i >= n)
            break;
        uint32_t out[8];
        const uint32_t in[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v0, v1, v2, v3;
            unpack_f16x2(e4m3x2_to_f16x2(in[q]), v0, v1);
            unpack_f16x2(e4m3x2_hi_to_f16x2(in[q]), v2, v3);
            out[2 * q] = ptx::pack_bf16x2(v0 * f[k], v1 * f[k]);
            out[2 * q + 1] = ptx::pack_bf16x2(v2 * f[k], v3 * f[k]);
        }
        uint4 *p = reinterpret_cast<uint4 *>(x + i * a.sl[side]);
        p[0] = make_uint4(out[0], out[1], out[2], out[3]);
        p[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
}

// Threads a row, 16 values each, as a power of two.
int row_shift(int D) { return D == 64 ? 2 : D == 128 ? 3 : 4; }

// Pages that L rows can touch: one, and one more for every page_size rows after the first.
int touched_pages(const MoveArgs &a)
{
    const int page_size = 1 << a.c.page_shift;
    return static_cast<int>((static_cast<long long>(a.L) + page_size - 2) / page_size) + 1;
}

// Blocks that read L rows of a head.
int read_chunks(const MoveArgs &a)
{
    const int rows = (READ_T >> row_shift(a.D)) * READ_ROWS;
    return static_cast<int>((static_cast<long long>(a.L) + rows - 1) / rows);
}

}  // namespace

// (B H and what they are multiplied by are below 2^31 each)
long long write_blocks(const MoveArgs &a) { return 2 * (static_cast<long long>(a.c.B) * a.c.H * touched_pages(a)); }
long long read_blocks(const MoveArgs &a) { return 2 * (static_cast<long long>(a.c.B) * a.c.H * read_chunks(a)); }

fa2_status launch_write(const MoveArgs &a, cudaStream_t stream)
{
    const int page_size = 1 << a.c.page_shift;
    const int lpr_shift = row_shift(a.D), touched = touched_pages(a);
    const long long blocks = write_blocks(a);
    // A page's rows in pieces of 16 values, four a thread where there are enough: in flight
    // together they hide each other's latency, and short blocks the next one's.  (Half a
    // million rows of 64, 134 MB: pages of 64 41 us with one piece, 29 with four, 31 with
    // eight; 75 with 512 threads.)
    const int pieces = (a.L < page_size ? a.L : page_size) << lpr_shift;
    if (pieces <= 32)
        return run_write<32, 1>(a, blocks, touched, lpr_shift, stream);
    if (pieces <= 64)
        return run_write<32, 2>(a, blocks, touched, lpr_shift, stream);
    if (pieces <= 128)
        return run_write<32, 4>(a, blocks, touched, lpr_shift, stream);
    if (pieces <= 256)
        return run_write<64, 4>(a, blocks, touched, lpr_shift, stream);
    if (pieces <= 512)
        return run_write<128, 4>(a, blocks, touched, lpr_shift, stream);
    if (pieces <= 1024)
        return run_write<256, 4>(a, blocks, touched, lpr_shift, stream);
    return run_write<512, 4>(a, blocks, touched, lpr_shift, stream);
}

fa2_status launch_read(const MoveArgs &a, cudaStream_t stream)
{
    read_kernel<<<static_cast<unsigned>(read_blocks(a)), READ_T, 0, stream>>>(a, read_chunks(a), row_shift(a.D));
    return cudaGetLastError() == cudaSuccess ? FA2_OK : FA2_ERR_CUDA;
}

}  // namespace cache
}  // namespace fa2
