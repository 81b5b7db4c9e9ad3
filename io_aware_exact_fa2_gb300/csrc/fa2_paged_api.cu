// fa2_paged_api.cu -- the C ABI declared in include/fa2_paged.h: argument checks, device
// selection, dispatch.
#include <climits>
#include <cmath>
#include <mutex>

#include "fa2_cache_host.h"
#include "fa2_paged.cuh"

#define FA2_EXPORT extern "C" __attribute__((visibility("default")))

namespace fa2 {
namespace paged {

using cache::aligned;
using cache::Device;
using cache::kMaxLength;
using cache::kMaxStride;
using cache::row_strides;

// Written by a kernel when one of its bounded waits runs out (first code wins).
static __device__ int g_paged_error;

namespace {

// Device address of g_paged_error on `dev`, which must be current (looked up once per device).
int *device_error_ptr(int dev)
{
    static std::mutex mu;
    static int *found[kMaxDevices] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < kMaxDevices && found[dev])
        return found[dev];
    void *ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, g_paged_error) != cudaSuccess) {
        (void)cudaGetLastError();
        return nullptr;
    }
    if (dev >= 0 && dev < kMaxDevices)
        found[dev] = static_cast<int *>(ptr);
    return static_cast<int *>(ptr);
}

bool type_ok(int dtype) { return dtype == FA2_BF16 || dtype == FA2_FP16; }

// (strides in bytes, as the kernels take them)
bool half_view(Half &x, void *data, const long long (&strides)[3], const fa2_paged *c)
{
    if (!data || !aligned(data, 16))
        return false;
    x.codes = static_cast<uint8_t *>(data);
    x.scale = nullptr;
    if (strides[0] == 0 && strides[1] == 0 && strides[2] == 0) {
        x.s_slot = 2ll * c->D;
        x.s_head = c->page_size * x.s_slot;
        x.s_page = x.s_head * c->H;
        return true;
    }
    for (long long s : strides)
        if (s <= 0 || s % 8 != 0 || s > kMaxStride)
            return false;
    x.s_page = 2 * strides[0];
    x.s_head = 2 * strides[1];
    x.s_slot = 2 * strides[2];
    return true;
}

// The cache as the kernels see it; host-side checks only.
fa2_status view_of(const fa2_paged *c, View &v)
{
    if (!c || c->B <= 0 || c->H <= 0 || c->num_pages <= 0 || c->max_pages <= 0 || c->D <= 0 || c->page_size <= 0)
        return FA2_ERR_INVALID_ARG;
    if (!half_view(v.k, c->k, c->k_strides, c) || !half_view(v.v, c->v, c->v_strides, c))
        return FA2_ERR_INVALID_ARG;
    if (!c->page_table || !aligned(c->page_table, 4))
        return FA2_ERR_INVALID_ARG;
    if (static_cast<long long>(c->B) * c->H > INT_MAX || static_cast<long long>(c->max_pages) * c->page_size > kMaxLength)
        return FA2_ERR_INVALID_ARG;
    switch (c->page_size) {
    case 16: v.page_shift = 4; break;
    case 32: v.page_shift = 5; break;
    case 64: v.page_shift = 6; break;
    case 128: v.page_shift = 7; break;
    default: return FA2_ERR_UNSUPPORTED;
    }
    if ((c->D != 64 && c->D != 128 && c->D != 256) || !type_ok(c->dtype))
        return FA2_ERR_UNSUPPORTED;
    v.table = c->page_table;
    v.num_pages = c->num_pages;
    v.H = c->H;
    v.B = c->B;
    v.max_pages = c->max_pages;
    return FA2_OK;
}

bool rotation_of(const fa2_rotation *r, int D, bool inverse, Rotation &out)
{
    if (!r->cos || !r->sin || !aligned(r->cos, 16) || !aligned(r->sin, 16) || r->positions <= 0 || r->positions > kMaxLength ||
        r->R <= 0 || r->R % 8 != 0 || 2ll * r->R > D)
        return false;
    out = Rotation{r->cos, r->sin, r->positions, r->R, r->interleaved != 0, inverse};
    return true;
}

// `heads` rows [B, heads, L, D] from x to out (null: the cache); false if the arguments do not fit.
bool rows_of(Rows &rows, const void *x, const long long *strides, void *out, const long long *out_strides, bool into_cache,
             int heads, int L, int D)
{
    if (!x || !aligned(x, 16) || !row_strides(strides, heads, L, D, rows.sb, rows.sh, rows.sl))
        return false;
    if (!into_cache && (!out || !aligned(out, 16) || !row_strides(out_strides, heads, L, D, rows.out_sb, rows.out_sh, rows.out_sl)))
        return false;
    rows.x = static_cast<const uint16_t *>(x);
    rows.out = into_cache ? nullptr : static_cast<uint16_t *>(out);
    rows.heads = heads;
    rows.rotated = rows.side = 0;
    return true;
}

fa2_status move(MoveArgs &a, bool f16, const void *owner, void *stream)
{
    if (a.L == 0)
        return FA2_OK;
    if (move_blocks(a) > INT_MAX)
        return FA2_ERR_UNSUPPORTED;
    const Device dev(owner);
    if (dev.status() != FA2_OK)
        return dev.status();
    const int sms = fa2::sm_count(dev.id());
    if (sms <= 0)
        return FA2_ERR_CUDA;
    return launch_move(a, f16, sms, static_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace paged
}  // namespace fa2

FA2_EXPORT fa2_status fa2_rope(const void *q, const void *k, void *q_out, void *k_out, const long long *q_strides,
                               const long long *k_strides, const long long *q_out_strides, const long long *k_out_strides,
                               const int *starts, const fa2_rotation *r, int B, int Hq, int H, int L, int D, int dtype,
                               int inverse, void *stream)
{
    using namespace fa2::paged;
    MoveArgs a = {};
    if (B <= 0 || Hq <= 0 || H < 0 || L < 0 || L > kMaxLength || D <= 0 || static_cast<long long>(B) * Hq > INT_MAX ||
        static_cast<long long>(B) * H > INT_MAX || !aligned(starts, 4) || !r)
        return FA2_ERR_INVALID_ARG;
    if ((D != 64 && D != 128 && D != 256) || !type_ok(dtype))
        return FA2_ERR_UNSUPPORTED;
    if (!rotation_of(r, D, inverse != 0, a.r) || !rows_of(a.rows[0], q, q_strides, q_out, q_out_strides, false, Hq, L, D))
        return FA2_ERR_INVALID_ARG;
    a.kinds = 1;
    if (H > 0) {
        if (!rows_of(a.rows[1], k, k_strides, k_out, k_out_strides, false, H, L, D))
            return FA2_ERR_INVALID_ARG;
        a.kinds = 2;
    } else if (k || k_out) {
        return FA2_ERR_INVALID_ARG;
    }
    a.rows[0].rotated = a.rows[1].rotated = 1;
    a.starts = starts;
    a.B = B;
    a.L = L;
    a.D = D;
    return move(a, dtype == FA2_FP16, q, stream);
}

FA2_EXPORT fa2_status fa2_paged_append(const fa2_paged *c, const void *k, const void *v, const long long *k_strides,
                                       const long long *v_strides, const int *starts, const int *counts,
                                       const fa2_rotation *r, const void *q, void *q_out, const long long *q_strides,
                                       const long long *q_out_strides, int Hq, int L, void *stream)
{
    using namespace fa2::paged;
    MoveArgs a = {};
    const fa2_status st = view_of(c, a.c);
    if (st != FA2_OK)
        return st;
    if (!starts || !aligned(starts, 4) || !aligned(counts, 4) || L < 0 || L > kMaxLength || Hq < 0 ||
        static_cast<long long>(c->B) * Hq > INT_MAX)
        return FA2_ERR_INVALID_ARG;
    if (!rows_of(a.rows[0], k, k_strides, nullptr, nullptr, true, c->H, L, c->D) ||
        !rows_of(a.rows[1], v, v_strides, nullptr, nullptr, true, c->H, L, c->D))
        return FA2_ERR_INVALID_ARG;
    if (r && !rotation_of(r, c->D, false, a.r))
        return FA2_ERR_INVALID_ARG;
    a.rows[1].side = 1;
    a.rows[0].rotated = r != nullptr;
    a.kinds = 2;
    if (Hq > 0) {
        if (!r || !rows_of(a.rows[2], q, q_strides, q_out, q_out_strides, false, Hq, L, c->D))
            return FA2_ERR_INVALID_ARG;
        a.rows[2].rotated = 1;
        a.kinds = 3;
    } else if (q || q_out) {
        return FA2_ERR_INVALID_ARG;
    }
    a.starts = starts;
    a.counts = counts;
    a.B = c->B;
    a.L = L;
    a.D = c->D;
    return move(a, c->dtype == FA2_FP16, c->k, stream);
}

FA2_EXPORT fa2_status fa2_paged_attn(const fa2_paged *c, const void *q, void *o, float *lse, const long long *q_strides,
                                     const long long *o_strides, const int *kv_lens, const int *q_lens, int Hq, int Lq,
                                     int causal, int window, float scale, void *workspace, size_t workspace_bytes,
                                     void *stream)
{
    using namespace fa2::paged;
    AttnArgs a;
    const fa2_status st = view_of(c, a.c);
    if (st != FA2_OK)
        return st;
    if (!q || !o || !lse || !kv_lens || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(kv_lens, 4) ||
        !aligned(q_lens, 4))
        return FA2_ERR_INVALID_ARG;
    if (Hq <= 0 || Hq % c->H != 0 || Lq < 0 || static_cast<long long>(c->B) * Hq > INT_MAX ||
        static_cast<long long>(Lq) * (Hq / c->H) > kMaxLength)
        return FA2_ERR_INVALID_ARG;
    if (!std::isfinite(scale * 1.4426950408889634f) || !(scale > 0.f) || window < -1 || (window >= 0 && !causal))
        return FA2_ERR_INVALID_ARG;
    if (!row_strides(q_strides, Hq, Lq, c->D, a.q_sb, a.q_sh, a.q_sl) ||
        !row_strides(o_strides, Hq, Lq, c->D, a.o_sb, a.o_sh, a.o_sl))
        return FA2_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 256))
        return FA2_ERR_INVALID_ARG;
    if (Lq == 0)
        return FA2_OK;
    a.q = q;
    a.o = o;
    a.lse = lse;
    a.kv_lens = kv_lens;
    a.q_lens = q_lens;
    a.Hq = Hq;
    a.Lq = Lq;
    a.D = c->D;
    a.G = Hq / c->H;
    a.causal = causal ? 1 : 0;
    a.window = window;
    a.scale = scale;
    a.workspace = workspace;
    a.workspace_bytes = workspace_bytes;
    a.stream = static_cast<cudaStream_t>(stream);
    const Device dev(c->k);
    if (dev.status() != FA2_OK)
        return dev.status();
    a.num_sms = fa2::sm_count(dev.id());
    a.err = device_error_ptr(dev.id());
    a.naps = fa2::cache::test_naps();
    a.drain_limit_ns = fa2::wait_limit_ns();
    a.wait_limit_ns = fa2::call_wait_limit_ns();
    if (a.num_sms <= 0 || !a.err)
        return FA2_ERR_CUDA;
    const bool f16 = c->dtype == FA2_FP16;
    return c->D == 64 ? launch_attn<64>(a, f16) : c->D == 128 ? launch_attn<128>(a, f16) : launch_attn<256>(a, f16);
}

FA2_EXPORT fa2_status fa2_paged_attn_workspace_size(int B, int Hq, int H, int Lq, int D, int device, size_t *bytes)
{
    using namespace fa2::paged;
    if (!bytes)
        return FA2_ERR_INVALID_ARG;
    *bytes = 0;
    if (B <= 0 || H <= 0 || Hq <= 0 || Hq % H != 0 || Lq < 0 || D <= 0 || device < 0 ||
        static_cast<long long>(B) * Hq > INT_MAX || static_cast<long long>(Lq) * (Hq / H) > kMaxLength)
        return FA2_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256)
        return FA2_ERR_UNSUPPORTED;
    if (Lq == 0)
        return FA2_OK;
    const int sms = fa2::sm_count(device);
    if (sms <= 0)
        return FA2_ERR_CUDA;
    const long long rows = static_cast<long long>(Lq) * (Hq / H);
    *bytes = D == 64    ? attn_workspace_bytes<64>(rows, sms)
             : D == 128 ? attn_workspace_bytes<128>(rows, sms)
                        : attn_workspace_bytes<256>(rows, sms);
    return FA2_OK;
}

FA2_EXPORT fa2_status fa2_paged_get_device_error(void *stream, int *detail)
{
    if (detail)
        *detail = 0;
    int v = 0;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess ||
        cudaMemcpyFromSymbol(&v, fa2::paged::g_paged_error, sizeof v) != cudaSuccess) {
        (void)cudaGetLastError();
        return FA2_ERR_CUDA;
    }
    if (v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(fa2::paged::g_paged_error, &zero, sizeof zero) != cudaSuccess) {
            (void)cudaGetLastError();
            return FA2_ERR_CUDA;
        }
    }
    if (detail)
        *detail = v;
    return v ? FA2_ERR_TIMEOUT : FA2_OK;
}
