// fa2_cache_api.cu -- the C ABI declared in include/fa2_cache.h: argument checks,
// device selection, dispatch.
#include <climits>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "fa2_cache_tile.cuh"
#include "fa2_host.h"

#define FA2_EXPORT extern "C" __attribute__((visibility("default")))

namespace fa2 {
namespace cache {

// Written by a kernel when one of its bounded waits runs out (first code wins).
static __device__ int g_cache_error;

EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

namespace {

constexpr long long kMaxStride = 1ll << 38;
constexpr long long kMaxLength = 1ll << 30;   // positions of a sequence, rows of a call

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Makes the device that owns `ptr` current, and the caller's current again at the end.
class Device {
public:
    explicit Device(const void *ptr)
    {
        cudaPointerAttributes attr;
        if (cudaPointerGetAttributes(&attr, ptr) != cudaSuccess) {
            (void)cudaGetLastError();
            return;
        }
        if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged) {
            status_ = FA2_ERR_INVALID_ARG;
            return;
        }
        if (cudaGetDevice(&before_) != cudaSuccess) {
            (void)cudaGetLastError();
            return;
        }
        device_ = attr.device;
        if (device_ != before_ && cudaSetDevice(device_) != cudaSuccess) {
            (void)cudaGetLastError();
            return;
        }
        status_ = FA2_OK;
    }
    ~Device()
    {
        if (before_ >= 0 && before_ != device_)
            (void)cudaSetDevice(before_);
    }
    Device(const Device &) = delete;
    Device &operator=(const Device &) = delete;
    fa2_status status() const { return status_; }
    int id() const { return device_; }

private:
    int device_ = -1, before_ = -1;
    fa2_status status_ = FA2_ERR_CUDA;
};

// Device address of g_cache_error on `dev`, which must be current (looked up once per device).
int *device_error_ptr(int dev)
{
    static std::mutex mu;
    static int *cache[kMaxDevices] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < kMaxDevices && cache[dev])
        return cache[dev];
    void *ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, g_cache_error) != cudaSuccess) {
        (void)cudaGetLastError();
        return nullptr;
    }
    if (dev >= 0 && dev < kMaxDevices)
        cache[dev] = static_cast<int *>(ptr);
    return static_cast<int *>(ptr);
}

int test_naps()
{
    const char *s = std::getenv("FA2_TEST_STALL");
    return s && std::strcmp(s, "2") == 0 ? TEST_NAPS : 0;
}

// (batch, head, row) element strides of a bf16 [B, H, L, D] view; NULL: contiguous.
bool row_strides(const long long *given, int H, int L, int D, long long &b, long long &h, long long &l)
{
    if (!given) {
        b = static_cast<long long>(H) * L * D;
        h = static_cast<long long>(L) * D;
        l = D;
        return true;
    }
    for (int i = 0; i < 3; ++i)
        if (given[i] <= 0 || given[i] % 8 != 0 || given[i] > kMaxStride)
            return false;
    b = given[0];
    h = given[1];
    l = given[2];
    return true;
}

bool half_view(Half &x, void *codes, void *scale, const long long (&strides)[3], const fa2_cache *c)
{
    if (!codes || !scale || !aligned(codes, 16))
        return false;
    x.codes = static_cast<uint8_t *>(codes);
    x.scale = static_cast<uint8_t *>(scale);
    if (strides[0] == 0 && strides[1] == 0 && strides[2] == 0) {
        x.s_slot = c->D;
        x.s_head = static_cast<long long>(c->page_size) * c->D;
        x.s_page = x.s_head * c->H;
        return true;
    }
    for (long long s : strides)
        if (s <= 0 || s % 16 != 0 || s > kMaxStride)
            return false;
    x.s_page = strides[0];
    x.s_head = strides[1];
    x.s_slot = strides[2];
    return true;
}

// The cache as the kernels see it; host-side checks only.
fa2_status view_of(const fa2_cache *c, View &v)
{
    if (!c || c->B <= 0 || c->H <= 0 || c->num_pages <= 0 || c->max_pages <= 0 || c->D <= 0 || c->page_size <= 0)
        return FA2_ERR_INVALID_ARG;
    if (!half_view(v.k, c->k, c->k_scale, c->k_strides, c) || !half_view(v.v, c->v, c->v_scale, c->v_strides, c))
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
    if (c->D != 64 && c->D != 128 && c->D != 256)
        return FA2_ERR_UNSUPPORTED;
    v.table = c->page_table;
    v.num_pages = c->num_pages;
    v.H = c->H;
    v.B = c->B;
    v.max_pages = c->max_pages;
    return FA2_OK;
}

fa2_status move(const fa2_cache *c, void *k, void *v, const long long *k_strides, const long long *v_strides,
                const int *starts, const int *counts, int L, bool write, void *stream)
{
    MoveArgs a;
    const fa2_status st = view_of(c, a.c);
    if (st != FA2_OK)
        return st;
    if (!k || !v || !starts || !aligned(k, 16) || !aligned(v, 16) || !aligned(starts, 4) || !aligned(counts, 4) ||
        L < 0 || L > kMaxLength)
        return FA2_ERR_INVALID_ARG;
    if (!row_strides(k_strides, c->H, L, c->D, a.sb[0], a.sh[0], a.sl[0]) ||
        !row_strides(v_strides, c->H, L, c->D, a.sb[1], a.sh[1], a.sl[1]))
        return FA2_ERR_INVALID_ARG;
    if (L == 0)
        return FA2_OK;
    a.x[0] = k;
    a.x[1] = v;
    a.starts = starts;
    a.counts = counts;
    a.L = L;
    a.D = c->D;
    if ((write ? write_blocks(a) : read_blocks(a)) > INT_MAX)
        return FA2_ERR_UNSUPPORTED;
    const Device dev(c->k);
    if (dev.status() != FA2_OK)
        return dev.status();
    return write ? launch_write(a, static_cast<cudaStream_t>(stream)) : launch_read(a, static_cast<cudaStream_t>(stream));
}

size_t workspace_bytes(int D, long long rows, int num_sms)
{
    return D == 64    ? attn_workspace_bytes<64>(rows, num_sms)
           : D == 128 ? attn_workspace_bytes<128>(rows, num_sms)
                      : attn_workspace_bytes<256>(rows, num_sms);
}

}  // namespace
}  // namespace cache
}  // namespace fa2

FA2_EXPORT fa2_status fa2_cache_write(const fa2_cache *c, const void *k, const void *v, const long long *k_strides,
                                      const long long *v_strides, const int *starts, const int *counts, int L,
                                      void *stream)
{
    return fa2::cache::move(c, const_cast<void *>(k), const_cast<void *>(v), k_strides, v_strides, starts, counts, L,
                            true, stream);
}

FA2_EXPORT fa2_status fa2_cache_read(const fa2_cache *c, void *k, void *v, const long long *k_strides,
                                     const long long *v_strides, const int *starts, const int *counts, int L,
                                     void *stream)
{
    return fa2::cache::move(c, k, v, k_strides, v_strides, starts, counts, L, false, stream);
}

FA2_EXPORT fa2_status fa2_cache_attn(const fa2_cache *c, const void *q, void *o, float *lse, const long long *q_strides,
                                     const long long *o_strides, const int *kv_lens, const int *q_lens, int Hq, int Lq,
                                     int causal, int window, float scale, void *workspace, size_t workspace_bytes,
                                     void *stream)
{
    fa2::cache::AttnArgs a;
    const fa2_status st = fa2::cache::view_of(c, a.c);
    if (st != FA2_OK)
        return st;
    using fa2::cache::aligned;
    if (!q || !o || !lse || !kv_lens || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(kv_lens, 4) ||
        !aligned(q_lens, 4))
        return FA2_ERR_INVALID_ARG;
    if (Hq <= 0 || Hq % c->H != 0 || Lq < 0 || static_cast<long long>(c->B) * Hq > INT_MAX ||
        static_cast<long long>(Lq) * (Hq / c->H) > fa2::cache::kMaxLength)
        return FA2_ERR_INVALID_ARG;
    if (!std::isfinite(scale * 1.4426950408889634f) || !(scale > 0.f) || window < -1 || (window >= 0 && !causal))
        return FA2_ERR_INVALID_ARG;
    if (!fa2::cache::row_strides(q_strides, Hq, Lq, c->D, a.q_sb, a.q_sh, a.q_sl) ||
        !fa2::cache::row_strides(o_strides, Hq, Lq, c->D, a.o_sb, a.o_sh, a.o_sl))
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
    const fa2::cache::Device dev(c->k);
    if (dev.status() != FA2_OK)
        return dev.status();
    a.num_sms = fa2::sm_count(dev.id());
    a.err = fa2::cache::device_error_ptr(dev.id());
    a.naps = fa2::cache::test_naps();
    a.drain_limit_ns = fa2::wait_limit_ns();
    a.wait_limit_ns = fa2::call_wait_limit_ns();
    if (a.num_sms <= 0 || !a.err)
        return FA2_ERR_CUDA;
    return c->D == 64    ? fa2::cache::launch_attn<64>(a)
           : c->D == 128 ? fa2::cache::launch_attn<128>(a)
                         : fa2::cache::launch_attn<256>(a);
}

FA2_EXPORT fa2_status fa2_cache_attn_workspace_size(int B, int Hq, int H, int Lq, int D, int device, size_t *bytes)
{
    if (!bytes)
        return FA2_ERR_INVALID_ARG;
    *bytes = 0;
    if (B <= 0 || H <= 0 || Hq <= 0 || Hq % H != 0 || Lq < 0 || D <= 0 || device < 0 ||
        static_cast<long long>(B) * Hq > INT_MAX || static_cast<long long>(Lq) * (Hq / H) > fa2::cache::kMaxLength)
        return FA2_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256)
        return FA2_ERR_UNSUPPORTED;
    if (Lq == 0)
        return FA2_OK;
    const int sms = fa2::sm_count(device);
    if (sms <= 0)
        return FA2_ERR_CUDA;
    *bytes = fa2::cache::workspace_bytes(D, static_cast<long long>(Lq) * (Hq / H), sms);
    return FA2_OK;
}

FA2_EXPORT fa2_status fa2_cache_get_device_error(void *stream, int *detail)
{
    if (detail)
        *detail = 0;
    int v = 0;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess ||
        cudaMemcpyFromSymbol(&v, fa2::cache::g_cache_error, sizeof v) != cudaSuccess) {
        (void)cudaGetLastError();
        return FA2_ERR_CUDA;
    }
    if (v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(fa2::cache::g_cache_error, &zero, sizeof zero) != cudaSuccess) {
            (void)cudaGetLastError();
            return FA2_ERR_CUDA;
        }
    }
    if (detail)
        *detail = v;
    return v ? FA2_ERR_TIMEOUT : FA2_OK;
}
