/*
 * fa2_cache.h -- C ABI of the 8-bit key/value cache of the GB300 (sm_103a)
 * FlashAttention-2 library: writing keys and values into a paged cache, reading
 * them back, and exact attention over the cache.
 *
 * These entry points live in a library of their own, libfa2_cache_gb300.so,
 * beside the dense passes of fa2.h; status codes are shared with it.
 *
 * The cache (struct fa2_cache):
 *   - A pool of num_pages pages.  A page holds page_size consecutive positions
 *     of one sequence, for every key/value head: e4m3 codes (OCP FP8 E4M3: bias
 *     7, largest finite 448, no infinities) [num_pages, H, page_size, D] for
 *     keys, the same for values.
 *   - One scale for each page and head, for keys and values apart: e8m0 bytes
 *     [num_pages, H] (contiguous), byte e standing for 2^(e - 127), 255 for NaN.
 *     The number a code stands for is code * scale.  Powers of two make that
 *     product exact, and make a larger scale taken later (see fa2_cache_write)
 *     move codes without a new rounding unless they become subnormal.
 *   - page_table [B, max_pages] int32: position p of sequence b is slot
 *     p % page_size of page page_table[b][p / page_size].  An entry outside
 *     [0, num_pages) names no page: what is written there is dropped, it reads
 *     as zeros, and attention does not see its positions.  Positions at or past
 *     max_pages * page_size have no page either.
 *
 * Conventions (as fa2.h where not stated):
 *   - page_size is 16, 32, 64 or 128; D is 64, 128 or 256.
 *   - Strides are in elements, rows of D contiguous.  Cache strides are positive
 *     multiples of 16 (16 bytes), strides of bf16 tensors positive multiples of
 *     8, at most 2^38; base pointers 16-byte aligned, int32 arrays 4-byte.
 *   - Lengths, starts and the page table are device memory, read by the kernels
 *     when they run (nothing is synchronised, so calls can be captured into a
 *     graph and replayed with other lengths).  Values outside their range are
 *     taken as the nearest value in it.
 *   - The device is the one that owns the cache; the calling thread's current
 *     device is left as it was.
 */
#ifndef FA2_CACHE_GB300_H
#define FA2_CACHE_GB300_H

#include <stddef.h>

#include "fa2.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct fa2_cache {
    void *k, *v;                  /* e4m3 codes, device */
    void *k_scale, *v_scale;      /* e8m0 [num_pages, H], device */
    const int *page_table;        /* [B, max_pages], device */
    long long k_strides[3];       /* page, head, slot; all 0: contiguous */
    long long v_strides[3];
    int num_pages, H, page_size, D;   /* H: key/value heads */
    int B, max_pages;             /* max_pages * page_size <= 2^30 */
} fa2_cache;

/*
 * fa2_cache_write -- quantise new keys and values into the cache.
 *
 * Row i < counts[b] of sequence b goes to position starts[b] + i.  For every
 * page and head that gets a row, keys and values apart, with a the largest
 * finite magnitude among the rows that this call puts there:
 *
 *     e = least e >= -96 with a <= 448 * 2^e, at most 119
 *     if the page also holds positions before starts[b]:  e = max(e, its present exponent)
 *     code = e4m3(x * 2^-e), round to nearest even, saturating (only above 448 * 2^119)
 *
 * and codes of earlier positions in the page are brought to the new scale,
 * e4m3(code * 2^(e_before - e)), when it grew.  A page whose first slot is
 * written by the call starts afresh; slots past the last row keep their bytes.
 * NaN and infinities are stored as the NaN code, so that attention shows them.
 *
 *   c          the cache; its pages and scales are written.
 *   k, v       bf16 [B, H, L, D] device views (read only), strides (batch, head,
 *              row) or NULL for contiguous.
 *   starts     int32 [B] device: tokens each sequence holds already.  Rows at
 *              negative positions are dropped.
 *   counts     int32 [B] device, 0..L: rows to write; NULL: L for all.
 *   L          rows a sequence in k and v, at most 2^30 (0: no-op).  A call's blocks, one for
 *              keys and one for values of each page that L rows can touch (write) or of each
 *              8192 / D rows (read), of B * H heads, are at most 2^31 - 1.
 *
 * A page that gets rows must be named once among the touched entries of the
 * page table: two sequences that write into one page race, and its contents
 * are then undefined.  Reading shared pages is always fine.
 *
 * Errors: FA2_ERR_INVALID_ARG for null or misaligned pointers, sizes or strides
 * that break the rules above; FA2_ERR_UNSUPPORTED for another D or page_size, or more
 * blocks than that; FA2_ERR_CUDA.
 */
fa2_status fa2_cache_write(const fa2_cache *c, const void *k, const void *v, const long long *k_strides,
                           const long long *v_strides, const int *starts, const int *counts, int L,
                           void *stream);

/*
 * fa2_cache_read -- keys and values out of the cache, as bf16.
 *
 * Row i < counts[b] of k and v gets position starts[b] + i of sequence b, code *
 * scale rounded to bf16 (exact unless it leaves bf16's range); positions without
 * a page give zeros.  Rows i >= counts[b] are left as they were.
 *
 *   k, v       bf16 [B, H, L, D] device views (written), strides as above; their
 *              rows must not overlap.
 *   (other arguments and errors as fa2_cache_write)
 */
fa2_status fa2_cache_read(const fa2_cache *c, void *k, void *v, const long long *k_strides,
                          const long long *v_strides, const int *starts, const int *counts, int L,
                          void *stream);

/*
 * fa2_cache_attn -- exact attention of the newest tokens over the cache.
 *
 * Sequence b holds kv_lens[b] positions, the last q_lens[b] of which are the
 * query tokens (their keys and values are in the cache already).  With
 * pos(i) = kv_lens[b] - q_lens[b] + i, K and V the numbers the cache stands for
 * and hk = h * c->H / Hq the key/value head that query head h shares:
 *
 *     s_ij = scale * sum_d Q[b,h,i,d] * K[b,hk,j,d]     for visible positions j
 *     O[b,h,i,:] = sum_j softmax_j(s_i.) * V[b,hk,j,:]
 *     LSE[b,h,i] = ln sum_j exp(s_ij)
 *
 * Visible: 0 <= j < kv_lens[b], with a page; with causal != 0 also j <= pos(i);
 * with window >= 0 (causal only) also j >= pos(i) - window.  A row that sees
 * nothing gets O = 0 and LSE = -infinity.  The products run on the cache's codes
 * as they are, with q as a sum of two e4m3 numbers times a power of two of its row:
 * that is q itself but for elements far below their row's largest, which are off by
 * at most 2^-21 of it (up to 16 rows, Lq * Hq / H) or 2^-17 (more).  Sums and softmax
 * are fp32; for the product with V a softmax weight is rounded to fp16 (11 bits), and up
 * to 16 rows taken as three e4m3 terms, which hold that.  What is rounded is the weight
 * times its page's value scale, against the largest such product, so a small one is off by
 * an absolute amount: 2^-25 of the largest among the 128 keys of its tile (up to 16 rows),
 * 2^-31 of the largest that the row sees (more rows).  A column of O in which strong pages
 * hold zeros shows it: values of pages weaker by more than that are lost there.  The sum of
 * the weights, and with it LSE, has no part in this; from it, keys may be missing whose
 * value scale is more than 2^100 below the largest that the row sees (a page of zeros has
 * 2^-96).  A row of q with an infinity or NaN gives NaN.  Scales are those that
 * fa2_cache_write gives, 2^-96 to 2^119, or NaN.
 *
 *   q          bf16 [B, Hq, Lq, D] device view, strides (batch, head, row) or NULL.
 *   o          bf16 [B, Hq, Lq, D] device view (written), likewise; its rows must not overlap
 *              one another, nor q.
 *   lse        fp32 [B, Hq, Lq] contiguous (written).
 *   kv_lens    int32 [B] device: positions held, the query tokens among them.
 *   q_lens     int32 [B] device, 0..Lq: query rows of each sequence; NULL: Lq for
 *              all.  Rows i >= q_lens[b] of o and lse are left as they were.
 *   Hq         query heads, a multiple of c->H.
 *   Lq         query rows a sequence (0: no-op); Lq * Hq / H at most 2^30.
 *   scale      > 0, and finite times log2 e (below 2.358e38).
 *   workspace  optional device workspace (256-byte aligned, fa2_cache_attn_workspace_size
 *              bytes, ZERO-FILLED before its first use, left ready by every
 *              completed call).  With it the keys of one sequence are shared out
 *              among SMs; without it (NULL) each block of query rows is one CTA's
 *              work.  Calls that may run at the same time must not share one.
 *
 * Results do not depend on timing: the parts of a row are merged in a fixed order.
 * The work of a call is counted in tiles of 128 keys by blocks of 8, 16, 128 or 256 of
 * a key/value head's Lq * Hq / H rows; sizes for which max_pages full pages would make
 * more than 2^30 of them are refused (FA2_ERR_UNSUPPORTED).
 * Errors as fa2_cache_write, also FA2_ERR_INVALID_ARG for a bad scale or window, Hq
 * not a multiple of H, or a workspace that is misaligned or too small.
 */
fa2_status fa2_cache_attn(const fa2_cache *c, const void *q, void *o, float *lse, const long long *q_strides,
                          const long long *o_strides, const int *kv_lens, const int *q_lens, int Hq, int Lq,
                          int causal, int window, float scale, void *workspace, size_t workspace_bytes,
                          void *stream);

/*
 * fa2_cache_attn_workspace_size -- bytes of workspace fa2_cache_attn can use for
 * any lengths with these sizes on `device`.  Errors as fa2_workspace_size.
 */
fa2_status fa2_cache_attn_workspace_size(int B, int Hq, int H, int Lq, int D, int device, size_t *bytes);

/*
 * fa2_cache_get_device_error -- synchronises `stream`, then reads and clears this
 * library's device-side error word on the current device, as fa2_get_device_error
 * does for the dense passes: every wait between warps in the attention kernels is
 * bounded (one second; FA2_WAIT_LIMIT_MS), one that runs out records a code, and the
 * kernel winds down.  Outputs of that call are then undefined, and a workspace it used
 * must be zero-filled again.
 *
 * For tests only (read on every call): FA2_TEST_WAIT_LIMIT_NS sets the limit of the waits
 * between fa2_cache_attn's warps (not of those for a CTA's own copies and products);
 * FA2_TEST_STALL=2 makes some of the warps tens of microseconds late, which must not change
 * a result, but with a limit of a nanosecond lets the others' waits on them run out.
 *
 *   detail   optional: the raw code (0 = none), the waiting role in bits 8-11, the
 *            barrier in the low byte.  Roles, up to 16 rows: 12 softmax, 13 loading,
 *            14 MMA issuer, 15 a CTA's final wait for its own work; more rows: 8, 11,
 *            10 and 7, and 9 conversion.
 *
 * Returns FA2_OK, FA2_ERR_TIMEOUT, or FA2_ERR_CUDA.
 */
fa2_status fa2_cache_get_device_error(void *stream, int *detail);

#ifdef __cplusplus
}
#endif

#endif /* FA2_CACHE_GB300_H */
