/*
 * fa2_paged.h -- C ABI of the 16-bit key/value cache and of the position rotation of
 * the GB300 (sm_103a) FlashAttention-2 library: rotating queries and keys by their
 * positions (and gradients back), appending keys and values to a paged cache, and
 * exact attention over it.
 *
 * These entry points live in a library of their own, libfa2_paged_gb300.so, beside
 * the dense passes of fa2.h and the 8-bit cache of fa2_cache.h; status codes are
 * shared with them.
 *
 * The cache (struct fa2_paged):
 *   - A pool of num_pages pages.  A page holds page_size consecutive positions of one
 *     sequence, for every key/value head: bf16 or fp16 [num_pages, H, page_size, D]
 *     for keys, the same for values.
 *   - page_table [B, max_pages] int32: position p of sequence b is slot
 *     p % page_size of page page_table[b][p / page_size].  An entry outside
 *     [0, num_pages) names no page: what is appended there is dropped, and attention
 *     does not see its positions.  Positions at or past max_pages * page_size have no
 *     page either.
 *
 * The rotation (struct fa2_rotation) turns the first 2 R of a row's D numbers in pairs.
 * With tables cos and sin, fp32 [positions, R], pair j = (x, y) of a row at position p
 * becomes
 *
 *     x' = x cos[p][j] - y sin[p][j],     y' = x sin[p][j] + y cos[p][j]
 *
 * in fp32, each rounded once to the row's type; the other D - 2 R numbers are copied.
 * A pair is numbers j and R + j of the row, or, interleaved, 2 j and 2 j + 1.  The
 * tables are the caller's, so any frequencies and any scaling of them will do.
 *
 * Conventions (as fa2.h where not stated):
 *   - page_size is 16, 32, 64 or 128; D is 64, 128 or 256; dtype is FA2_BF16 or
 *     FA2_FP16, one for all 16-bit tensors of a call.
 *   - Strides are in elements, rows of D contiguous; strides are positive multiples of
 *     8 (16 bytes), at most 2^38; base pointers 16-byte aligned, the fp32 tables too,
 *     int32 arrays 4-byte.
 *   - Lengths, starts and the page table are device memory, read by the kernels when
 *     they run (nothing is synchronised, so calls can be captured into a graph and
 *     replayed with other lengths).  Values outside their range are taken as the
 *     nearest value in it.
 *   - The device is the one that owns the cache (fa2_rope: q); the calling thread's
 *     current device is left as it was.
 */
#ifndef FA2_PAGED_GB300_H
#define FA2_PAGED_GB300_H

#include <stddef.h>

#include "fa2.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { FA2_BF16 = 0, FA2_FP16 = 1 };

typedef struct fa2_paged {
    void *k, *v;                  /* device */
    const int *page_table;        /* [B, max_pages], device */
    long long k_strides[3];       /* page, head, slot; all 0: contiguous */
    long long v_strides[3];
    int num_pages, H, page_size, D;   /* H: key/value heads */
    int B, max_pages;             /* max_pages * page_size <= 2^30 */
    int dtype;
} fa2_paged;

typedef struct fa2_rotation {
    const float *cos, *sin;       /* [positions, R], contiguous, device */
    int positions, R;             /* R a multiple of 8, 2 R <= D; positions at most 2^30 */
    int interleaved;              /* 0: pairs (j, R + j); otherwise (2 j, 2 j + 1) */
} fa2_rotation;

/*
 * fa2_rope -- queries and keys rotated by their positions, or back.
 *
 * Row i of sequence b is at position starts[b] + i; positions outside the tables are
 * taken as the nearest in them.  inverse != 0 turns the other way (sin negated): the
 * rotation is orthogonal where cos^2 + sin^2 = 1, and this, its transpose, is what takes
 * the gradients of the rotated rows back to those of the rows.
 *
 *   q, q_out   16-bit [B, Hq, L, D] device views, strides (batch, head, row) or NULL for
 *              contiguous.  q_out may be q itself (with the same strides), and k_out k;
 *              otherwise a row that is written must not overlap any other row of the call.
 *   k, k_out   the same with H heads; NULL with H = 0: queries only.
 *   starts     int32 [B] device; NULL: 0 for all.
 *   r          the rotation.
 *   L          rows a sequence, at most 2^30 (0: no-op).
 *
 * Errors: FA2_ERR_INVALID_ARG for null or misaligned pointers, sizes or strides that
 * break the rules above; FA2_ERR_UNSUPPORTED for another D or dtype, or more than
 * 2^31 - 1 tokens (B * L) or blocks of up to 2048 / D tokens and 8 heads; FA2_ERR_CUDA.
 */
fa2_status fa2_rope(const void *q, const void *k, void *q_out, void *k_out, const long long *q_strides,
                    const long long *k_strides, const long long *q_out_strides, const long long *k_out_strides,
                    const int *starts, const fa2_rotation *r, int B, int Hq, int H, int L, int D, int dtype,
                    int inverse, void *stream);

/*
 * fa2_paged_append -- new keys and values into the cache, rotated on the way.
 *
 * Row i < counts[b] of sequence b goes to position starts[b] + i: its key rotated for
 * that position, its value as it is.  Rows at negative positions, or without a page,
 * are dropped; slots that get no row keep their bytes.  With q, row i < counts[b] of
 * q_out gets the query of the same token rotated for the same position (whether it has
 * a page or not); other rows of q_out are left as they were.
 *
 *   c          the cache; its pages are written.
 *   k, v       16-bit [B, H, L, D] device views (read only), strides (batch, head, row)
 *              or NULL for contiguous.
 *   starts     int32 [B] device: tokens each sequence holds already.
 *   counts     int32 [B] device, 0..L: rows to append; NULL: L for all.
 *   r          the rotation; NULL: none (keys are stored as they are, and q must be NULL).
 *   q, q_out   16-bit [B, Hq, L, D] device views, or both NULL with Hq = 0.  q_out may be
 *              q itself, as in fa2_rope.
 *   L          rows a sequence in k, v and q, at most 2^30 (0: no-op).
 *
 * A slot must not get two rows in one call (two sequences whose tables name one page
 * may append to different slots of it).  The new rows must not overlap the cache.
 * Errors as fa2_rope.
 */
fa2_status fa2_paged_append(const fa2_paged *c, const void *k, const void *v, const long long *k_strides,
                            const long long *v_strides, const int *starts, const int *counts,
                            const fa2_rotation *r, const void *q, void *q_out, const long long *q_strides,
                            const long long *q_out_strides, int Hq, int L, void *stream);

/*
 * fa2_paged_attn -- exact attention of the newest tokens over the cache.
 *
 * Sequence b holds kv_lens[b] positions, the last q_lens[b] of which are the query
 * tokens (their keys and values are in the cache already).  With
 * pos(i) = kv_lens[b] - q_lens[b] + i, and hk = h * c->H / Hq the key/value head that
 * query head h shares:
 *
 *     s_ij = scale * sum_d Q[b,h,i,d] * K[b,hk,j,d]     for visible positions j
 *     O[b,h,i,:] = sum_j softmax_j(s_i.) * V[b,hk,j,:]
 *     LSE[b,h,i] = ln sum_j exp(s_ij)
 *
 * Visible: 0 <= j < kv_lens[b], with a page; with causal != 0 also j <= pos(i);
 * with window >= 0 (causal only) also j >= pos(i) - window.  A row that sees nothing,
 * or nothing but scores of -infinity, gets O = 0 and LSE = -infinity.  What lies in
 * positions that a row does not see, NaN and infinities included, has no part in it; an
 * infinity or NaN in a value that it sees makes that column of its O infinite or NaN,
 * one in a key or in the row of q the row's scores.
 *
 * Scores, sums, softmax statistics and O are fp32, O rounded once to the cache's type.
 * For the product with V a softmax weight is rounded: up to 16 rows (Lq * Hq / H), up to
 * 32 for D of 64 and 128, and for bf16 at D of 256 whatever the rows, to two terms of the
 * cache's type together, off by 2^-16 of the weight for bf16 and 2^-22 for fp16; for more rows
 * to one term, off by 2^-9 and 2^-12 on average and 2^-8 and 2^-11 at most.  An fp16 weight
 * may in either case be off by 2^-31 of the row's largest weight, where that is more (so one
 * below 2^-20 of it is held in fewer bits, and one below 2^-31 may count as 0); a bf16 one
 * by 2^-114.  Where bf16 has one term O is divided by the sum of the rounded weights (where one
 * key dominates, its rounding cancels); LSE, and all else, takes the sum before.
 * O is finite where values are, unless a column's sum_j exp(s_ij - max_j s_ij) |V_j| is 2^131
 * or more: not with 8 keys of the largest finite bf16 value, nor with any number of values
 * below 2^101.  A bf16 key's part in it counts down to 2^-137.
 *
 *   q          16-bit [B, Hq, Lq, D] device view, strides (batch, head, row) or NULL.
 *   o          16-bit [B, Hq, Lq, D] device view (written), likewise; its rows must not
 *              overlap one another, nor q.
 *   lse        fp32 [B, Hq, Lq] contiguous (written).
 *   kv_lens    int32 [B] device: positions held, the query tokens among them.
 *   q_lens     int32 [B] device, 0..Lq: query rows of each sequence; NULL: Lq for
 *              all.  Rows i >= q_lens[b] of o and lse are left as they were.
 *   Hq         query heads, a multiple of c->H.
 *   Lq         query rows a sequence (0: no-op); Lq * Hq / H at most 2^30.
 *   scale      > 0, and finite times log2 e (below 2.358e38).
 *   workspace  optional device workspace (256-byte aligned, fa2_paged_attn_workspace_size
 *              bytes, ZERO-FILLED before its first use, left ready by every completed
 *              call).  With it the keys of one sequence are shared out among SMs;
 *              without it (NULL) each block of query rows is one CTA's work.  Calls that
 *              may run at the same time must not share one.
 *
 * Results do not depend on timing: the parts of a row are merged in a fixed order.
 * The work of a call is counted in blocks of 8, 16, 32 (D < 256), 128 (D = 256) or 256 of
 * a key/value head's Lq * Hq / H rows, by its keys: 4 a tile of 128 keys and 12 a block, or
 * for blocks of 128 and 256 rows 8 a tile and 32 a block.  Sizes for which max_pages full
 * pages would make more than 2^30 of these are refused (FA2_ERR_UNSUPPORTED).
 * Errors as fa2_rope, also FA2_ERR_INVALID_ARG for a bad scale or window, Hq not a
 * multiple of H, or a workspace that is misaligned or too small.
 */
fa2_status fa2_paged_attn(const fa2_paged *c, const void *q, void *o, float *lse, const long long *q_strides,
                          const long long *o_strides, const int *kv_lens, const int *q_lens, int Hq, int Lq,
                          int causal, int window, float scale, void *workspace, size_t workspace_bytes,
                          void *stream);

/*
 * fa2_paged_attn_workspace_size -- bytes of workspace fa2_paged_attn can use for any
 * lengths with these sizes on `device`.  Errors as fa2_workspace_size.
 */
fa2_status fa2_paged_attn_workspace_size(int B, int Hq, int H, int Lq, int D, int device, size_t *bytes);

/*
 * fa2_paged_get_device_error -- synchronises `stream`, then reads and clears this
 * library's device-side error word on the current device, as fa2_get_device_error does
 * for the dense passes: every wait between warps in the attention kernels is bounded
 * (one second; FA2_WAIT_LIMIT_MS), one that runs out records a code, and the kernel
 * winds down.  Outputs of that call are then undefined, and a workspace it used must be
 * zero-filled again.
 *
 * For tests only (read on every call): FA2_TEST_WAIT_LIMIT_NS sets the limit of the
 * waits between fa2_paged_attn's warps (not of those for a CTA's own copies and
 * products); FA2_TEST_STALL=2 makes some of the warps tens of microseconds late, which
 * must not change a result, but with a limit of a nanosecond lets the others' waits on
 * them run out.
 *
 *   detail   optional: the raw code (0 = none), the waiting role in bits 8-11, the
 *            barrier in the low byte.
 *
 * Returns FA2_OK, FA2_ERR_TIMEOUT, or FA2_ERR_CUDA.
 */
fa2_status fa2_paged_get_device_error(void *stream, int *detail);

#ifdef __cplusplus
}
#endif

#endif /* FA2_PAGED_GB300_H */
