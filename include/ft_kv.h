/*
 * ft_kv.h -- C ABI of libft's paged key/value cache and the attention half of
 * a step that surrounds the MoE layer of ft.h: the page operations (extend,
 * fork, free, compact), the pass that normalises and rotates the heads of
 * queries and keys and stores keys and values into their pages, and attention
 * over the page table, with a prefix that the requests of a group share
 * computed once for all of them.
 *
 * Conventions: those of ft.h.  All calls but ft_kv_init, ft_kv_destroy,
 * ft_kv_status and ft_kv_last are async on the cache's stream, allocate
 * nothing, do not synchronise and can be captured in a CUDA graph.  What the
 * device finds wrong latches an error word that ft_kv_status returns.
 *
 * The cache is memory of the caller (an engine that carves device memory into
 * its own pools keeps doing so):
 *
 *   pool   n_pages complete page records.  A record holds `page` tokens of all
 *          layers: [L][2: K, V][Hkv][page][D], 16-bit values (dtype), so that
 *          every bank of a page belongs to the same tokens.
 *   table  int32 [n_rows, row_pages].  Row r lists the pages of sequence r in
 *          order: token t is in page table[r][t / page] at t % page; entries
 *          past the last page are -1.
 *   lens   int32 [n_rows], tokens of each row (0: the row is empty).
 *   refs   int32 [n_pages], how many rows hold the page (0: free).
 *
 * An empty cache has table = -1, lens = 0, refs = 0 (the caller fills them).
 * Contents of the pool beyond a row's length are never used, whatever they
 * are (NaN included).
 */
#ifndef FT_KV_H
#define FT_KV_H

#include "ft.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FT_KV_BF16 0
#define FT_KV_F16  1

typedef struct ft_kv ft_kv;   /* opaque; created by ft_kv_init, freed by ft_kv_destroy */

/* What the last page operation did (ft_kv_last). */
typedef struct {
    int32_t allocated;   /* pages taken from the free ones                        */
    int32_t copied;      /* page records copied, whole or in part                 */
    int32_t live;        /* after ft_kv_compact: pages in use (they are 0..live-1); else -1 */
} ft_kv_info;

/* Bytes of one page record, L*2*Hkv*page*D*2; 0 where ft_kv_init refuses the sizes. */
size_t ft_kv_page_bytes(int32_t L, int32_t Hkv, int32_t D, int32_t page);

/* Bytes of device scratch that ft_kv_init allocates for these sizes on the
 * current device (the plan, the copy list and the partial results of
 * attention); 0 where it refuses the sizes or there is no device. */
size_t ft_kv_scratch_bytes(int32_t Hq, int32_t Hkv, int32_t D, int32_t n_pages, int32_t n_rows, int32_t T_max,
                           int32_t B_max);

/*
 * ft_kv_init -- a handle on a cache; syncs.
 *   L, Hq, Hkv, D  layers, query heads, key/value heads (Hq a multiple of Hkv,
 *                  at most 128 query heads per key/value head; query head i
 *                  reads key/value head i / (Hq/Hkv)), head size 64, 128 or 256.
 *   page           tokens of a page: 16, 32, 64 or 128.
 *   n_pages, n_rows, row_pages  sizes of the pool and the table;
 *                  row_pages*page and n_pages*L*2*Hkv below 2^31, n_rows
 *                  at most 65536.
 *   dtype          FT_KV_BF16 or FT_KV_F16: type of the pool, the queries and
 *                  the outputs.
 *   T_max, B_max   largest number of query tokens and of requests of an
 *                  ft_attn_plan; 1 <= B_max <= 1024, T_max >= 1, T_max*Hq below
 *                  2^30, 2*T_max*Hq + 128*Hkv*(B_max + 1) below 2^31 - 2^23.
 *   pool           DEVICE, 128-byte aligned;  table, lens, refs DEVICE, 4-byte
 *                  aligned.  All four stay valid until ft_kv_destroy.
 *   stream         cudaStream_t that every call runs on (NULL = legacy default
 *                  stream); it must outlive the handle.
 * Errors: FT_ERR_ARG, FT_ERR_OOM, FT_ERR_CUDA.
 */
ft_status ft_kv_init(ft_kv** out, int32_t L, int32_t Hq, int32_t Hkv, int32_t D, int32_t page, int32_t n_pages,
                     int32_t n_rows, int32_t row_pages, int32_t dtype, int32_t T_max, int32_t B_max, void* pool,
                     int32_t* table, int32_t* lens, int32_t* refs, void* stream);

/*
 * Page operations.  Each is one control pass on the device and, where pages
 * move, one copy kernel over all layers.  Pages are taken lowest free index
 * first, in the order of the list, so a result does not depend on timing.  A
 * call that finds a bad argument on the device (a row out of range, a row
 * twice in the list, a fork onto a row that is not empty or that is a parent
 * in the same call, a length past row_pages*page, a page index out of range) latches FT_ERR_DEVICE, one that
 * finds too few free pages FT_ERR_CAPACITY; either changes nothing.
 * n is 0..n_rows; list pointers are DEVICE int32 [n].
 */

/* Row rows[i] grows by add[i] >= 0 tokens; the pages that this needs are
 * taken, their contents are left as they are. */
ft_status ft_kv_extend(ft_kv* kv, int32_t n, const int32_t* rows, const int32_t* add);

/* Row children[i], which is empty, becomes a copy of row parents[i]: its
 * complete pages are shared (their counts grow), of a last page that is not
 * complete the tokens are copied to a new page.  A parent may be listed
 * more than once. */
ft_status ft_kv_fork(ft_kv* kv, int32_t n, const int32_t* parents, const int32_t* children);

/* Rows rows[i] become empty; pages that no row holds any more are free.  A
 * page whose count is already 0 latches FT_ERR_DEVICE (the row is emptied
 * all the same). */
ft_status ft_kv_free(ft_kv* kv, int32_t n, const int32_t* rows);

/* The pages in use become pages 0..live-1: the pages in use at index >= live
 * move to the free ones below live, the lowest first into the lowest, and table
 * and refs follow.  The upper part of the pool then holds nothing, but a handle
 * keeps its n_pages and may take those pages again.  To use that memory for
 * something else: ft_kv_destroy, then ft_kv_init with a smaller n_pages >= live
 * on the same pool, table, lens and refs, which goes on with the same rows. */
ft_status ft_kv_compact(ft_kv* kv);

/*
 * ft_qk_rope_store -- one pass over the projection's output of T tokens:
 * RMS norm of every query and key head over its D values, rotation of the
 * first `rot` values by the token's position, queries to q_out, keys and
 * values into their pages of `layer`.  All arithmetic in fp32, one rounding
 * at the end; values are copied bit for bit.
 *   qkv      DEVICE [T, >= (Hq+2*Hkv)*D], dtype of the cache, row stride ld
 *            elements: the query heads, the key heads, the value heads.
 *   row_of, pos  DEVICE int32 [T]: row of the table and position in it of each
 *            token.  A token with row -1 is padding: its queries become 0 and
 *            nothing is stored.  A position whose page the row does not have,
 *            or past max_pos, latches FT_ERR_DEVICE and is treated the same.
 *            No two tokens of a call may name the same place.
 *   q_norm, k_norm  DEVICE [D] weights, dtype of the cache; NULL: that head
 *            kind is not normalised.  eps is added to the mean square.
 *   cos_sin  DEVICE fp32 [max_pos, rot]: cosines of the rot/2 angles, then
 *            their sines.  rot is 0..D, a multiple of 16 (0: no rotation,
 *            cos_sin and max_pos are ignored).
 *   pair     0: value i turns with value i + rot/2; 1: 2i with 2i+1.
 *   q_out    DEVICE [T, >= Hq*D], row stride ld_q; may be qkv itself, or other
 *            columns of its rows (same stride); must not overlap it otherwise.
 * ld, ld_q multiples of 8; qkv, q_out, norms and cos_sin 16-byte aligned.
 */
ft_status ft_qk_rope_store(ft_kv* kv, int32_t layer, int32_t T, const void* qkv, int64_t ld, const int32_t* row_of,
                           const int32_t* pos, void* q_out, int64_t ld_q, const void* q_norm, const void* k_norm,
                           float eps, const float* cos_sin, int32_t max_pos, int32_t rot, int32_t pair);

/*
 * ft_attn_plan -- lay out the work of attention for a batch from the lengths
 * in `lens` as they are on the stream now.  One plan serves every layer of a
 * step: ft_attn_forward uses the last one.
 *   B, T     requests (0..B_max) and query tokens (0..T_max).
 *   cu_q     DEVICE int32 [B+1], ascending from 0: request b has the query
 *            tokens cu_q[b]..cu_q[b+1]-1 (none is allowed), cu_q[B] <= T.  Outputs of the
 *            tokens from cu_q[B] on are not written.
 *   rows     DEVICE int32 [B], the table row of each request; NULL: row b.
 *   n_groups, group_start, group_tokens
 *            DEVICE int32 [n_groups+1] and [n_groups]: the requests
 *            group_start[g]..group_start[g+1]-1 share their first
 *            group_tokens[g] tokens, that is, their rows start with the same
 *            pages.  Taken as shared are the whole pages that precede every
 *            query of the group and that the rows of all its requests with
 *            queries have in common; a claim that is too large is cut to that,
 *            so what is claimed changes the speed, never the result.
 *            n_groups = 0 (then both may be NULL): nothing is shared; requests
 *            of few tokens then run a form of their own, which is the faster
 *            one for them, so a caller without a shared prefix passes 0.
 *            n_groups <= B.
 * Errors found on the device (cu_q or groups not ascending or out of range, a
 * row out of range, a length out of range): FT_ERR_DEVICE; the plan is empty.
 */
ft_status ft_attn_plan(ft_kv* kv, int32_t B, int32_t T, const int32_t* cu_q, const int32_t* rows, int32_t n_groups,
                       const int32_t* group_start, const int32_t* group_tokens);

/*
 * ft_attn_forward -- attention of the planned queries over `layer`:
 * out = softmax(scale * q K^T) V per head, query i of the n of a request
 * seeing its row's keys 0 .. len - n + i (the new tokens are the last of the
 * row).  A query that sees no key gives zeros.  Scores, softmax statistics
 * and sums are fp32; the softmax weights are rounded to the cache's type for
 * the product with V (f16: to its 11 bits down to 2^-22 of a row's largest
 * weight, and to multiples of 2^-32 of it below).  Keys that a query does not
 * see may hold anything.  Values must be finite at places within the row's
 * length that some query of the same tile of 128 rows does not see: one that is
 * not reaches the queries of the tile that precede it.
 *   q        DEVICE [T, >= Hq*D], row stride ld_q;  out the same with ld_o;
 *            out must not overlap q.  ld_q, ld_o multiples of 8, both pointers
 *            16-byte aligned.
 *   scale    finite, > 0.
 * Errors: FT_ERR_ARG, FT_ERR_STATE (no plan yet), FT_ERR_CUDA; a page index
 * out of range within a row's length latches FT_ERR_DEVICE.
 */
ft_status ft_attn_forward(ft_kv* kv, int32_t layer, const void* q, int64_t ld_q, void* out, int64_t ld_o, float scale);

/* Summary of the last page operation; syncs. */
ft_status ft_kv_last(ft_kv* kv, ft_kv_info* out);

/* Synchronise the stream and return, then clear, what the device latched since
 * the last call: FT_OK, FT_ERR_DEVICE, FT_ERR_CAPACITY or FT_ERR_TIMEOUT (a
 * bounded wait gave up; outputs since the last status are not valid). */
ft_status ft_kv_status(ft_kv* kv);

/* Free the handle and its scratch, not the caller's memory.  Syncs.  kv may be NULL. */
void ft_kv_destroy(ft_kv* kv);

#ifdef __cplusplus
}
#endif
#endif /* FT_KV_H */
