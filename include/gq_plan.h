/*
 * gq_plan.h -- the lists of a batch, made on the GPU from the requests'
 * lengths (part of libgq; conventions as in gq.h, the batch and the paged
 * cache as in gq_kv.h).
 *
 * Sources: "Gemma 4 M4 Max kernel roadmap", K4 "scheduling and memory"
 * (arenas are allocated once; generation performs no tensor-sized
 * allocation): the cache's pages are handed out by a kernel, so that a
 * captured step can be replayed while requests grow, start and end.
 */
#ifndef GQ_PLAN_H
#define GQ_PLAN_H

#include "gq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest n_seq of gq_kv_plan. */
#define GQ_MAX_PLAN_SEQ 8192

/* ---------------------------------------------------------------------------
 * Plan one step.  Request b has kv_len_in[b] tokens in the cache and gets
 * n_new[b] more (0 or more), or has ended (n_new[b] < 0).
 *   kv_len[b]  = kv_len_in[b] + n_new[b], or 0 if it has ended
 *   q_start    = 0 and the running sums of max(n_new, 0)   (int32[n_seq + 1])
 *   block_table: a request's entries ceil(kv_len_in / page_tokens) ..
 *                ceil(kv_len / page_tokens) - 1 get the pages that it takes;
 *                no other entry is written.
 * The lists are those that gq_kv_append_q8_0 and gq_kv_attention_q8_0 take.
 *
 * Free pages.  `free_pages` (int32[n_pages]) is a ring; ring_in = {first,
 * count} says that its entries first .. first + count - 1 (modulo n_pages)
 * are free.  The requests take pages from its front, in the order of b and
 * of their positions; the pages of ended requests join its end, in the same
 * order, and can be taken in the next step.  ring = {first, count} after
 * that.  A program begins with all page numbers in the ring, {0, n_pages}.
 * Only the entries that join are written.
 *
 * Per token (each may be NULL): for row t of the token arrays
 *   slot[t]      page * page_tokens + offset of its place in the cache (int64)
 *   position[t]  its position in its request
 *   sequence[t]  its request b
 * Rows q_start[n_seq] .. n_tokens - 1, where the arrays are longer than the
 * step needs (a captured batch of a fixed size), get -1 in all three.  (The
 * attention and the append take n_tokens = q_start[n_seq] or more; they leave
 * rows behind the last request alone.)
 *
 * kv_len may be kv_len_in and ring may be ring_in; no other lists may
 * overlap.  All lists are device memory, 4-byte aligned (slot: 8-byte).
 *
 * A step that cannot be planned changes nothing: kv_len = kv_len_in, ring =
 * ring_in, q_start = 0 everywhere, -1 for every token, and the device status
 * (gq_device_status) becomes GQ_ERR_SHAPE.  That is a step with more new
 * tokens than n_tokens, a request longer than max_pages * page_tokens, a
 * negative kv_len_in, fewer free pages than the requests take, or a ring that
 * does not fit n_pages.  A page number outside 0 .. n_pages - 1 (in the ring or
 * the table) gives slot -1 and the same status; the append and the attention
 * do not follow it either.
 *
 * Range: 1 <= n_seq <= GQ_MAX_PLAN_SEQ, page_tokens a multiple of 16 up to
 * 4096, max_pages * page_tokens at most 2^28, 0 <= n_tokens <= 2^28,
 * 1 <= n_pages <= 2^28.  Errors before the launch: GQ_ERR_NULL, GQ_ERR_ALIGN,
 * GQ_ERR_SHAPE; after it GQ_ERR_CUDA.
 * ------------------------------------------------------------------------ */
int gq_kv_plan(const int32_t *n_new, const int32_t *kv_len_in, const int32_t *ring_in, int32_t *free_pages,
               int32_t *block_table, int32_t *kv_len, int32_t *q_start, int32_t *ring, int64_t *slot_or_null,
               int32_t *position_or_null, int32_t *sequence_or_null, int n_pages, int max_pages, int page_tokens,
               int n_seq, int n_tokens, gq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GQ_PLAN_H */
