/*
 * gq_sample.h -- the next token of every request from its logits and a given
 * random number (part of libgq; conventions as in gq.h).
 *
 * Sources: "Gemma 4 M4 Max kernel roadmap", K5 (device top-k with (value,
 * token) pairs): here the whole choice is made on the GPU, for a batch of
 * requests with settings of their own.
 */
#ifndef GQ_SAMPLE_H
#define GQ_SAMPLE_H

#include "gq.h"
#include "gq_kv.h" /* GQ_TYPE_* */

#ifdef __cplusplus
extern "C" {
#endif

/* Largest vocab and n_rows of gq_sample. */
#define GQ_MAX_VOCAB 1048576
#define GQ_MAX_SAMPLE_ROWS 16384

/* ---------------------------------------------------------------------------
 * For every row l of the logits, with temperature T, top_k, top_p, min_p and u:
 *   order   the candidates by falling logit, equal ones by rising index.  A
 *           NaN or -infinity is no candidate (a masked token).
 *   weight  w_i = exp((l_i - max l) / T)
 *   top_k   if > 0: the first top_k of the order
 *   top_p   if < 1: of these the shortest beginning whose weight is at least
 *           top_p times the weight of all of these; always the first
 *   min_p   if > 0: of these the ones with w_i >= min_p, which counts as at most
 *           1: then the ones that share the largest weight
 *   token   the first of the kept whose running sum of weights, in the order,
 *           exceeds u times the sum of all kept
 *   prob    its weight over that sum
 * T <= 0 takes the first of the order (prob 1).  A row without a candidate
 * gives token -1 and prob 0.  u counts as brought into [0, 1]: a NaN or a
 * negative one gives the first, a u of 1 or more the last of the kept that has
 * weight (one some 43 octaves below the largest has none: no u draws it).  T below 2^-100
 * counts as 2^-100; an infinite T gives equal weights.  If the largest logit
 * is +infinity the infinite ones share the weight, whatever T is.  A NaN among T, top_p or
 * min_p gives token -1, prob 0 and GQ_ERR_SHAPE in the device status
 * (gq_device_status).
 *   logits  n_rows rows of vocab elements of `type` (GQ_TYPE_*), ldl elements
 *           apart (any ldl >= vocab), aligned as their type.
 *   temperature, top_p, min_p, u  f32[n_rows], top_k int32[n_rows], 4-byte
 *           aligned.  temperature, top_k, top_p, min_p may each be NULL: 1, no
 *           limit, no limit, no limit.
 *   token   int32[n_rows]; prob f32[n_rows] or NULL.
 *   workspace  device memory, 16-byte aligned, at least
 *           gq_sample_workspace_bytes bytes, scratch before and after the call.
 *           Two calls that may run concurrently must not share it.  The size does
 *           not fall with n_rows: for one vocab, what the largest batch needs serves
 *           every smaller one.
 * Arithmetic: weights are whole numbers of 2^-43 of about the largest weight, each within
 * 2^-23 of itself and 2^-42 of the largest, and added exactly.  The same call
 * gives the same token and prob.  The weight of a whole row may be put together
 * from parts of it, each in units of its own largest, and how a row is divided
 * goes by n_rows: between batches it differs by less than vocab 2^-42 of the
 * largest weight, so prob in its last bits.  A token differs from that of exact
 * weights, or from that in another batch, only where u (or top_p, min_p) lies
 * within rounding of a boundary.
 * Range: 1 <= vocab <= GQ_MAX_VOCAB, 0 <= n_rows <= GQ_MAX_SAMPLE_ROWS (0:
 * nothing to do).
 * Errors before the launches: GQ_ERR_FORMAT (type), GQ_ERR_NULL, GQ_ERR_ALIGN,
 * GQ_ERR_SHAPE, GQ_ERR_WORKSPACE; after them GQ_ERR_CUDA.
 * ------------------------------------------------------------------------ */
size_t gq_sample_workspace_bytes(int vocab, int n_rows); /* 0 if out of range */
int gq_sample(const void *logits, long long ldl, int type, const float *temperature, const int32_t *top_k,
              const float *top_p, const float *min_p, const float *u, int32_t *token, float *prob_or_null,
              void *workspace, size_t workspace_bytes, int vocab, int n_rows, gq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GQ_SAMPLE_H */
