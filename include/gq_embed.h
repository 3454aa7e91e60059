/*
 * gq_embed.h -- rows of a packed quantized table by token id (part of libgq;
 * conventions as in gq.h).
 *
 * Source: "Gemma 4 M4 Max kernel roadmap", K2 "Metal decode path" step 6: the
 * embedding is tied to the output projection, so the table that
 * gq_logits_topk multiplies with is the one that a step begins with.
 */
#ifndef GQ_EMBED_H
#define GQ_EMBED_H

#include "gq.h"
#include "gq_kv.h" /* GQ_TYPE_* */

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Y[t][j] = scale * w_{ids[t], j},  t < M, j < K, with w decoded from the
 * block (gq.h).  The arithmetic is f32: the weight as a matvec decodes it
 * (Q4_K: one rounding, of the difference; Q6_K: of the last product; Q4_0 and
 * Q8_0 are exact), one rounding of the product with scale, and one to the type
 * of Y.
 *   format  GQ_FORMAT_*; W packed (gq_pack), rows x K.
 *   ids     int32[M], 4-byte aligned.  A negative id gives a row of zeros (the
 *           rows behind a padded batch, or a sampled token that there was not);
 *           one of rows or more as well, and the device status
 *           (gq_device_status) becomes GQ_ERR_SHAPE.
 *   Y       M rows of K elements of `type` (GQ_TYPE_*), ldy elements apart,
 *           16-byte aligned with rows a whole multiple of 16 bytes apart.
 *   1 <= rows, 0 <= M (M = 0: nothing to do, ids and Y may be null), K whole
 *   blocks up to 2^24, scale finite.
 * Errors before the launch: GQ_ERR_FORMAT (format or type), GQ_ERR_NULL,
 * GQ_ERR_ALIGN, GQ_ERR_SHAPE; after it GQ_ERR_CUDA.
 * ------------------------------------------------------------------------ */
int gq_embed(int format, const void *W, const int32_t *ids, float scale, void *Y, long long ldy, int type, int rows,
             int K, int M, gq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GQ_EMBED_H */
