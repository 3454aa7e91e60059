/*
 * gq_lora.h -- low-rank adapters of many requests beside a shared projection
 * (part of libgq; conventions as in gq.h).
 *
 * The source pages have no counterpart.  The shared weights stay quantized and
 * are multiplied once for the whole batch (gq_q4_0_matvec,
 * gq_q4_0_gemm_q8act); what differs between the requests is added here.
 */
#ifndef GQ_LORA_H
#define GQ_LORA_H

#include "gq.h"
#include "gq_kv.h" /* GQ_TYPE_* */

#ifdef __cplusplus
extern "C" {
#endif

/* Largest rank of an adapter. */
#define GQ_MAX_LORA_RANK 128

/* ---------------------------------------------------------------------------
 * For every token t < M with adapter a = adapter[sequence[t]]:
 *   Y[t] = Y0[t] + scale[a] * B_a (A_a x_t)
 * and Y[t] = Y0[t] for a token without one (a < 0, or sequence[t] < 0).
 *   A       [n_adapters][rank][K] and B [n_adapters][rows][rank], both of
 *           `type` GQ_TYPE_F16 or GQ_TYPE_BF16, row-major and contiguous.
 *           An adapter of a smaller rank is filled up with zeros in A and B.
 *   scale   f32[n_adapters]
 *   adapter int32[n_seq]: the requests' adapters.
 *   sequence int32[M]: the tokens' requests (as gq_kv_plan writes it), or NULL:
 *           token t belongs to request t (a decode batch; M = n_seq then).
 *   X       f32, M rows of K elements, ldx elements apart; or, for
 *           gq_lora_add_q8act, Xq int8[M][K] and dx f32[M][K / 32] as
 *           gq_quantize_q8_0 writes them, x = dx * Xq.
 *   Y0, Y   f32, M rows of `rows` elements, ldy0 and ldy elements apart.  Y may
 *           be Y0 (then ldy = ldy0; rows without an adapter are not touched);
 *           otherwise they may not overlap.  A part of a wider projection
 *           (q, k or v) is a pointer to its first column and the wider row's
 *           stride.
 *   workspace  device memory, at least gq_lora_workspace_bytes bytes, scratch
 *           before and after the call.  Two calls that may run concurrently
 *           must not share it.  The size does not fall with M, K or rank: what the
 *           largest batch needs serves every smaller one.
 * An adapter number of n_adapters or more, or a request number of n_seq or
 * more, counts as none, and the device status (gq_device_status) becomes
 * GQ_ERR_SHAPE.
 *
 * Accuracy: |error| <= 2^-24 |Y| +
 *   (2^-17 + 2^-32 K) |scale| sum_j |B_ij| sum_k |A_jk x_k|
 * (operands of 22 bits or more, f32 sums, those of the tensor cores truncated;
 * this is every rounding at its worst), and within 1e-6 of the added term in
 * the 2-norm.  With f16 adapters a token's numbers scale (A x)_j are cut at
 * 2^-38 of the largest of them: up to
 *   2^-38 |scale| sum_j |B_ij| max_j sum_k |A_jk x_k|
 * more, which shows only where a row of B takes none but numbers 21 octaves
 * below the largest.  Numbers below 2^-126 may count as 0 on the way.
 * A non-finite
 * x, A or B gives non-finite sums where the definition's are (NaN possibly for
 * an infinity), for the tokens of that adapter and that row alone.
 * Deterministic for the same arguments.
 *
 * Range: rank a multiple of 8 up to GQ_MAX_LORA_RANK; K a multiple of 32;
 * rows a multiple of 4; K, rows <= 2^24; ldx, ldy0, ldy multiples of 4 and at
 * least the rows' length; M >= 0 (0: nothing to do); pointers 16-byte aligned
 * (scale, adapter, sequence: 4-byte).
 * Errors before the launches: GQ_ERR_FORMAT (type), GQ_ERR_NULL, GQ_ERR_ALIGN,
 * GQ_ERR_SHAPE, GQ_ERR_WORKSPACE; after them GQ_ERR_CUDA.
 * Two kernels are launched on `stream`, three for prompts (a sequence list and
 * 8 tokens or more a request on average, or 4 from 256 tokens on).
 * ------------------------------------------------------------------------ */
size_t gq_lora_workspace_bytes(int rank, int K, int M); /* 0 if out of range */
int gq_lora_add(const void *A, const void *B, int type, const float *scale, const int32_t *adapter,
                const int32_t *sequence_or_null, const float *X, long long ldx, const float *Y0, long long ldy0,
                float *Y, long long ldy, void *workspace, size_t workspace_bytes, int n_adapters, int rank, int rows,
                int K, int n_seq, int M, gq_stream_t stream);
int gq_lora_add_q8act(const void *A, const void *B, int type, const float *scale, const int32_t *adapter,
                      const int32_t *sequence_or_null, const int8_t *Xq, const float *dx, const float *Y0,
                      long long ldy0, float *Y, long long ldy, void *workspace, size_t workspace_bytes,
                      int n_adapters, int rank, int rows, int K, int n_seq, int M, gq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GQ_LORA_H */
