/*
 * gq_kv.h -- a paged key/value cache in Q8_0 blocks, and the attention of
 * new tokens over it (part of libgq; conventions as in gq.h).
 *
 * Three operators share one description of a batch:
 *   append     quantizes new keys and values into the cache's pages,
 *   read       gives them back in a floating type,
 *   attention  runs the new tokens' queries against everything cached; one
 *              new token per sequence is its decode form.
 *
 * The batch.  `n_seq` sequences; the new tokens of all of them are the
 * `n_tokens` rows of the token arrays, sequence b owning rows
 * q_start[b] .. q_start[b + 1] - 1 (int32[n_seq + 1], non-decreasing,
 * q_start[0] = 0, q_start[n_seq] = n_tokens; a sequence may own none).
 * kv_len[b] (int32) is how many tokens of sequence b are cached, the new
 * ones included: they are its last positions, row q_start[b] + i at position
 * kv_len[b] - (q_start[b + 1] - q_start[b]) + i.  block_table
 * (int32[n_seq][max_pages]) names the page that holds positions
 * page_tokens * k .. page_tokens * (k + 1) - 1 in entry k.  Entries past a
 * sequence's last page, and those below an attention window, are not read.
 * The three lists are device memory, 4-byte aligned; nothing of them is read
 * on the host, so a call can be captured in a graph and replayed with other
 * lengths and pages.
 *
 * The cache.  gq_kv_cache_bytes bytes of device memory: n_pages pages of
 * page_tokens tokens (a multiple of 16), each holding for every kv head, in
 * order, one record of 34 * head_dim bytes for every 16 tokens:
 *   16 * head_dim bytes   K codes: block b (32 elements) of token t in the
 *                         32-byte unit t * nb + (b ^ key(t)),
 *   head_dim bytes        K scales, fp16 [16 tokens][nb],
 *   16 * head_dim bytes   V codes: for each group g of four tokens and each
 *                         element e one 4-byte word holding the four tokens'
 *                         codes; the 16-byte chunk e / 4 of group g is stored
 *                         at chunk position (e / 4) ^ (2 g),
 *   head_dim bytes        V scales, fp16 [nb][16 tokens],
 * with nb = head_dim / 32, key(t) = (t & 1) | ((t >> 1) & 2) for nb > 2 and
 * (t >> 2) & 1 for nb = 2; a code byte is code XOR 0x80.  The two exclusive
 * ors are there so that the attention kernels, which copy whole records into
 * shared memory, read the codes without bank conflicts; keys are contiguous
 * along the head (the contraction of q k) and values along the tokens (the
 * contraction of p v).
 *
 * Token arrays (K, V, Q, O) have rows of heads * head_dim contiguous
 * elements and a row stride in elements (so that q, k and v may be parts of
 * one projection's rows).  Pointers are 16-byte aligned and strides whole
 * multiples of 16 bytes.  `type` is the element type of all token arrays of
 * a call.
 *
 * Range: head_dim 64, 128 or 256; heads a multiple of kv_heads; page_tokens
 * a multiple of 16, at most 4096; max_pages * page_tokens at most 2^28;
 * n_tokens = 0 is a valid call that does nothing (the token arrays may then be
 * null).
 * Errors before any launch: GQ_ERR_NULL, GQ_ERR_ALIGN, GQ_ERR_SHAPE,
 * GQ_ERR_FORMAT for an unknown type, GQ_ERR_WORKSPACE; after it GQ_ERR_CUDA.
 * What only the device can see -- a page number outside 0 .. n_pages - 1, a
 * kv_len beyond max_pages * page_tokens, a q_start beyond n_tokens, an append
 * at a negative position -- is never followed out of bounds: the tokens
 * concerned are not written (append), read as zeros (read) or not attended
 * to (attention), and the device status (gq_device_status) becomes
 * GQ_ERR_SHAPE.  All other rows keep the positions that the lists give them,
 * and nothing else that is cached changes.
 */
#ifndef GQ_KV_H
#define GQ_KV_H

#include "gq.h"

/* Sources: "Metal kernel capability table (Phase B ground truth)", section 3
 * (attention over a cache, append fused with it) and section 9 (legal
 * dimensions are checked at dispatch); "Gemma 4 M4 Max kernel roadmap", K3 and
 * K5 (split attention over long caches, grouped heads, sliding windows). */

#ifdef __cplusplus
extern "C" {
#endif

enum {
    GQ_TYPE_F32 = 0,
    GQ_TYPE_F16 = 1,
    GQ_TYPE_BF16 = 2
};

/* Bytes of a cache of n_pages pages (0 if an argument is out of range). */
size_t gq_kv_cache_bytes(int n_pages, int page_tokens, int kv_heads, int head_dim);

/* ---------------------------------------------------------------------------
 * Write the new tokens' keys and values.  For every 32-block x of a head:
 *   d = fp16(min(max|x| / 127, 515.5))   (the f32 quotient as in
 *       gq_quantize_q8_0, then one rounding: the scale is kept in 11 bits),
 *   q = clamp(round_half_away(x / d), -127, 127) with the f32 quotient by the
 *       stored d; q = 0 when d = 0.
 * 515.5 keeps d * q within fp16: larger magnitudes saturate at +-65468.5.  An
 * infinity saturates likewise; a NaN does not enter max|x| and is stored as
 * -127 (0 in a block of nothing else).  Bit-exact.
 *   K, V: row stride ldk, ldv elements, read only.
 * Only the new tokens' codes and scales are written.
 * ------------------------------------------------------------------------ */
int gq_kv_append_q8_0(const void *K, long long ldk, const void *V, long long ldv, int type, void *cache,
                      const int32_t *block_table, const int32_t *kv_len, const int32_t *q_start, int n_pages,
                      int max_pages, int page_tokens, int kv_heads, int head_dim, int n_seq, int n_tokens,
                      gq_stream_t stream);

/* ---------------------------------------------------------------------------
 * The cached keys and values of the tokens that the batch names (the last
 * q_start[b + 1] - q_start[b] positions of every sequence): d * q, rounded
 * once to `type`.  K and V are overwritten.
 * ------------------------------------------------------------------------ */
int gq_kv_read_q8_0(const void *cache, const int32_t *block_table, const int32_t *kv_len, const int32_t *q_start,
                    void *K, long long ldk, void *V, long long ldv, int type, int n_pages, int max_pages,
                    int page_tokens, int kv_heads, int head_dim, int n_seq, int n_tokens, gq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Causal attention of the new tokens.  The query of head h at position p
 * reads kv head h / (heads / kv_heads) at the positions
 *   max(0, p - window + 1) <= j <= p     (window 0: 0 <= j <= p),
 *   s_j = scale * (q . k_j),  s_j <- softcap * tanh(s_j / softcap) if
 *   softcap > 0,  o = sum_j exp(s_j) v_j / sum_j exp(s_j),
 * with k_j, v_j the cached values d * q.  A query with no position to read
 * (p < 0, or a sequence of length 0) gives zeros.
 *   Q, O: row stride ldq, ldo elements; O is overwritten.  scale and softcap
 *   finite, window >= 0.
 * Accuracy: with A = sum_j w_j |v_j| (w_j the softmax weights, element by
 * element) and Z the row's largest |scale| * sum_i |q_i k_ji|,
 *   GQ_TYPE_F32:  |error| <= (2.1 * 2^-20 Z + 2^-16) A.  Operands of 22 bits or
 *     more, f32 sums.  In the 2-norm, where roundings average, within 1e-5 of
 *     the result for scores of ordinary size (Z up to about 16).
 *   16-bit types: |error| <= (2.1 * 2^-10 Z + 2^-10 + 2^-27 N) A for N visible
 *     tokens, and the rounding of O.  Keys and values d * q and the weights may
 *     be rounded to 11 bits; sums are f32, truncated by the tensor core (N).
 *     Rounded keys shift a score by some 2^-12 of its terms, so large scores
 *     cost accuracy: with scores of standard deviation 2.5 the error in the
 *     2-norm is 6e-4 before O is rounded.  For less, use GQ_TYPE_F32.
 * Beside that, tokens whose w_j max|v_j| is below 2^-26 of the row's largest may
 * count as 0.
 * Range: |q| < 2^100, and |scale * (q . k_j)| <= 2^19.
 *   workspace: device memory, 16-byte aligned, at least
 *   gq_kv_attention_workspace_bytes bytes.  ZERO-FILL IT ONCE before its
 *   first use; every completed call leaves it ready for the next.  Zero-fill it
 *   again after GQ_ERR_TIMEOUT: a call whose waits gave up leaves counts in it.
 *   Two calls that may run concurrently must not share it.
 * ------------------------------------------------------------------------ */
size_t gq_kv_attention_workspace_bytes(int heads, int kv_heads, int head_dim); /* 0 if out of range */
int gq_kv_attention_q8_0(const void *Q, long long ldq, const void *cache, const int32_t *block_table,
                         const int32_t *kv_len, const int32_t *q_start, void *O, long long ldo, int type, float scale,
                         float softcap, int window, void *workspace, size_t workspace_bytes, int heads, int n_pages,
                         int max_pages, int page_tokens, int kv_heads, int head_dim, int n_seq, int n_tokens,
                         gq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GQ_KV_H */
