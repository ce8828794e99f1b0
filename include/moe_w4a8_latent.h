/*
 * moe_w4a8_latent.h -- C ABI of latent attention over a paged cache: the
 * attention operators of layers that keep one vector per token for all heads
 * (CUDA, sm_103a).  They stand beside those of moe_w4a8_attention.h, whose
 * ragged batch, pages, edge cases and error rules are theirs too.
 *
 * What they compute.  A cache row holds a token's latent vector c (Dc
 * components) and behind it a key part of R components that carries the
 * position.  With the products that expand c into the heads' keys and values
 * absorbed into the queries and the output projection, a row is the key of
 * every head and its latent part is every head's value:
 *
 *   append  c' = c * rsqrt(mean(c^2) + eps) * (w + weight_offset) (c itself if
 *           the weight is null); the key part and every head's R rotated query
 *           components are turned by position as in moe_w4a8_kv_append;
 *           cache row of t <- (c', turned k_rot[t]); q_rot_out[t] = turned
 *           q_rot[t].
 *   attend  out[t][h] = sum_j softmax_j(scale q[t][h] . x_j) x_j[0 .. Dc) over
 *           the positions j <= p of t's sequence, x_j the cache row of j
 *           (Dc + R components, as q has);
 *           lse[t][h] = log sum_j exp(scale q[t][h] . x_j).
 *
 * Rounding as in moe_w4a8_attention.h: fp32 between the inputs and the single
 * rounding of each output, except attend's weights, which are rounded to the
 * element type as operands of the matrix units (their sum is not).  In fp16 the
 * weights are 2^7 exp(s - m), m at most the row's maximum and at most a factor of
 * 2^8 behind it, so that what is rounded to a multiple of 2^-24 is a weight 2^-21
 * below the largest, and what counts in the sum alone one 2^-32 below it.  The
 * edge cases are the same: rows that see nothing give out = 0 and lse = -inf,
 * tokens of no sequence too, append takes a token below position zero or past
 * the table of cosines as padding (q_rot_out = 0, nothing stored), rows past
 * kv_len never reach a result, a NaN or an infinity at a position reaches the
 * rows that see it and no others (a row that ends with a NaN is taken again key
 * by key, about a microsecond each, at the end of the call), a bad page id is
 * never dereferenced.  A row all of whose scores are -inf has weights of zero:
 * lse = -inf, out = 0, a NaN in the components where it sees an infinity or a NaN.
 *
 * Layout.  bf16 or fp16.  The cache is [pages][page_size][Dc + R] with any page
 * and row strides, a row contiguous.  Token arrays have any token and head
 * strides, the components contiguous.  Every address and stride is a multiple
 * of 16 bytes.  q_start, kv_len and block_table are int32 DEVICE arrays whose
 * contents are never read on the host.
 *
 * Ownership, streams and errors as for moe_w4a8.h.  MOE_ERR_INVALID_ARG: a null
 * or misaligned pointer or stride, sizes below one, Dc or R not a multiple of
 * 8, a row stride below Dc + R, a scale that is not positive and finite, an
 * unknown dtype, a prep that does not fit (see below).  MOE_ERR_UNSUPPORTED:
 * Dc > 512, R > 64, a page size that is not a multiple of 8, n_heads > 1024,
 * B > 2048, more than 2^31 - 513 rows (tokens times heads), page and row strides
 * of 2^39 elements and more.
 */
#ifndef MOE_W4A8_LATENT_H
#define MOE_W4A8_LATENT_H

#include "moe_w4a8_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A paged cache of latent rows and the batch that uses it; see moe_kv_batch_t. */
typedef struct {
    int64_t n_seqs;      /* B */
    int64_t n_heads;     /* of the queries */
    int64_t latent_dim;  /* Dc */
    int64_t rot_dim;     /* R, 0 for rows without a key part */
    int64_t page_size;
    int64_t n_pages;
    int64_t table_width; /* pages per row of block_table */
    int64_t max_q_len;
    int64_t max_kv_len;
    int64_t dtype;       /* MOE_DTYPE_* of every token array and the cache */
    int64_t page_stride, row_stride; /* elements */
    void* cache;
    const int32_t* block_table;
    const int32_t* q_start;
    const int32_t* kv_len;
} moe_latent_batch_t;

/*
 * append, in one kernel.  prep: k_weight [Dc] is the weight of the latent
 * vector's norm (null: no norm), q_weight must be null, rot_dim must be the
 * batch's.  latent [T][Dc], k_rot [T][R] with a token stride each (for example
 * two parts of one projection's rows), q_rot and q_rot_out [T][n_heads][R].
 * With R = 0 the last three are not looked at.  q_rot_out may be q_rot itself
 * with the same strides; apart from that the outputs must not overlap the
 * inputs.  T = 0 enqueues nothing.
 */
int moe_w4a8_latent_append(const moe_latent_batch_t* batch, const moe_head_prep_t* prep, int64_t n_tokens,
                           const void* latent, int64_t latent_token_stride, const void* k_rot, int64_t k_rot_token_stride,
                           const void* q_rot, int64_t q_rot_token_stride, int64_t q_rot_head_stride,
                           void* q_rot_out, int64_t q_rot_out_token_stride, int64_t q_rot_out_head_stride, void* stream);

/* Bytes of workspace moe_w4a8_latent_attention needs for `batch` on the current
 * device, whatever the tokens (0 if `batch` is invalid). */
size_t moe_w4a8_latent_attention_workspace_size(const moe_latent_batch_t* batch);

/*
 * attend.  q: [T][n_heads][Dc + R], out: [T][n_heads][Dc], with strides in
 * elements; lse: float [T][n_heads] contiguous, or null.  out and lse must not
 * overlap q or the cache (a row that is taken again reads its query at the end of
 * the call).  Two runs on the same inputs give the same bits.  T = 0 enqueues
 * nothing.
 */
int moe_w4a8_latent_attention(const moe_latent_batch_t* batch, int64_t n_tokens,
                              const void* q, int64_t q_token_stride, int64_t q_head_stride,
                              void* out, int64_t out_token_stride, int64_t out_head_stride,
                              float* lse, float scale, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_W4A8_LATENT_H */
