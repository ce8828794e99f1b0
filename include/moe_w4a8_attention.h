/*
 * moe_w4a8_attention.h -- C ABI of the attention operators that run next to
 * the routed-expert layer in a serving step (CUDA, sm_103a).
 *
 * What they compute.  A ragged batch of B sequences: sequence b has
 * q_len[b] = q_start[b+1] - q_start[b] new tokens, rows q_start[b] .. of
 * the token arrays, and kv_len[b] tokens in all, the new ones among them.
 * Its i-th new token is at position p = kv_len[b] - q_len[b] + i.  Position
 * p of sequence b lives in the paged cache at row p % page_size of page
 * block_table[b][p / page_size].
 *
 *   append   n(x) = x * rsqrt(mean(x^2) + eps) * (w + weight_offset), per
 *            head of D components (left out if the weight is null);
 *            rotation of the head's first R components by position: pairs
 *            (i, i + R/2), or (2i, 2i + 1) if interleaved, i < R/2:
 *            (a, b) -> (a c - b s, b c + a s), c = cos_sin[p][i],
 *            s = cos_sin[p][R/2 + i];
 *            q_out[t] = rotated n(q[t]); cache row of t <- rotated n(k[t]),
 *            v[t].
 *   attend   out[t][h] = sum_j softmax_j(scale q[t][h] . K_j) V_j over the
 *            positions j <= p (and j > p - window, if window > 0) of t's
 *            sequence, K and V of head h / (Hq / Hkv);
 *            lse[t][h] = log sum_j exp(scale q[t][h] . K_j).
 *
 * Everything between the inputs and the single rounding of each output is
 * fp32, except that attend's weights are rounded to the element type as
 * operands of the matrix units (their sum is not).  A weight is exp(s - m)
 * for a reference m that may lag behind the row's maximum by a factor of up
 * to 2^8; in fp16 a weight below 2^-14 is rounded to a multiple of 2^-24, so
 * off by 2^-25 at most, and one below 2^-25 counts in the sum alone.
 *
 * Edge cases.  A row that sees no position (position below zero, kv_len 0)
 * gives out = 0 and lse = -inf; append treats a token at a position below
 * zero, or past the table of cosines, as padding: q_out = 0, nothing is
 * stored.  Tokens outside [q_start[0], q_start[B]) belong to no sequence
 * and give q_out = 0, out = 0, lse = -inf.  Cache rows past kv_len are
 * never part of a result, whatever they hold; a NaN or an infinity at a
 * position that a row does not see does not reach that row; a row that ends
 * with a NaN is for that taken again key by key, about half a microsecond
 * each, at the end of the call.  Any window of 2^31 - 1 or more is none.  A page id
 * outside [0, n_pages) is never dereferenced: append stores nothing there,
 * attend reads zeros.  Positions at table_width * page_size and beyond do
 * not exist.  q_start entries are clamped into [0, n_tokens].
 *
 * Layout.  Elements are bf16 or fp16.  Token arrays are [T][heads][D] with
 * any token and head strides (elements), D contiguous; the caches are
 * [pages][page_size][Hkv][D] with any page, row and head strides, D
 * contiguous (head-major pages are the same with other strides).  Every
 * address and stride is a multiple of 16 bytes.  q_start [B+1], kv_len [B]
 * and block_table [B][table_width] (contiguous) are int32 DEVICE arrays:
 * a step's lengths are never read on the host.
 *
 * Ownership, streams and errors as for moe_w4a8.h: caller-owned device
 * memory, nothing allocated, nothing kept between calls, no
 * synchronisation, host-detected errors returned before anything is
 * enqueued.  MOE_ERR_INVALID_ARG: a null or misaligned pointer or stride,
 * sizes below one, Hq not a multiple of Hkv, D not a multiple of 8, R odd
 * or above D, a scale that is not positive and finite, an unknown dtype.
 * MOE_ERR_UNSUPPORTED: D > 256, Hq > 1024, B > 2048, or Hq tokens at or
 * above 2^31 rows.
 */
#ifndef MOE_W4A8_ATTENTION_H
#define MOE_W4A8_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_DTYPE_BF16 0
#define MOE_DTYPE_FP16 1

/* A paged cache and the batch that uses it.  The arrays' contents may change
 * between calls (that is how a step advances); the addresses and sizes are
 * the caller's promise.  max_q_len and max_kv_len are the caller's bounds on
 * the batch's lengths, used on the host to choose a kernel and a launch
 * size: longer sequences give the same results, slower. */
typedef struct {
    int64_t n_seqs;       /* B */
    int64_t n_q_heads;    /* Hq */
    int64_t n_kv_heads;   /* Hkv */
    int64_t head_dim;     /* D */
    int64_t page_size;
    int64_t n_pages;
    int64_t table_width;  /* pages per row of block_table */
    int64_t max_q_len;
    int64_t max_kv_len;
    int64_t dtype;        /* MOE_DTYPE_* of every token array and cache */
    int64_t k_page_stride, k_row_stride, k_head_stride; /* elements */
    int64_t v_page_stride, v_row_stride, v_head_stride;
    void* k_cache;
    void* v_cache;
    const int32_t* block_table;
    const int32_t* q_start;
    const int32_t* kv_len;
} moe_kv_batch_t;

/* What append does to queries and keys. */
typedef struct {
    const float* cos_sin;   /* [table_rows][R]: R/2 cosines, then R/2 sines; null if R = 0 */
    int64_t table_rows;
    int64_t rot_dim;        /* R */
    int64_t interleaved;
    const float* q_weight;  /* [D], or null: no norm of the queries */
    const float* k_weight;  /* [D], or null: no norm of the keys */
    const int32_t* positions; /* [T] row of cos_sin for each token, or null: its position in the cache */
    float eps;
    float weight_offset;    /* 1 for weights held as their distance from one, else 0 */
} moe_head_prep_t;

/*
 * append, in one kernel.  q, k, v: [T][heads][D] with strides in elements
 * (for example the three parts of one fused projection's rows).  q_out may
 * be q itself with the same strides; apart from that the outputs must not
 * overlap the inputs.  T = 0 enqueues nothing.
 */
int moe_w4a8_kv_append(const moe_kv_batch_t* batch, const moe_head_prep_t* prep, int64_t n_tokens,
                       const void* q, int64_t q_token_stride, int64_t q_head_stride,
                       const void* k, int64_t k_token_stride, int64_t k_head_stride,
                       const void* v, int64_t v_token_stride, int64_t v_head_stride,
                       void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void* stream);

/* Bytes of workspace moe_w4a8_paged_attention needs for `batch` on the
 * current device, whatever the tokens (0 if `batch` is invalid). */
size_t moe_w4a8_paged_attention_workspace_size(const moe_kv_batch_t* batch);

/*
 * attend.  q, out: [T][Hq][D] with strides in elements; lse: float [T][Hq]
 * contiguous, or null.  window = 0: no window.  Two runs on the same inputs
 * give the same bits.  T = 0 enqueues nothing.
 */
int moe_w4a8_paged_attention(const moe_kv_batch_t* batch, int64_t n_tokens,
                             const void* q, int64_t q_token_stride, int64_t q_head_stride,
                             void* out, int64_t out_token_stride, int64_t out_head_stride,
                             float* lse, float scale, int64_t window,
                             void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_W4A8_ATTENTION_H */
