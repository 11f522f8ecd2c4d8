/*
 * mbrs_sequence.h -- C ABI of the sequence attention calls on GB300 (sm_103a):
 * attention over packed prompts of different lengths, attention of new tokens
 * over a paged key/value cache, and the append that writes new keys and values
 * to that cache with their position rotation.  All take grouped heads: query
 * head h reads key/value head h / (heads / kv_heads).
 *
 * A batch of sequences.  The new tokens of all sequences are packed along one
 * axis: sequence b owns the rows q_starts[b] .. q_starts[b + 1] - 1 of q, k, v
 * and o.  n_b = q_starts[b + 1] - q_starts[b] may be zero.  Rows from
 * q_starts[batch] on belong to no sequence: no call writes them.
 *
 * The operation, for query i < n_b of sequence b with c_b keys (packed
 * prompts: c_b = n_b; paged: c_b = kv_lens[b], the new tokens included, the
 * last n_b of them being the new ones):
 *
 *     x_j   = sm_scale * sum_d q[i,d] k[j,d]     kept: j < c_b, and with causal
 *                                                != 0 also j <= c_b - n_b + i
 *     o[i]  = sum_j softmax_j(x_j) v[j]          over the kept keys
 *     lse   = log sum_j exp(x_j)                 (natural log, optional output)
 *
 * A query that keeps no key gets o = 0 and lse = -inf.  Keys outside the kept
 * ones never reach a query's result, whatever their bits are (values that are
 * infinite or NaN included).  An infinite or NaN value of a key that is kept makes
 * its element of the result infinite or NaN, however small the key's weight.
 *
 * The cache.  k and v are arrays of pages: element (page, slot, head, d) lies
 * at page * page_stride + slot * token_stride + head * head_stride + d, so both
 * the order [page, slot, head, d] and the order [page, head, slot, d] are taken.
 * Position p of sequence b lies in page page_table[b * table_stride +
 * p / page_size], slot p % page_size.  Sequences may share pages.  Entries of
 * the table past a sequence's last page are not read.  For attention a page
 * index outside [0, pages) reads as a page of zeros; the append writes nothing
 * there.
 *
 * Values read on the device (q_starts, kv_lens, page_table) cannot be checked
 * before the launch.  Whatever they hold, no call reads or writes outside the
 * buffers it was given: q_starts are clamped to [0, tokens] and a sequence that
 * ends before it starts is empty; attention clamps kv_lens to [0, max_pages *
 * page_size], and the append, which takes positions from them as they are, drops
 * the keys and values of positions that have no page.  They may change between launches (and between the replays of a
 * captured graph) with the sizes below kept.
 *
 * Types: SOFTMAX_F16 or SOFTMAX_BF16; head_dim 64 or 128; heads a multiple of
 * kv_heads, at most 128 query heads to one key/value head; page_size a multiple
 * of 8.  Arithmetic: products of the 16-bit inputs accumulated in fp32, exp in
 * fp32, the probabilities rounded to the input type for the second product (in
 * fp16 with all its bits down to 2^-21 of a row's largest, and none below 2^-32),
 * o accumulated in fp32, divided by the fp32 normaliser and rounded once.
 *
 * Ownership: the caller owns every buffer and the stream.  The calls are
 * asynchronous on `stream`, allocate nothing on the device, keep nothing from
 * one call to the next, and may be captured into a CUDA graph.  The workspace
 * needs no initialisation; calls that share one must not run at the same time
 * (two captured graphs that may run together need one each).
 *
 * Every base pointer is 16-byte aligned (int32 arrays and lse 4-byte), every
 * stride a multiple of 8 elements, the last dimension contiguous.
 *
 * Errors (checked on the host before any launch):
 *   SOFTMAX_ERR_ARG         args NULL, causal not 0 or 1, sm_scale not finite and
 *                           > 0, fields of the other call set, rotary sizes
 *   SOFTMAX_ERR_SHAPE       negative sizes, heads not a multiple of kv_heads, sizes
 *                           beyond the index range (2^31 - 1 rows, keys or pages)
 *   SOFTMAX_ERR_DTYPE       dtype not a softmax_dtype_t
 *   SOFTMAX_ERR_UNSUPPORTED SOFTMAX_F32, head_dim not 64 or 128, more than 128 query
 *                           heads to a key/value head, page_size not a multiple of 8
 *   SOFTMAX_ERR_STRIDE      a stride not a multiple of 8 elements, smaller than the
 *                           rows it separates, or 2^40 bytes and more
 *   SOFTMAX_ERR_NULL        a NULL pointer while there is work to do
 *   SOFTMAX_ERR_ALIGN       a pointer not aligned as above
 *   SOFTMAX_ERR_OVERLAP     an output overlaps an input, another output or the
 *                           workspace (the append's q_out may be q itself)
 *   SOFTMAX_ERR_SCRATCH_LIMIT  the workspace is smaller than the call needs
 *   SOFTMAX_ERR_CUDA        a CUDA call or launch failed
 * A call with no rows (tokens == 0 or batch == 0) returns SOFTMAX_OK without a
 * launch.  A bounded wait inside a kernel that runs out is reported by
 * softmax_check_device_error as SOFTMAX_ERR_TIMEOUT; what that call leaves in o
 * and lse is undefined.
 */
#ifndef MBRS_SEQUENCE_H
#define MBRS_SEQUENCE_H

#include "mbrs_softmax.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Strides are in elements.  heads, kv_heads, head_dim, dtype: see above. */
typedef struct {
    const void *q;           /* [tokens, heads, head_dim] */
    const void *k, *v;       /* packed: [tokens, kv_heads, head_dim]; paged: the cache */
    void *o;                 /* [tokens, heads, head_dim] */
    float *lse;              /* [tokens, heads] contiguous, or NULL */
    const int32_t *q_starts; /* batch + 1 row offsets */
    const int32_t *kv_lens;  /* paged: batch key counts; packed: NULL */
    const int32_t *page_table; /* paged: [batch, max_pages]; packed: NULL */
    int64_t q_token_stride, q_head_stride;
    int64_t k_page_stride, k_token_stride, k_head_stride; /* packed: page strides 0 */
    int64_t v_page_stride, v_token_stride, v_head_stride;
    int64_t o_token_stride, o_head_stride;
    int64_t table_stride;
    int64_t tokens, batch, heads, kv_heads, head_dim;
    int64_t pages, page_size, max_pages; /* packed: 0 */
    int dtype, causal;
    float sm_scale;
} softmax_sequence_args_t;

/*
 * softmax_attention_varlen_fwd -- attention over packed prompts.
 * softmax_attention_paged_fwd  -- attention of new tokens over the paged cache
 *                                 (their own keys and values are in it already).
 *   workspace        device memory, 256-byte aligned, of at least
 *                    softmax_sequence_workspace_bytes(args) bytes
 */
int softmax_attention_varlen_fwd(const softmax_sequence_args_t *args, void *workspace, int64_t workspace_bytes,
                                 cudaStream_t stream);
int softmax_attention_paged_fwd(const softmax_sequence_args_t *args, void *workspace, int64_t workspace_bytes,
                                cudaStream_t stream);

/*
 * The workspace bytes of either call for these sizes on the current device
 * (paged when page_table is not NULL), or a negated softmax_status_t on bad
 * sizes.  Pointers other than page_table are not looked at.
 */
int64_t softmax_sequence_workspace_bytes(const softmax_sequence_args_t *args);

typedef struct {
    const void *k, *v;       /* [tokens, kv_heads, head_dim]: the new keys (not rotated) and values */
    void *k_cache, *v_cache; /* [pages, page_size, kv_heads, head_dim] by their strides */
    const void *q;           /* [tokens, heads, head_dim] queries to rotate as well, or NULL */
    void *q_out;             /* [tokens, heads, head_dim]; may be q; NULL when q is */
    const int32_t *q_starts, *kv_lens, *page_table;
    const float *inv_freq;   /* rotary_dim / 2 angles per position, or NULL: no rotation */
    int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride;
    int64_t q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride;
    int64_t k_cache_page_stride, k_cache_token_stride, k_cache_head_stride;
    int64_t v_cache_page_stride, v_cache_token_stride, v_cache_head_stride;
    int64_t table_stride;
    int64_t tokens, batch, heads, kv_heads, head_dim; /* heads: 0 when q is NULL */
    int64_t pages, page_size, max_pages;
    int64_t rotary_dim;      /* leading elements of a head that are rotated: a multiple of 16, at most head_dim; 0
                                without inv_freq */
    int interleaved;         /* 0: element d pairs with d + rotary_dim / 2; 1: 2d pairs with 2d + 1 */
    int dtype;
} softmax_append_args_t;

/*
 * softmax_kv_cache_append -- for new token i of sequence b, whose position is
 * p = kv_lens[b] - n_b + i (kv_lens counts the new tokens): its value and its
 * rotated key go to slot p of the sequence's pages, and its rotated query to
 * q_out.  Pair m of a head turns by the angle p * inv_freq[m],
 *     (x, y) -> (x cos - y sin, y cos + x sin),
 * the angle reduced in 64 bits, the rotation in fp32, rounded once; elements
 * from rotary_dim on are copied.  A token whose position is negative or has no
 * page in [0, pages) writes no cache (its query is rotated all the same).  Two
 * tokens of one call on the same slot leave elements of either there, in pieces
 * of 8.
 */
int softmax_kv_cache_append(const softmax_append_args_t *args, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MBRS_SEQUENCE_H */
