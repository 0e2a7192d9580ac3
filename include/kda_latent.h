/*
 * kda_latent.h -- latent attention, whose keys and values come from one shared
 * vector a token (a latent of 512 values and 64 values of positions), and the
 * paged cache of those vectors:
 *
 *   kda_latent_fwd, _bwd   the expanded form, with keys and values of every head:
 *                          prompts, training;
 *   kda_latent_decode      the absorbed form, over the cached vectors themselves:
 *                          generation, drafted tokens, pieces of prompts;
 *   kda_latent_store       tokens' vectors into the cache, normalised on the way;
 *   kda_page_assign        pages, slots and offsets of a serving step, from the
 *                          requests' lengths.
 *
 * The conventions are those of kda_layer.h: device pointers on the current HIP
 * device, work enqueued on `stream` without synchronising, status codes returned
 * before anything is enqueued, caller-owned workspaces (or, when NULL, one taken
 * and released on the stream), packed batches described by a device int64
 * cu_seqlens, strides in elements, written tensors contiguous and apart from
 * everything else that the call touches (KDA_ERR_OVERLAP).  Results do not depend
 * on the order in which workgroups run: the same call gives the same bits.  The order in
 * which a token's sums are added up goes by the sizes of the call, though (batch, heads,
 * tokens, sequences), so that their last bits may differ from those of a call of other sizes.
 * Sums are fp32 of probabilities that may stand a common factor of up to 2^8 (expanded form)
 * or 2^40 (absorbed form) above their value until the sum's end: values (cached latents) of up to
 * 2^56 in magnitude are safe, larger ones may come out infinite.
 *
 * Activations are bf16.  They are read 16 bytes at a time, at addresses that are
 * multiples of 16 bytes, with strides that are multiples of 8 elements
 * (KDA_ERR_ALIGN otherwise); written tensors of activations and caches begin at
 * such addresses too.  Token strides of 2^24 elements and more, other strides of
 * more than 2^40, more than 2^31 - 512 tokens, 65535 heads or 2^31 - 1 sequences are
 * refused (KDA_ERR_SHAPE), and scales that are not finite and above zero
 * (KDA_ERR_PARAM).
 */
#ifndef KDA_LATENT_H_
#define KDA_LATENT_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- the expanded form ---------------------------------------------------------
 * For head h, query i of a sequence's Lq and key j of its Lk, with the query's 192
 * values q = (q_n, q_p), the head's 256 values kv = (k, v) of a token and the 64
 * values k_pe that all heads share:
 *   s_ij = scale (q_n . k_j + q_p . k_pe_j),   with causal: only j <= i + Lk - Lq,
 *   lse_i = log sum_j e^s_ij,   out_i = sum_j e^(s_ij - lse_i) v_j.
 * A query that sees no key has out = 0 and lse = -infinity. */
typedef struct {
    int64_t B, T, Tk, H;                    /* queries and keys per batch row (packed: in all), heads */
    int64_t num_seqs;                       /* B, or the packed batch's sequences */
    int64_t q_stride_b, q_stride_t;         /* q [B, T, H, 192] */
    int64_t kv_stride_b, kv_stride_t;       /* kv [B, Tk, H, 256] */
    int64_t pe_stride_b, pe_stride_t;       /* k_pe [B, Tk, 64] */
    int64_t out_stride_b, out_stride_t;     /* gradient only: out [B, T, H, 128] */
    int64_t d_out_stride_b, d_out_stride_t; /* gradient only: d_out [B, T, H, 128] */
    float scale;                            /* finite, > 0 */
    int32_t causal;                         /* 0 or 1 */
    void *workspace;                        /* 256-byte aligned */
    size_t workspace_bytes;
    int64_t launch_piece;                   /* most workgroups of one launch, rounded up to a multiple of 8; 0: 2^23 */
} kda_latent_desc_t;

/* q, kv, k_pe: bf16; cu_seqlens, cu_seqlens_k: int64 [num_seqs + 1] or NULL:
 * with cu_seqlens (B = 1) sequence n has the queries cu_seqlens[n] .. and the keys
 * cu_seqlens_k[n] .. (cu_seqlens again when that is NULL, which takes T = Tk).
 * out: bf16 [B, T, H, 128]; lse: fp32 [B, T, H] or NULL.  Queries behind the last
 * sequence are left as they were.  A NaN or infinity in a key reaches the queries
 * that see it, and no others. */
kda_status_t kda_latent_fwd(const void *q, const void *kv, const void *k_pe, const int64_t *cu_seqlens,
                            const int64_t *cu_seqlens_k, void *out, float *lse, const kda_latent_desc_t *desc,
                            hipStream_t stream);
/* The gradient of <d_out, out>, from what the forward wrote: with
 * p_ij = e^(s_ij - lse_i) and ds_ij = scale p_ij (d_out_i . v_j - d_out_i . out_i),
 *   dq_i = sum_j ds_ij (k_j, k_pe_j),   dk_j = sum_i ds_ij q_n,   dv_j = sum_i p_ij d_out_i,
 *   dk_pe_j = sum over heads and i of ds_ij q_p.
 * out, d_out: bf16; lse: fp32.  dq: bf16 [B, T, H, 192]; dkv: bf16 [B, Tk, H, 256];
 * dk_pe: bf16 [B, Tk, 64].  p and ds enter the products as bf16, sums are fp32.  A
 * NaN or infinity in a token may reach the gradients of the other tokens of its
 * sequence's tiles of 64 queries and 64 keys. */
kda_status_t kda_latent_bwd(const void *q, const void *kv, const void *k_pe, const int64_t *cu_seqlens,
                            const int64_t *cu_seqlens_k, const void *out, const float *lse, const void *d_out, void *dq,
                            void *dkv, void *dk_pe, const kda_latent_desc_t *desc, hipStream_t stream);
/* Bytes of workspace the calls need (0 if the shapes are invalid; with B = 1 enough
 * for a packed batch too).  The forward needs some for packed batches and for few
 * queries with many keys. */
size_t kda_latent_fwd_workspace_size(const kda_latent_desc_t *desc);
size_t kda_latent_bwd_workspace_size(const kda_latent_desc_t *desc);

/* ---- the absorbed form -----------------------------------------------------------
 * The last T tokens of each of N sequences attend to the sequence's rows in the
 * cache.  A cached row is (c, r), 512 + 64 values, key and (c) value of all heads:
 *   s = scale (q_latent . c + q_pe . r),   out = sum softmax(s) c.
 * Token t of sequence n sees the rows 0 .. lengths[n] - T + t; row i is
 * cache[block_table[n][i / page_size]][i % page_size].  lengths count the T tokens
 * too.  A token that sees no row has out = 0 and lse = -infinity. */
typedef struct {
    int64_t N, T, H;
    int64_t pages, page_size;               /* cache [pages, page_size, 576]; page_size: a power of two up to 2^16 */
    int64_t max_pages;                      /* block_table [N, max_pages] */
    int64_t ql_stride_n, ql_stride_t, ql_stride_h;  /* q_latent [N, T, H, 512] */
    int64_t qp_stride_n, qp_stride_t, qp_stride_h;  /* q_pe [N, T, H, 64] */
    float scale;
    void *workspace;
    size_t workspace_bytes;
} kda_latent_decode_desc_t;

/* q_latent, q_pe, cache: bf16; lengths: int64 [N]; block_table: int32 [N, max_pages]
 * (entries behind a sequence's pages are not used).  out: bf16 [N, T, H, 512]; lse:
 * fp32 [N, T, H] or NULL.  Lengths are clamped to 0 .. max_pages page_size and pages
 * to 0 .. pages - 1, so that wrong ones give wrong results but no access outside the
 * tensors.  Cached rows at and behind a sequence's length are not used, whatever
 * they hold.  Refused (KDA_ERR_SHAPE) are N T H of more than 2^24, caches of 2^31 rows
 * and more, and N ceil(T H / 64) max_pages page_size of more than 2^43. */
kda_status_t kda_latent_decode(const void *q_latent, const void *q_pe, const void *cache, const int64_t *lengths,
                               const int32_t *block_table, void *out, float *lse, const kda_latent_decode_desc_t *desc,
                               hipStream_t stream);
/* Bytes of workspace kda_latent_decode needs (0 if the shapes are invalid). */
size_t kda_latent_decode_workspace_size(const kda_latent_decode_desc_t *desc);

/* ---- the cache ---------------------------------------------------------------------
 * For every token m with slots[m] in 0 .. num_slots - 1:
 *   cache[slots[m]] = (n_m, k_pe_m),   n = latent / sqrt(mean(latent^2) + eps) * weight
 * (n = latent without weight), rounded once to bf16.  Tokens with other slots are
 * not stored.  Slots have to differ: of tokens that share one, each value of the
 * row is that of one of them.  normed takes n of every token. */
typedef struct {
    int64_t tokens, num_slots;              /* cache [num_slots, 576] */
    int64_t latent_stride, pe_stride;       /* latent [tokens, 512], k_pe [tokens, 64] */
    int32_t weight_dtype;                   /* kda_dtype_t */
    float eps;                              /* with a weight: finite, >= 2^-126 */
} kda_latent_store_desc_t;

/* latent, k_pe, cache: bf16; weight: [512] or NULL; slots: int64 [tokens]; normed:
 * bf16 [tokens, 512] or NULL. */
kda_status_t kda_latent_store(const void *latent, const void *k_pe, const void *weight, const int64_t *slots, void *cache,
                              void *normed, const kda_latent_store_desc_t *desc, hipStream_t stream);

/* One serving step of N requests: request n holds lengths[n] tokens in the pages
 * block_table[n][0 .. ceil(lengths[n] / page_size) - 1] and gets new_tokens[n] more.
 *   1. A request with ended[n] gives its pages back: they are put on the stack
 *      free_pages (free_count of them in use), requests in order, each request's
 *      pages in order; its length becomes 0.  (Its new tokens begin the next request
 *      of that row.)
 *   2. Each request needs the pages its new tokens reach beyond those it has.
 *      Running through the requests, one is granted its tokens while the pages needed
 *      so far (by those refused too) do not pass those on the stack; a request that needs
 *      none always is.  A request that would pass max_pages pages or `tokens` rows is
 *      refused and counts no pages.  Pages come from the stack's end, requests in order.
 *   3. cu_seqlens: running sums of new_tokens, the packed batch of the new tokens;
 *      slots: page * page_size + offset of each of its rows, -1 for rows of refused
 *      requests and behind the last; lengths_out: the new lengths; granted: new_tokens
 *      where granted, else 0; free_count_out: pages left.
 * Negative numbers count as 0, lengths and totals are clamped to what the tables
 * hold (a stack that is full keeps no more pages, cu_seqlens ends at `tokens`). */
typedef struct {
    int64_t N, max_pages, page_size;        /* N up to 2^20; page_size: a power of two up to 2^16; N max_pages below 2^31 */
    int64_t stack;                          /* entries of free_pages */
    int64_t tokens;                         /* entries of slots */
    void *workspace;                        /* >= kda_page_workspace_size(), 256-byte aligned */
    size_t workspace_bytes;
} kda_page_desc_t;

/* lengths, new_tokens, lengths_out, granted: int64 [N]; ended: uint8 [N] or NULL;
 * block_table: int32 [N, max_pages], updated; free_pages: int32 [stack], updated;
 * free_count, free_count_out: int64 [1]; slots: int64 [tokens]; cu_seqlens: int64
 * [N + 1].  lengths_out may be lengths, and free_count_out free_count. */
kda_status_t kda_page_assign(const int64_t *lengths, const int64_t *new_tokens, const uint8_t *ended,
                             int32_t *block_table, int32_t *free_pages, const int64_t *free_count, int64_t *slots,
                             int64_t *cu_seqlens, int64_t *lengths_out, int64_t *granted, int64_t *free_count_out,
                             const kda_page_desc_t *desc, hipStream_t stream);
/* Bytes of workspace kda_page_assign needs (0 if the sizes are invalid). */
size_t kda_page_workspace_size(const kda_page_desc_t *desc);

#ifdef __cplusplus
}
#endif
#endif /* KDA_LATENT_H_ */
