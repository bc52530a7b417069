/*
 * moe_attention.h -- C ABI of the attention operators of libmoe_nvfp4.so: a
 * paged cache of keys and values, the attention that reads it, and attention
 * over whole prompts. Next to the routed-expert step of moe_nvfp4.h they are
 * the other half of a decoder block in serving.
 *
 * Conventions are those of moe_nvfp4.h: device pointers owned by the caller
 * (16-byte aligned), nothing allocated, every call asynchronous on `stream`,
 * status codes checked on the host before anything is enqueued, results
 * deterministic, and a token's output independent of the other sequences of
 * its call. What only the device can see (a sequence id or page id out of
 * range, a pool without enough free pages) leaves the sequence or the call
 * that it concerns undone and is reported by moe_nvfp4_check_status
 * (MOE_ERR_INVALID, MOE_ERR_PAGES); no index from device memory is followed
 * unchecked. Tensors are bf16 or fp16 (`dtype`), 16-bit patterns.
 *
 * The math (one sequence, head h of the queries, kv head h / (heads_q /
 * heads_kv)):
 *   s_ij = scale * sum_d q[i, d] k[j, d]       over the keys j that i sees
 *   out[i] = sum_j exp(s_ij - lse_i) v[j],     lse_i = log sum_j exp(s_ij)
 * A query that sees no key gives out = 0 and lse = -inf; so do all queries of
 * a sequence whose id, length (past max_pages pages) or a page id within its
 * length is out of range (MOE_ERR_INVALID). Keys and values that
 * a query does not see have no influence on it, NaN and infinities included.
 * Scores, the running maximum and sum, and the sum over the values are held
 * in fp32; the weights exp(s_ij - lse_i) are rounded to the tensors' type for
 * the product with the values (in fp16 those below 2^-32 of a row's largest
 * are 0 there).
 */
#ifndef MOE_ATTENTION_H
#define MOE_ATTENTION_H

#include "moe_nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MOE_BF16 = 0, MOE_FP16 = 1 };

/* Rows of heads: element (token t, head h, d) at data[t * token_stride + h *
 * head_stride + d]. Strides are in elements, non-negative multiples of 8. */
typedef struct {
  void* data;
  long long token_stride;
  long long head_stride;
} moe_heads_t;

/* A paged cache. pages: [planes, n_pages, page_size, heads_kv, head_dim],
 * contiguous; plane 2l holds the keys of layer l, plane 2l+1 its values. One
 * table serves all layers. Sequence s (a row of the table) has length[s]
 * tokens in held[s] = ceil(length[s] / page_size) pages: token p is row p %
 * page_size of page table[s, p / page_size]; entries from held[s] on are -1.
 * refs[page] counts the table entries that name the page (0: free). A fresh
 * cache has table -1 and the other three 0. */
typedef struct {
  void* pages;
  int planes, n_pages, page_size, heads_kv, head_dim, dtype;
  int32_t* table;  /* [max_seqs, max_pages] */
  int32_t* length; /* [max_seqs] */
  int32_t* held;   /* [max_seqs] */
  int32_t* refs;   /* [n_pages] */
  int max_seqs, max_pages;
} moe_kv_cache_t;

#define MOE_KV_MAX_CALL 4096 /* sequences of one upkeep call at most (else MOE_ERR_INVALID) */

/* Device scratch of moe_kv_extend, moe_kv_keep and moe_kv_compact on this
 * cache: bytes (256-byte aligned, any contents). 0 for an invalid cache. */
size_t moe_kv_workspace_size(const moe_kv_cache_t* cache /* host */);

/* Grows sequence seqs[i] by add[i] >= 0 tokens (i < n; the seqs distinct).
 * New pages are the free ones of lowest id, handed out in order of (i, place
 * in the sequence). Where the sequence's last page is partly filled and held
 * by others too, it first gets a page of its own (before its other new
 * pages) with the rows in use copied, in all planes. All or nothing: a bad
 * argument, more than max_pages pages, or too few free pages
 * (MOE_ERR_PAGES) leave the cache as it was. */
int moe_kv_extend(const moe_kv_cache_t* cache, const int32_t* seqs, const int32_t* add, int n, void* workspace,
                  size_t ws_bytes, cudaStream_t stream);

/* Writes the keys and values of each sequence's last tokens in one layer:
 * rows cu[i] .. cu[i+1] of k and v ([total, heads_kv] rows of heads) are the
 * last cu[i+1] - cu[i] tokens of seqs[i] (moe_kv_extend made room). A row
 * whose page is shared or missing is not written (MOE_ERR_INVALID). */
int moe_kv_append(const moe_kv_cache_t* cache, int layer, const int32_t* seqs, const int32_t* cu, int n, int total,
                  const moe_heads_t* k, const moe_heads_t* v, cudaStream_t stream);

/* The empty sequence dst[i] becomes src[i]: it shares all of its pages. Each
 * pair is checked by itself: a dst that is not empty, repeats, or is a src of
 * the call too is left alone (MOE_ERR_INVALID). */
int moe_kv_fork(const moe_kv_cache_t* cache, const int32_t* src, const int32_t* dst, int n, cudaStream_t stream);

/* Cuts sequence seqs[i] to at most new_len[i] >= 0 tokens and lets go of the
 * pages past them; 0 frees the sequence. */
int moe_kv_truncate(const moe_kv_cache_t* cache, const int32_t* seqs, const int32_t* new_len, int n,
                    cudaStream_t stream);

/* Of the last drafted[i] tokens of seqs[i], keeps those at keep[i, 0 ..
 * kept[i]) (strictly ascending places among the drafted, row i of [n,
 * max_keep]): their rows move together in all planes, behind the tokens before
 * the drafted ones, and the sequence is cut after them. A sequence whose
 * arguments are bad, or whose drafted rows lie in a shared page, is left
 * alone (MOE_ERR_INVALID). */
int moe_kv_keep(const moe_kv_cache_t* cache, const int32_t* seqs, const int32_t* drafted, const int32_t* keep,
                int max_keep, const int32_t* kept, int n, void* workspace, size_t ws_bytes, cudaStream_t stream);

/* Copies page src[i] to page dst[i] in all planes; tables and counts stay.
 * The dst must be distinct and none of them a src (of another pair); any
 * number of pairs. */
int moe_kv_copy_pages(const moe_kv_cache_t* cache, const int32_t* src, const int32_t* dst, int n,
                      cudaStream_t stream);

/* Moves the pages in use to the front of the pool: with U pages in use, the
 * k-th used page of id >= U goes to the k-th free page of id < U (all planes,
 * tables and counts follow). Afterwards pages U .. n_pages-1 are free. */
int moe_kv_compact(const moe_kv_cache_t* cache, void* workspace, size_t ws_bytes, cudaStream_t stream);

/* Tree masks from parents: drafted token t of sequence i (packed rows cu[i] ..
 * cu[i+1], total rows) has parent parents[t], the place of an earlier token
 * of its tree or -1. Row t of mask [total, mask_words] gets bit b of word w set
 * where the token is, or descends from, token 32 w + b of its tree. A parent
 * that is not an earlier token ends the walk there (MOE_ERR_INVALID unless
 * -1); a tree of more than 32 * mask_words tokens gets zeros
 * (MOE_ERR_INVALID). */
int moe_tree_mask(const int32_t* parents, const int32_t* cu, int n, int total, int32_t* mask, int mask_words,
                  cudaStream_t stream);

/* Causal attention over whole prompts, n sequences packed one after the
 * other: queries cu_q[i] .. cu_q[i+1] of q [total_q, heads_q], keys and values
 * cu_k[i] .. cu_k[i+1] of k and v [total_k, heads_kv]. Query a of a sequence of
 * nq queries and nk keys sees its keys 0 .. a + nk - nq (the queries are the
 * last nq tokens). out [total_q, heads_q] rows of heads, lse [total_q,
 * heads_q] fp32 or null. head_dim % 8 == 0, head_dim <= 128, heads_q a
 * multiple of heads_kv with at most 128 query heads per kv head, total_q *
 * heads_q <= 2^30, total_k <= 2^31 - 128 (else MOE_ERR_SHAPE); scale finite and
 * > 0. Rows past cu_q[n] are left alone. Offsets outside the tensors are cut to
 * them; a sequence whose offsets run backwards is empty. Where more than 256
 * sequences have more queries together than total_q the call is left undone
 * (MOE_ERR_INVALID). */
int moe_attention_prompt(const moe_heads_t* q, const moe_heads_t* k, const moe_heads_t* v, const int32_t* cu_q,
                         const int32_t* cu_k, int n, int total_q, int total_k, int heads_q, int heads_kv,
                         int head_dim, int dtype, float scale, const moe_heads_t* out, float* lse,
                         cudaStream_t stream);

/* Attention of drafted tokens over the cache: rows cu_q[i] .. cu_q[i+1] of q
 * [total_q, heads_q] are the last tokens of sequence seqs[i], whose keys and
 * values (theirs among them) are in layer `layer` of the cache. Every query
 * sees the tokens before the drafted ones. Among the drafted: with mask null
 * those up to itself (a chain; one token a sequence is a plain decode step),
 * else those with a set bit in its row of mask [total_q, mask_words] (bit b of
 * word w: drafted token 32 w + b; tokens past the row's words are not seen).
 * Long sequences are cut into pieces whose partial results are joined in a
 * fixed order; the cut depends on the sequence's own length and rows only.
 * workspace: moe_attention_cached_workspace_size() bytes, 256-byte aligned,
 * any contents. out, lse, limits as moe_attention_prompt. */
size_t moe_attention_cached_workspace_size(const moe_kv_cache_t* cache, int n, int total_q, int heads_q);
int moe_attention_cached(const moe_heads_t* q, const moe_kv_cache_t* cache, int layer, const int32_t* seqs,
                         const int32_t* cu_q, int n, int total_q, int heads_q, const int32_t* mask, int mask_words,
                         float scale, const moe_heads_t* out, float* lse, void* workspace, size_t ws_bytes,
                         cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ATTENTION_H */
