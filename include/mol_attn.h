/*
 * mol_attn.h -- the attention half of a decoder layer, on GB300 (sm_103a).
 *
 * Next to the MoE block of mol_block.h a layer has its attention over a cache
 * of keys and values held in pages:
 *
 *   mol_rope             rotary positions of query or key heads;
 *   mol_cache_append     the new tokens' keys (turned on the way) and values
 *                        into their slots of the cache, and the queries turned
 *                        by the same launch;
 *   mol_paged_attention  attention of the new tokens, one or thousands for each
 *                        sequence, over the cached ones.
 *
 * The conventions of mol.h hold: device pointers owned by the caller, calls
 * only enqueue on `stream`, arguments are checked on the host first, nothing
 * is launched on an error status. Values are bf16; head rows are 16-byte
 * aligned (pointers, and strides in elements a multiple of 8 and at least a
 * head's width, in any order of tokens and heads). Heads that are written do
 * not overlap.
 */
#ifndef MOL_ATTN_H_
#define MOL_ATTN_H_

#include "mol.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOL_ROPE_MAX_HEAD_DIM 512  /* widest head of mol_rope and mol_cache_append */
#define MOL_ATTN_MAX_GROUP 64      /* most query heads to a key head */

/*
 * Rotary positions: pair i < rotary_dim / 2 of a head, (x[i], x[i + rotary_dim/2])
 * or, interleaved, (x[2i], x[2i + 1]), is turned by the angle position *
 * inv_freq[i] and multiplied by magnitude:
 *   (a, b) -> magnitude * (a cos - b sin, b cos + a sin)
 * in fp32, the angle in 64 bits (far positions keep their fraction of a turn),
 * rounded to bf16 once. Elements from rotary_dim on stay as they are.
 * Contract: rotary_dim a multiple of 16, at most the head's width; magnitude
 * finite.
 */
typedef struct mol_rope_table {
  const float* inv_freq;  /* fp32 [rotary_dim / 2] */
  int32_t rotary_dim;
  int32_t interleaved;    /* 0: halves, 1: neighbours */
  float magnitude;
} mol_rope_table;

/*
 * A paged cache: head h of token o of page p is head_dim bf16 values at
 * k + p * page_stride + o * token_stride + h * head_stride (elements), and the
 * same from v. A token's slot is p * page_size + o.
 * Contract: 1 <= page_size, num_pages * page_size < 2^31, strides multiples of 8.
 */
typedef struct mol_paged_cache {
  void* k;
  void* v;
  int64_t page_stride, token_stride, head_stride;
  int64_t num_pages;
  int32_t page_size, num_heads, head_dim;
} mol_paged_cache;

/*
 * out[t, h] = x[t, h] with positions[t] (int32, any sign) turned into it.
 * out may be x itself (same strides); any other overlap is outside the contract.
 * Contract: head_dim a multiple of 8 up to MOL_ROPE_MAX_HEAD_DIM, strides
 * multiples of 8, num_tokens < 2^31, num_heads <= 65536.
 */
int32_t mol_rope(const void* x, int64_t x_token_stride, int64_t x_head_stride,
                 const int32_t* positions, const mol_rope_table* rope, int64_t num_tokens,
                 int32_t num_heads, int32_t head_dim, void* out, int64_t out_token_stride,
                 int64_t out_head_stride, void* stream);

/*
 * Token t's key heads (turned by positions[t] when rope is not NULL) and value
 * heads into slot slots[t] of the cache; a token whose slot is outside the
 * cache (-1: a padding row) writes nothing there. With q, its num_q_heads heads
 * of head_dim are turned into q_out by the same launch, padding rows too; q_out
 * may be q itself (same strides). Tokens name different slots: of two that name
 * one, either's values, or some of each, remain. k, v and q lie outside the cache.
 *   rope        NULL: keys are copied (positions is not read then; q NULL)
 * Contract: as mol_rope for the heads, cache->head_dim their width.
 */
int32_t mol_cache_append(const void* k, int64_t k_token_stride, int64_t k_head_stride,
                         const void* v, int64_t v_token_stride, int64_t v_head_stride,
                         const int32_t* slots, const int32_t* positions,
                         const mol_rope_table* rope, int64_t num_tokens,
                         const mol_paged_cache* cache, const void* q, int64_t q_token_stride,
                         int64_t q_head_stride, int32_t num_q_heads, void* q_out,
                         int64_t q_out_token_stride, int64_t q_out_head_stride, void* stream);

/*
 * Attention of new tokens over the paged cache. Sequence b has the rows
 * q_starts[b] .. q_starts[b + 1] - 1 of q (q_starts NULL: row b, num_tokens =
 * num_seqs), n of them, and kv_lens[b] cached tokens, of which the new ones are
 * the last n: its row i sits at position kv_lens[b] - n + i and sees the cached
 * tokens at positions up to its own, the last `window` of them (its own among
 * them) where window > 0. Token j lies at offset j % page_size of page
 * page_table[b * table_stride + j / page_size]; a token whose page is outside
 * the cache (-1: given back) is seen by no row. Query head h reads key head
 * h / (num_q_heads / cache->num_heads):
 *   out[row, h] = sum_j w_j v[j],  w = softmax over the seen j of scale * q[row, h] . k[j]
 * A row that sees no token, or whose every score is -infinity, is 0; one with a
 * score of +infinity or NaN is NaN. Rows of q that belong to no sequence leave out
 * as it was. Products of bf16 with fp32 sums; the weights are rounded to bf16
 * before they meet the values, their sum is not; out is rounded once. What a
 * row does not see does not reach it, whatever it holds (NaN, infinities).
 * A kv_lens[b] past the table's width is taken as that width; q_starts outside
 * [0, num_tokens] as the nearer end. They do not decrease: a call in which one
 * does leaves all of out as it was.
 *   workspace   mol_paged_attention_workspace_bytes of scratch, of these sizes or
 *               larger ones, 16-byte aligned; calls that may run at the same
 *               time need one each
 * out may be q itself (same strides).
 * Contract: head_dim 64, 128 or 256; num_q_heads a multiple of cache->num_heads,
 * at most MOL_ATTN_MAX_GROUP times it; scale > 0, it and its product with
 * log2(e) finite; window >= 0; num_q_heads <= 65536; num_seqs < 2^24;
 * num_tokens * num_q_heads < 2^31;
 * num_tokens + max_pages * page_size <= 2^31 - 1024; with g query heads to a key
 * head, num_tokens * g <= 2^31 - 1024 and
 * (num_tokens * g / 16 + num_seqs) * (max_pages * page_size / 64 + 4) < 2^31
 * (16 K tokens of group 8 over tables of 8 M).
 */
int32_t mol_paged_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                            const mol_paged_cache* cache, const int32_t* page_table,
                            int64_t table_stride, int32_t max_pages, const int32_t* kv_lens,
                            const int32_t* q_starts, int64_t num_seqs, int64_t num_tokens,
                            int32_t num_q_heads, float scale, int32_t window, void* out,
                            int64_t out_token_stride, int64_t out_head_stride, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * Bytes of workspace with which every mol_paged_attention call of at most
 * num_seqs sequences and num_tokens tokens of these heads is served (host
 * arithmetic): a buffer of the largest sizes serves all calls. 0 for sizes that
 * the call refuses.
 */
size_t mol_paged_attention_workspace_bytes(int64_t num_seqs, int64_t num_tokens,
                                           int32_t num_q_heads, int32_t num_kv_heads,
                                           int32_t head_dim);

#ifdef __cplusplus
}
#endif

#endif /* MOL_ATTN_H_ */
