/*
 * pagedkv_tree.h -- C ABI of tree verification and of cross attention over the
 * bf16 paged KV cache (GB300, sm_103a).
 *
 * Speculative decoding checks drafted tokens in one pass over the cache
 * ("PagedAttention from First Principles", §14).  A chain of drafts is
 * pk_paged_attention_multi_query; a TREE of drafts needs a mask among them, and
 * after the check the accepted path lies scattered in the cache.  One step:
 *
 *   pk_rope_and_cache          append the tree's nodes (positions: context + depth)
 *   pk_paged_attention_tree    every node over the context and its ancestors
 *   pk_accept_tree             the path that the target model agrees with
 *   pk_keep_tokens(_layers)    that path's K and V rows, moved together
 *   pk_bm_truncate             (host) the pages behind them, freed
 *
 * pk_paged_attention_cross attends to keys of another length, all visible: the
 * cross attention of a decoder to an encoder's states in the paged cache.
 *
 * Pointers, streams, errors and supported sizes are those of pagedkv.h.  All of them
 * take the bf16 cache.  The 8-bit one (pagedkv_fp8.h) has chains of drafts only: its
 * rows share a block's scale, so none can be moved alone, and its keys can be attended
 * to here only after pk_gather_kv_fp8 has copied them out as bf16.
 */
#ifndef PAGEDKV_TREE_H
#define PAGEDKV_TREE_H

#include "pagedkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Bytes of workspace that the two attention calls need: partial results of
 * sequences split over CTAs (two slots for each of at most 160 CTAs, 128 or 256
 * query rows each).  0 when nothing can be split (max_seq_len <= 128) or the
 * sizes are invalid.
 */
size_t pk_tree_workspace_bytes(int num_heads, int num_kv_heads, int head_dim, int max_q_len, int max_seq_len);

/*
 * Attention of a tree of drafted tokens per sequence over the paged cache.
 * Sequence s owns query rows cu_q_lens[s] .. cu_q_lens[s+1]-1: its n newest
 * tokens, whose K/V are already in the cache.  With L = seq_lens[s], row r of
 * them attends to positions 0 .. L-n-1 (the context, all of it) and to position
 * L-n+i wherever bit i % 64 of word i / 64 of its mask row is set.  Nothing is
 * added to the mask: a node that sees itself has its own bit set.  Bits i >= n
 * are ignored.  A row that sees nothing gets zeros.
 *
 *   out, q, cu_q_lens, max_q_len, caches, tables, lengths, scale
 *                 as for pk_paged_attention_multi_query
 *   tree_mask     [total_q, mask_words] 64-bit words, row r that of query row r,
 *                 8-byte aligned
 *   mask_words    at least ceil(max_q_len / 64)
 *   workspace     pk_tree_workspace_bytes(...); its contents do not matter.
 *                 Calls that share one must be ordered on the GPU (same stream,
 *                 from any number of host threads)
 *
 * Any number of nodes and any supported group run on one kernel: 128 (node, head)
 * rows to a tile.  A sequence with a negative length or one beyond max_seq_len or
 * its table, with more rows than max_q_len or than tokens, or with rows outside
 * the total_q given, sets PK_DEVERR_SEQ_LEN and its rows are left as they were,
 * as are rows that no sequence owns.  Keys behind a block id outside the pool are
 * not seen (PK_DEVERR_BLOCK_ID).  Weights are rounded to bf16 for the product
 * with V, and the denominator sums the rounded weights, each of which is at most 1:
 * results are finite while the number of keys times the largest value is below
 * 2^127 and the scaled scores below 2^27.  A value that is not
 * finite in a node of the tree shows in all rows of its tree; a key that is not
 * finite shows only in the rows that see it.  The same call gives the same bits; those
 * of a sequence may change with the rest of the batch, which decides where it is cut and
 * against which reference its weights are taken.
 */
int pk_paged_attention_tree(void *out, int out_dtype, const void *q, int total_q, const int32_t *cu_q_lens,
                            int max_q_len, const uint64_t *tree_mask, int mask_words, const void *k_cache,
                            const void *v_cache, const int32_t *block_tables, int max_blocks_per_seq,
                            const int32_t *seq_lens, int max_seq_len, int num_seqs, int num_heads,
                            int num_kv_heads, int head_dim, int num_blocks, int block_size, float scale,
                            void *workspace, size_t workspace_bytes, pk_stream_t stream);

/*
 * Attention of any number of query rows per sequence over ALL keys of the
 * sequence, whose number has nothing to do with that of the rows (an encoder's
 * states; no causal limit): out[r,h,:] = sum_j softmax_j(scale * q[r,h,:] . k_j)
 * v_j, j = 0 .. seq_lens[s]-1.  A sequence without keys gets zeros.  Everything
 * else is as for pk_paged_attention_tree.  One query row per sequence is
 * pk_paged_attention_decode.
 */
int pk_paged_attention_cross(void *out, int out_dtype, const void *q, int total_q, const int32_t *cu_q_lens,
                             int max_q_len, const void *k_cache, const void *v_cache,
                             const int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens,
                             int max_seq_len, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                             int num_blocks, int block_size, float scale, void *workspace,
                             size_t workspace_bytes, pk_stream_t stream);

/*
 * Self-test of the attention kernel's bounded waits, as
 * pk_selftest_decode_wait_timeout is for decode: CTA 0's key copies stop before
 * tile `stall_tile` (>= 1) of its range, and waits give up after wait_limit_us
 * (in [100, 1000000]).  The other arguments are those of pk_paged_attention_cross.
 */
int pk_selftest_cross_wait_timeout(void *out, int out_dtype, const void *q, int total_q, const int32_t *cu_q_lens,
                                   int max_q_len, const void *k_cache, const void *v_cache,
                                   const int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens,
                                   int max_seq_len, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                   int num_blocks, int block_size, float scale, void *workspace,
                                   size_t workspace_bytes, int stall_tile, unsigned int wait_limit_us,
                                   pk_stream_t stream);

/*
 * Self-test of the second look at the lengths, as pk_selftest_decode_stale_lengths is
 * for decode.  The attention kernel plans its work before the programmatic wait on the
 * kernel before it and plans again where the lengths read after the wait differ; here
 * the first plan is made from stale_seq_lens [num_seqs] and stale_cu_q_lens
 * [num_seqs + 1] (any values; out-of-range ones are not reported).  The result is that
 * of pk_paged_attention_cross, whose arguments the others are.  (With more than 384
 * sequences nothing is planned ahead.)  PK_ERR_NULL if either array is NULL.
 */
int pk_selftest_cross_stale_lengths(void *out, int out_dtype, const void *q, int total_q, const int32_t *cu_q_lens,
                                    int max_q_len, const void *k_cache, const void *v_cache,
                                    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens,
                                    int max_seq_len, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                    int num_blocks, int block_size, float scale, const int32_t *stale_seq_lens,
                                    const int32_t *stale_cu_q_lens, void *workspace, size_t workspace_bytes,
                                    pk_stream_t stream);

/*
 * The accepted path of each tree.  Node 0 is the root (the token sampled last, so
 * it is right); node c > 0 hangs below parents[c].  The path starts at node 0 and
 * goes on, from node p, to the lowest c > p of the tree with parents[c] == p and
 * draft_tokens[c] == target_tokens[p], until there is none.  Parents outside
 * [0, c) are never reached (padding).
 *
 *   accepted       [num_seqs, max_q_len] int32: the path's nodes, -1 behind them
 *   num_accepted   [num_seqs] int32 (0 for a sequence without nodes)
 *   next_tokens    [num_seqs] int64: target_tokens of the last accepted node, -1
 *                  for a sequence without nodes
 *   new_seq_lens   [num_seqs] int32: seq_lens[s] - n + num_accepted[s]; may be
 *                  seq_lens itself where no pk_keep_tokens call follows (that call
 *                  takes the lengths before)
 *   draft_tokens, target_tokens  [total_q] int64: each node's token, and the
 *                  target model's choice (sampled or greedy) after it
 *   parents        [total_q] int32, indices within the tree
 *   cu_q_lens, max_q_len, seq_lens  as in the attention call
 * max_q_len <= 8192.  A sequence whose rows run backwards, outside total_q, beyond
 * max_q_len or beyond its length sets PK_DEVERR_SEQ_LEN; it counts as one without
 * nodes, and its new length is its old one.
 */
int pk_accept_tree(int32_t *accepted, int32_t *num_accepted, int64_t *next_tokens, int32_t *new_seq_lens,
                   const int64_t *draft_tokens, const int32_t *parents, const int64_t *target_tokens, int total_q,
                   const int32_t *cu_q_lens, int max_q_len, const int32_t *seq_lens, int num_seqs,
                   pk_stream_t stream);

/*
 * Moves the accepted tokens of each sequence together: with base = seq_lens[s] -
 * n, the K and V rows of position base + accepted[s, i] go to position base + i,
 * i < num_accepted[s].  Lists are strictly increasing, as pk_accept_tree writes
 * them, so that no row is written before it is read.  Rows from base +
 * num_accepted[s] on keep their old bits.
 *
 *   seq_lens, cu_q_lens  as in the attention call: lengths with the whole tree
 *   accepted       [num_seqs, accepted_stride] int32
 *   num_accepted   [num_seqs] int32
 * A list that is not strictly increasing, names a node outside the tree or is
 * longer than the tree or accepted_stride sets PK_DEVERR_DRAFT and moves nothing;
 * a bad length sets PK_DEVERR_SEQ_LEN likewise.  A row whose source or
 * destination block is outside the pool is not moved (PK_DEVERR_BLOCK_ID).  The
 * blocks of a tree belong to one sequence, as copy-on-write leaves them.
 * Bit-exact.
 */
int pk_keep_tokens(void *k_cache, void *v_cache, const int32_t *block_tables, int max_blocks_per_seq,
                   const int32_t *seq_lens, const int32_t *cu_q_lens, const int32_t *accepted, int accepted_stride,
                   const int32_t *num_accepted, int num_seqs, int num_kv_heads, int head_dim, int num_blocks,
                   int block_size, pk_stream_t stream);

/* The same on every layer in one launch; pointer arrays and layers as for
 * pk_copy_blocks_layers (num_layers in [1, 32767]).  A layer whose K or V pointer is
 * NULL or not 16-byte aligned sets PK_DEVERR_POINTER and neither its K nor its V is
 * moved, so that both stay rows of the same tokens. */
int pk_keep_tokens_layers(void *const *k_cache_layers, void *const *v_cache_layers, const int32_t *block_tables,
                          int max_blocks_per_seq, const int32_t *seq_lens, const int32_t *cu_q_lens,
                          const int32_t *accepted, int accepted_stride, const int32_t *num_accepted, int num_seqs,
                          int num_layers, int num_kv_heads, int head_dim, int num_blocks, int block_size,
                          pk_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_TREE_H */
