/*
 * pagedkv_fp8.h -- C ABI of the 8-bit paged KV cache (GB300, sm_103a).
 *
 * Decode attention is bound by the bytes of the cache, so a cache of half the
 * bytes is what makes it faster, and holds twice the tokens:
 *
 *   pk_rope_and_cache_fp8           rotate q and k, append k and v
 *   pk_paged_attention_decode_fp8   attention, one query token a sequence
 *   pk_paged_attention_multi_query_fp8  a few causal query tokens a sequence
 *   pk_gather_kv_fp8                rows back as bf16 (for prompt chunks)
 *   pk_copy_blocks_fp8, pk_swap_blocks_fp8  blocks with their scales
 *
 * The pages have no counterpart of these calls.  Pointers, streams, errors and
 * supported sizes are those of pagedkv.h.
 *
 * Cache.  k_cache and v_cache are [num_blocks, num_kv_heads, block_size,
 *   head_dim] e4m3 (OCP 8-bit floating point: 1 sign, 4 exponent, 3 significand
 *   bits; largest 448; one NaN, no infinity).  k_scales and v_scales are
 *   [num_blocks, num_kv_heads] fp32: the value stored as e stands for e * scale.
 *   The tokens of a block and KV head share a scale, so they lie together (the
 *   bf16 cache keeps the heads of a token together instead).
 * Scales.  Positive, in [2^-64, 2^64]; the append writes powers of two, other
 *   sources may use any.  A scale outside sets PK_DEVERR_SCALE.  Attention and
 *   gather then treat its block and head as one whose id is outside the pool
 *   (skipped); the append gives its older rows up (below).
 */
#ifndef PAGEDKV_FP8_H
#define PAGEDKV_FP8_H

#include "pagedkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The rotary position embedding of each sequence's newest tokens and their
 * append to the 8-bit cache, in one pass.  Sequence s owns rows cu_q_lens[s] ..
 * cu_q_lens[s+1]-1 of q, k and v: its n newest tokens, at positions
 * seq_lens[s] - n .. seq_lens[s] - 1 of its block table, as in
 * pk_paged_attention_multi_query_fp8, which takes the same arrays.  (Slots
 * would not do: the writer of a block has to know which of its tokens are
 * new.)  A block that takes new tokens belongs to one sequence, as
 * copy-on-write leaves it; two that write one block leave it unspecified.
 *
 * Scale of a block and KV head that takes new tokens: the smallest 2^e, -64 <=
 * e <= 64, with m2 <= (448 * 2^e)^2, and at least the scale of the block's
 * older tokens if it has any (rows below the first new one); a block whose
 * first row is new starts afresh, whatever its scale held.  m2 is the largest,
 * over the block's new tokens, of (x1^2 + x2^2) * factor^2 for the pairs of K
 * that are rotated -- a bound on both results that does not depend on the
 * position -- and of x^2 for every other element, in fp32 (what overflows counts
 * as the largest fp32 number: the scale is then 2^56).  If the scale
 * grows, the older rows are rounded to it again (exact where they stay above
 * 2^-6 times the new scale).  A new value y is stored as y * (1 / scale)
 * rounded to nearest even, at most +-448; one that is not finite is stored as
 * NaN and left out of m2.  Rows behind the last new token are left as they
 * were.
 *   Where the scale of older tokens is out of range, nothing says what their
 * rows stood for: that head's older rows (of K or of V, whichever scale it is)
 * become NaN, the block takes the scale that the new tokens need, and
 * PK_DEVERR_SCALE is set.  What attends to those rows is NaN from then on.
 *
 *   q, k, v, q_out and their strides, inv_freq, rot_dim, interleaved, factor:
 *                 as for pk_rope_and_cache
 *   k_scales, v_scales, k_cache, v_cache: updated in place
 *   block_tables  [num_seqs, max_blocks_per_seq] int32
 *   seq_lens      [num_seqs] int32, lengths after the append
 *   cu_q_lens     [num_seqs + 1] int32 device array, or NULL: one new token a
 *                 sequence (num_tokens == num_seqs)
 *   max_q_len     host-side bound of the new tokens of a sequence (unused
 *                 without cu_q_lens)
 *   positions     [num_tokens] int64 device array of the angles' positions, or
 *                 NULL: the positions in the block table
 * A sequence whose length is negative or beyond its table, that has more new
 * tokens than tokens or than max_q_len, or whose rows are not within the
 * num_tokens given sets PK_DEVERR_SEQ_LEN, and nothing of it is written.  A
 * block id outside the pool sets PK_DEVERR_BLOCK_ID: that block's K and V are
 * not written.  num_seqs <= 65535.  Rows of q_out that no sequence owns are left
 * as they were: a batch of fixed size is padded with sequences of length 0 and no
 * rows (cu_q_lens stays at its last value).  Where cu_q_lens runs backwards, tokens
 * of later sequences may be left out too.
 */
int pk_rope_and_cache_fp8(void *q_out, const void *q, const void *k, const void *v, int64_t q_out_stride,
                          int64_t q_stride, int64_t k_stride, int64_t v_stride, void *k_cache,
                          void *v_cache, float *k_scales, float *v_scales, const int32_t *block_tables,
                          int max_blocks_per_seq, const int32_t *seq_lens, const int32_t *cu_q_lens,
                          int max_q_len, int num_seqs, const int64_t *positions, const float *inv_freq,
                          int rot_dim, int interleaved, float factor, int num_tokens, int num_heads,
                          int num_kv_heads, int head_dim, int num_blocks, int block_size,
                          pk_stream_t stream);

/*
 * Bytes of workspace the two attention calls below need for these sizes; 0
 * when no sequence can be split or the sizes are invalid.  As for
 * pk_decode_workspace_bytes, whose layout of partial results they share.
 */
size_t pk_decode_fp8_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                     int max_seq_len);

/*
 * Single-query decode attention over the 8-bit paged cache:
 *
 *   out[s,h,:] = sum_j softmax_j(scale * q[s,h,:] . (ks_j k_j)) vs_j v_j,  j = 0 .. L-1,
 *
 * with k_j, v_j the e4m3 rows of token j and KV head h / G and ks_j, vs_j the
 * scales of its block and that head.  Everything else -- arguments, table
 * walk, lengths, workspace, errors, determinism -- is as for
 * pk_paged_attention_decode.  Queries are bf16, used exactly down to 2^-13 of
 * their row's largest and to 2^-22 of it below.  Numerators take a weight (times
 * its value scale) to 2^-11 of itself and to 2^-24 of the row's largest one;
 * denominators and the partial results of split sequences are fp32.
 * A NaN in a key or a value of an attended token shows in its output.
 */
int pk_paged_attention_decode_fp8(void *out, int out_dtype, const void *q, const void *k_cache,
                                  const void *v_cache, const float *k_scales, const float *v_scales,
                                  const int32_t *block_tables, int max_blocks_per_seq,
                                  const int32_t *seq_lens, int max_seq_len, int num_seqs, int num_heads,
                                  int num_kv_heads, int head_dim, int num_blocks, int block_size,
                                  float scale, void *workspace, size_t workspace_bytes,
                                  pk_stream_t stream);

/*
 * Self-tests of pk_paged_attention_decode_fp8, as pk_selftest_decode_wait_timeout
 * and pk_selftest_decode_stale_lengths are for the bf16 call: the kernel's bounded
 * waits run out where CTA 0's producers stop before tile `stall_tile` of its range
 * (>= 1; wait_limit_us in [100, 1000000]), and its first plan comes from the device
 * array `stale_seq_lens` (unused where the kernel keeps no lengths in shared memory:
 * above 256 sequences, 2,048 with 16 heads per KV head, or 8 at head dim 64 with an
 * even number of KV heads).  The other arguments are those of
 * pk_paged_attention_decode_fp8.
 */
int pk_selftest_decode_fp8_wait_timeout(void *out, int out_dtype, const void *q, const void *k_cache,
                                        const void *v_cache, const float *k_scales, const float *v_scales,
                                        const int32_t *block_tables, int max_blocks_per_seq,
                                        const int32_t *seq_lens, int max_seq_len, int num_seqs, int num_heads,
                                        int num_kv_heads, int head_dim, int num_blocks, int block_size,
                                        float scale, void *workspace, size_t workspace_bytes, int stall_tile,
                                        unsigned int wait_limit_us, pk_stream_t stream);
int pk_selftest_decode_fp8_stale_lengths(void *out, int out_dtype, const void *q, const void *k_cache,
                                         const void *v_cache, const float *k_scales, const float *v_scales,
                                         const int32_t *block_tables, int max_blocks_per_seq,
                                         const int32_t *seq_lens, int max_seq_len, int num_seqs, int num_heads,
                                         int num_kv_heads, int head_dim, int num_blocks, int block_size,
                                         float scale, const int32_t *stale_seq_lens, void *workspace,
                                         size_t workspace_bytes, pk_stream_t stream);

/*
 * Attention of a FEW new tokens per sequence over the 8-bit paged cache,
 * causal among them (verification of drafted tokens), as
 * pk_paged_attention_multi_query defines it: sequence s owns query rows
 * cu_q_lens[s] .. cu_q_lens[s+1]-1, its newest tokens.  G * q <= 16 with q =
 * max_q_len rounded up to a power of two (the query columns of the decode
 * kernel); wider blocks are PK_ERR_UNSUPPORTED: see pk_gather_kv_fp8.
 *
 * A sequence with more queries than max_q_len (rounded up) or than tokens, or
 * with rows outside the total_q given, sets PK_DEVERR_SEQ_LEN; its rows are
 * left unwritten (unspecified where it has more queries than tokens).  A NaN in
 * the value of one of the block's own tokens shows in all of its queries.
 */
int pk_paged_attention_multi_query_fp8(void *out, int out_dtype, const void *q, int total_q,
                                       const int32_t *cu_q_lens, int max_q_len, const void *k_cache,
                                       const void *v_cache, const float *k_scales, const float *v_scales,
                                       const int32_t *block_tables, int max_blocks_per_seq,
                                       const int32_t *seq_lens, int max_seq_len, int num_seqs,
                                       int num_heads, int num_kv_heads, int head_dim, int num_blocks,
                                       int block_size, float scale, void *workspace,
                                       size_t workspace_bytes, pk_stream_t stream);

/*
 * Rows of the 8-bit cache as bf16 through the block tables:
 * out_k[cu_seq_lens[s] + j] = bf16(k scale * k row of token j), j < seq_lens[s]
 * (same for V); exact when the scales are powers of two.  A prompt chunk that
 * attends to an 8-bit prefix gathers it first: with cu_seq_lens at multiples of
 * the block size the rows are the pages of a bf16 cache whose tables count up,
 * which pk_paged_attention_multi_query reads (the chunk's work grows with
 * queries times keys, the gather's with the keys alone).
 *
 *   out_k, out_v  [out_rows, num_kv_heads, head_dim] bf16
 *   cu_seq_lens   [num_seqs] int64 device array: first output row of each
 *                 sequence; one whose rows are not within out_rows sets
 *                 PK_DEVERR_SEQ_LEN and is left out
 *   max_seq_len   host-side bound of seq_lens; a longer one sets
 *                 PK_DEVERR_SEQ_LEN and its first max_seq_len rows are written
 * Rows of a block whose id or scale is bad are left unwritten.  max_seq_len = 0 or
 * out_rows = 0 is a no-op.
 */
int pk_gather_kv_fp8(void *out_k, void *out_v, const void *k_cache, const void *v_cache,
                     const float *k_scales, const float *v_scales, const int32_t *block_tables,
                     int max_blocks_per_seq, const int32_t *seq_lens, const int64_t *cu_seq_lens,
                     int64_t out_rows, int max_seq_len, int num_seqs, int num_kv_heads, int head_dim,
                     int num_blocks, int block_size, pk_stream_t stream);

/*
 * pk_copy_blocks and pk_swap_blocks for the 8-bit cache: whole blocks of K and
 * V with their scales, one launch for all pairs.  Pairs, errors and what is
 * left unspecified are as there; bit-exact.
 */
int pk_copy_blocks_fp8(void *k_cache, void *v_cache, float *k_scales, float *v_scales,
                       const int64_t *src_dst_pairs, int num_pairs, int num_kv_heads, int head_dim,
                       int num_blocks, int block_size, pk_stream_t stream);
int pk_swap_blocks_fp8(void *dst_k, void *dst_v, float *dst_k_scales, float *dst_v_scales,
                       const void *src_k, const void *src_v, const float *src_k_scales,
                       const float *src_v_scales, const int64_t *pairs, int num_pairs, int num_kv_heads,
                       int head_dim, int block_size, int src_num_blocks, int dst_num_blocks,
                       pk_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_FP8_H */
