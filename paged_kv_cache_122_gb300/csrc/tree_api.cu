// Host entry points of tree and cross attention: argument checks and the launch.
#include "../../include/pagedkv_tree.h"
#include "rows_attention.cuh"
#include "stream_turn.cuh"

#include <cmath>

namespace {

bool group_supported(int G) { return G == 1 || G == 2 || G == 4 || G == 8 || G == 16; }

int attend(void *out, int out_dtype, const void *q, int total_q, const int32_t *cu_q_lens, int max_q_len,
           bool tree, const uint64_t *tree_mask, int mask_words, const void *k_cache, const void *v_cache,
           const int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens, int max_seq_len, int num_seqs,
           int num_heads, int num_kv_heads, int head_dim, int num_blocks, int block_size, float scale, void *workspace,
           size_t workspace_bytes, pk_stream_t stream, int stall_tile, uint64_t wait_limit_ns,
           const int32_t *lens_ahead, const int32_t *cu_ahead) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_blocks < 0 || max_blocks_per_seq < 0 ||
        max_seq_len < 0 || block_size <= 0 || total_q < 0 || max_q_len < 0)
        return PK_ERR_SHAPE;
    if (num_heads % num_kv_heads) return PK_ERR_SHAPE;
    if (static_cast<int64_t>(max_seq_len) > static_cast<int64_t>(max_blocks_per_seq) * block_size)
        return PK_ERR_SHAPE;
    if (out_dtype != PK_BF16 && out_dtype != PK_FP32) return PK_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PK_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PK_ERR_UNSUPPORTED;
    if (!group_supported(num_heads / num_kv_heads)) return PK_ERR_UNSUPPORTED;
    if (!std::isfinite(scale)) return PK_ERR_SHAPE;
    if (num_seqs > 65535) return PK_ERR_SHAPE;
    // (The kernel counts a mask row in 32-bit words.)
    if (tree && (mask_words > (1 << 30) - 1 || static_cast<int64_t>(mask_words) * 64 < max_q_len)) return PK_ERR_SHAPE;
    if (num_seqs == 0 || total_q == 0 || max_q_len == 0) return PK_OK;
    if (!out || !q || !cu_q_lens || !seq_lens || (tree && !tree_mask) ||
        (max_seq_len > 0 && (!k_cache || !v_cache || !block_tables)))
        return PK_ERR_NULL;
    if (!pk::aligned16(out) || !pk::aligned16(q) || !pk::aligned16(k_cache) || !pk::aligned16(v_cache) ||
        (reinterpret_cast<uintptr_t>(tree_mask) & 7u))
        return PK_ERR_ALIGNMENT;
    pk::RowsParams p{};
    if (max_seq_len > 128) {
        // A sequence longer than one tile may span several CTAs: its parts need slots.
        if (!workspace || workspace_bytes < pk::rows_workspace_bytes(num_heads, num_kv_heads, head_dim, max_q_len))
            return PK_ERR_WORKSPACE;
        if (!pk::aligned16(workspace)) return PK_ERR_ALIGNMENT;
        p.slots = workspace;
    }
    p.out = out;
    p.out_fp32 = out_dtype == PK_FP32;
    p.q = static_cast<const uint16_t *>(q);
    p.k_cache = max_seq_len > 0 ? static_cast<const uint16_t *>(k_cache) : nullptr;
    p.v_cache = max_seq_len > 0 ? static_cast<const uint16_t *>(v_cache) : nullptr;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.cu_q_lens = cu_q_lens;
    p.tree_mask = tree ? reinterpret_cast<const uint32_t *>(tree_mask) : nullptr;
    p.mask_words = tree ? 2 * mask_words : 0;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_seq_len = max_seq_len;
    p.max_q_len = max_q_len;
    p.total_q = total_q;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    // (Not 0: the kernel multiplies it with infinities, and a factor this small makes
    // every finite score 0 all the same.)
    p.scale_log2 = scale * pk::kLog2e;
    if (p.scale_log2 == 0.f) p.scale_log2 = 1.17549435e-38f;
    p.wait_limit_ns = wait_limit_ns;
    p.stall_tile = stall_tile;
    p.lens_ahead = lens_ahead;
    p.cu_ahead = cu_ahead;
    p.err = pk::error_word_ptr();
    if (!p.err) return PK_ERR_NO_DEVICE;
    const pk::StreamTurn turn(pk::current_device(), stream);
    return pk::launch_rows_attention(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

}  // namespace

extern "C" size_t pk_tree_workspace_bytes(int num_heads, int num_kv_heads, int head_dim, int max_q_len,
                                          int max_seq_len) {
    if (num_heads <= 0 || num_kv_heads <= 0 || max_q_len <= 0 || max_seq_len <= 128) return 0;
    if (num_heads % num_kv_heads || !group_supported(num_heads / num_kv_heads)) return 0;
    if (head_dim != 64 && head_dim != 128) return 0;
    return pk::rows_workspace_bytes(num_heads, num_kv_heads, head_dim, max_q_len);
}

extern "C" int pk_paged_attention_tree(void *out, int out_dtype, const void *q, int total_q, const int32_t *cu_q_lens,
                                       int max_q_len, const uint64_t *tree_mask, int mask_words, const void *k_cache,
                                       const void *v_cache, const int32_t *block_tables, int max_blocks_per_seq,
                                       const int32_t *seq_lens, int max_seq_len, int num_seqs, int num_heads,
                                       int num_kv_heads, int head_dim, int num_blocks, int block_size, float scale,
                                       void *workspace, size_t workspace_bytes, pk_stream_t stream) {
    return attend(out, out_dtype, q, total_q, cu_q_lens, max_q_len, true, tree_mask, mask_words, k_cache, v_cache,
                  block_tables, max_blocks_per_seq, seq_lens, max_seq_len, num_seqs, num_heads, num_kv_heads, head_dim,
                  num_blocks, block_size, scale, workspace, workspace_bytes, stream, 0, 0, nullptr, nullptr);
}

extern "C" int pk_paged_attention_cross(void *out, int out_dtype, const void *q, int total_q, const int32_t *cu_q_lens,
                                        int max_q_len, const void *k_cache, const void *v_cache,
                                        const int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens,
                                        int max_seq_len, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                        int num_blocks, int block_size, float scale, void *workspace,
                                        size_t workspace_bytes, pk_stream_t stream) {
    return attend(out, out_dtype, q, total_q, cu_q_lens, max_q_len, false, nullptr, 0, k_cache, v_cache, block_tables,
                  max_blocks_per_seq, seq_lens, max_seq_len, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks,
                  block_size, scale, workspace, workspace_bytes, stream, 0, 0, nullptr, nullptr);
}

extern "C" int pk_selftest_cross_wait_timeout(void *out, int out_dtype, const void *q, int total_q,
                                              const int32_t *cu_q_lens, int max_q_len, const void *k_cache,
                                              const void *v_cache, const int32_t *block_tables, int max_blocks_per_seq,
                                              const int32_t *seq_lens, int max_seq_len, int num_seqs, int num_heads,
                                              int num_kv_heads, int head_dim, int num_blocks, int block_size,
                                              float scale, void *workspace, size_t workspace_bytes, int stall_tile,
                                              unsigned int wait_limit_us, pk_stream_t stream) {
    if (stall_tile < 1 || wait_limit_us < 100 || wait_limit_us > 1000000) return PK_ERR_SHAPE;
    return attend(out, out_dtype, q, total_q, cu_q_lens, max_q_len, false, nullptr, 0, k_cache, v_cache, block_tables,
                  max_blocks_per_seq, seq_lens, max_seq_len, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks,
                  block_size, scale, workspace, workspace_bytes, stream, stall_tile,
                  static_cast<uint64_t>(wait_limit_us) * 1000u, nullptr, nullptr);
}

extern "C" int pk_selftest_cross_stale_lengths(void *out, int out_dtype, const void *q, int total_q,
                                               const int32_t *cu_q_lens, int max_q_len, const void *k_cache,
                                               const void *v_cache, const int32_t *block_tables, int max_blocks_per_seq,
                                               const int32_t *seq_lens, int max_seq_len, int num_seqs, int num_heads,
                                               int num_kv_heads, int head_dim, int num_blocks, int block_size,
                                               float scale, const int32_t *stale_seq_lens,
                                               const int32_t *stale_cu_q_lens, void *workspace, size_t workspace_bytes,
                                               pk_stream_t stream) {
    if (!stale_seq_lens || !stale_cu_q_lens) return PK_ERR_NULL;
    return attend(out, out_dtype, q, total_q, cu_q_lens, max_q_len, false, nullptr, 0, k_cache, v_cache, block_tables,
                  max_blocks_per_seq, seq_lens, max_seq_len, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks,
                  block_size, scale, workspace, workspace_bytes, stream, 0, 0, stale_seq_lens, stale_cu_q_lens);
}
