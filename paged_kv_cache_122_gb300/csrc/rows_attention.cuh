// Parameters and launcher of attention with many query rows per sequence over
// the split paged keys (a tree of drafted tokens; cross attention).
#pragma once

#include "common.cuh"

namespace pk {

struct RowsParams {
    void *out;
    int out_fp32;
    const uint16_t *q;            // [total_q, H, D]
    const uint16_t *k_cache;      // [P, B, Hkv, D]
    const uint16_t *v_cache;
    const int32_t *block_tables;  // [N, MB]
    const int32_t *seq_lens;      // [N]
    const int32_t *cu_q_lens;     // [N + 1]
    const uint32_t *tree_mask;    // [total_q, mask_words] bits, or NULL: every key is seen
    int mask_words;               // 32-bit words of a row
    int max_blocks_per_seq, max_seq_len, max_q_len, total_q;
    int num_seqs, num_heads, num_kv_heads, head_dim, num_blocks, block_size;
    float scale_log2;
    void *slots;                  // partial results of cut segments, or NULL: nothing is cut
    uint64_t wait_limit_ns;       // bounded waits (0 = 1 s)
    int stall_tile;               // self-test of the bounded waits (0 = off)
    const int32_t *lens_ahead, *cu_ahead;   // self-test of the second look at the lengths (NULL = off)
    unsigned int *err;
};

// Largest persistent grid (one CTA an SM; the workspace has two slots for each).
constexpr int kRowsMaxCtas = 160;
size_t rows_workspace_bytes(int num_heads, int num_kv_heads, int head_dim, int max_q_len);
cudaError_t launch_rows_attention(const RowsParams &p, cudaStream_t stream);

}  // namespace pk
