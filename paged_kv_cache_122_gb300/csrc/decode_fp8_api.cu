// Host entry points of attention over the 8-bit paged cache: argument checks
// and the launch.
#include "decode_fp8.cuh"

#include <cmath>

namespace {

// max_seq_len == 0: every sequence is empty, so nothing of the cache is read and
// the work is the rows' zeros.  CTA s checks sequence s as the attention kernel
// does and writes its rows alone (not whole `out`: rows that no sequence owns, or
// one whose rows are bad, stay as they are).
__global__ void __launch_bounds__(128) empty_sequences_kernel(const pk::DecodeParams p) {
    const int s = blockIdx.x;
    int r0 = s, r1 = s + 1;
    bool bad = p.seq_lens[s] != 0;
    if (p.cu_q_lens) {
        r0 = p.cu_q_lens[s];
        r1 = p.cu_q_lens[s + 1];
        bad = bad || r1 != r0;                      // more queries than tokens, or rows that run backwards
    }
    if (bad && threadIdx.x == 0) pk::set_error(p.err, PK_DEVERR_SEQ_LEN);
    if (p.cu_q_lens && (r0 < 0 || r1 < r0 || r1 > p.total_q || r1 - r0 > p.q_len)) return;
    const int64_t row = static_cast<int64_t>(p.num_heads) * p.head_dim * (p.out_fp32 ? 4 : 2) / 16;
    uint4 *out = static_cast<uint4 *>(p.out) + r0 * row;
    for (int64_t i = threadIdx.x; i < (r1 - r0) * row; i += blockDim.x) out[i] = make_uint4(0, 0, 0, 0);
}

bool group_supported(int G) { return G == 1 || G == 2 || G == 4 || G == 8 || G == 16; }

// Both calls; cu_q_lens is NULL for one query token a sequence.  `stall_tile` and
// `wait_limit_ns` serve the self-test of the bounded waits (0 = off / the default
// limit), `lens_ahead` that of the second look at the lengths (NULL = off).
int attend(void *out, int out_dtype, const void *q, int total_q, const int32_t *cu_q_lens, int max_q_len,
           const void *k_cache, const void *v_cache, const float *k_scales, const float *v_scales,
           const int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens, int max_seq_len, int num_seqs,
           int num_heads, int num_kv_heads, int head_dim, int num_blocks, int block_size, float scale, void *workspace,
           size_t workspace_bytes, pk_stream_t stream, bool multi, int stall_tile = 0, uint64_t wait_limit_ns = 0,
           const int32_t *lens_ahead = nullptr) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_blocks < 0 || max_blocks_per_seq < 0 ||
        max_seq_len < 0 || block_size <= 0 || total_q < 0 || max_q_len < 0)
        return PK_ERR_SHAPE;
    if (num_heads % num_kv_heads) return PK_ERR_SHAPE;
    if (static_cast<int64_t>(max_seq_len) > static_cast<int64_t>(max_blocks_per_seq) * block_size)
        return PK_ERR_SHAPE;
    if (out_dtype != PK_BF16 && out_dtype != PK_FP32) return PK_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PK_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PK_ERR_UNSUPPORTED;
    const int G = num_heads / num_kv_heads;
    if (!group_supported(G)) return PK_ERR_UNSUPPORTED;
    int q_len = 1;                                  // query tokens a sequence, padded to a power of two
    while (q_len < max_q_len && q_len <= 16) q_len <<= 1;
    if (G * q_len > 16) return PK_ERR_UNSUPPORTED;
    if (!std::isfinite(scale)) return PK_ERR_SHAPE;
    // A piece (block, KV head) is one step of a TMA coordinate.
    if (num_seqs > 65535 || num_kv_heads * 2 > 65535 ||
        static_cast<int64_t>(num_blocks) * num_kv_heads > 0x7fffffff)
        return PK_ERR_SHAPE;
    if (num_seqs == 0 || total_q == 0) return PK_OK;
    if (!out || !q || !seq_lens || (multi && !cu_q_lens) ||
        (max_seq_len > 0 && (!k_cache || !v_cache || !k_scales || !v_scales || !block_tables)))
        return PK_ERR_NULL;
    if (!pk::aligned16(out) || !pk::aligned16(q) || !pk::aligned16(k_cache) || !pk::aligned16(v_cache))
        return PK_ERR_ALIGNMENT;

    pk::DecodeFp8Params p{};
    p.out = out;
    p.out_fp32 = out_dtype == PK_FP32;
    p.q = static_cast<const uint16_t *>(q);
    p.k8 = static_cast<const uint8_t *>(k_cache);
    p.v8 = static_cast<const uint8_t *>(v_cache);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_seq_len = max_seq_len;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.scale_log2 = scale * pk::kLog2e;
    p.cu_q_lens = cu_q_lens;
    p.q_len = q_len;
    p.total_q = total_q;
    p.stall_tile = stall_tile;
    p.wait_limit_ns = wait_limit_ns;
    p.lens_ahead = lens_ahead;
    if (max_seq_len > 128) {       // a longer sequence may span several CTAs: its parts need slots
        if (!workspace || workspace_bytes < pk::tc_workspace_bytes()) return PK_ERR_WORKSPACE;
        if (!pk::aligned16(workspace)) return PK_ERR_ALIGNMENT;
        p.tc_slots = workspace;
    }
    p.err = pk::error_word_ptr();
    if (!p.err) return PK_ERR_NO_DEVICE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (max_seq_len == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(num_seqs));
        cfg.blockDim = dim3(128);
        cfg.stream = st;
        return cudaLaunchKernelEx(&cfg, empty_sequences_kernel, static_cast<const pk::DecodeParams &>(p)) == cudaSuccess
                   ? PK_OK : PK_ERR_CUDA;
    }
    return pk::launch_decode_fp8_tensor_core(p, st) == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

}  // namespace

extern "C" size_t pk_decode_fp8_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                                int max_seq_len) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || max_seq_len < 0) return 0;
    if (num_heads % num_kv_heads) return 0;
    if (head_dim != 64 && head_dim != 128) return 0;
    return max_seq_len > 128 ? pk::tc_workspace_bytes() : 0;
}

extern "C" int pk_paged_attention_decode_fp8(void *out, int out_dtype, const void *q, const void *k_cache,
                                             const void *v_cache, const float *k_scales, const float *v_scales,
                                             const int32_t *block_tables, int max_blocks_per_seq,
                                             const int32_t *seq_lens, int max_seq_len, int num_seqs, int num_heads,
                                             int num_kv_heads, int head_dim, int num_blocks, int block_size,
                                             float scale, void *workspace, size_t workspace_bytes,
                                             pk_stream_t stream) {
    return attend(out, out_dtype, q, num_seqs, nullptr, 1, k_cache, v_cache, k_scales, v_scales, block_tables,
                  max_blocks_per_seq, seq_lens, max_seq_len, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks,
                  block_size, scale, workspace, workspace_bytes, stream, false);
}

extern "C" int pk_selftest_decode_fp8_wait_timeout(void *out, int out_dtype, const void *q, const void *k_cache,
                                                   const void *v_cache, const float *k_scales, const float *v_scales,
                                                   const int32_t *block_tables, int max_blocks_per_seq,
                                                   const int32_t *seq_lens, int max_seq_len, int num_seqs, int num_heads,
                                                   int num_kv_heads, int head_dim, int num_blocks, int block_size,
                                                   float scale, void *workspace, size_t workspace_bytes, int stall_tile,
                                                   unsigned int wait_limit_us, pk_stream_t stream) {
    if (stall_tile < 1 || wait_limit_us < 100 || wait_limit_us > 1000000) return PK_ERR_SHAPE;
    return attend(out, out_dtype, q, num_seqs, nullptr, 1, k_cache, v_cache, k_scales, v_scales, block_tables,
                  max_blocks_per_seq, seq_lens, max_seq_len, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks,
                  block_size, scale, workspace, workspace_bytes, stream, false, stall_tile,
                  static_cast<uint64_t>(wait_limit_us) * 1000u);
}

extern "C" int pk_selftest_decode_fp8_stale_lengths(void *out, int out_dtype, const void *q, const void *k_cache,
                                                    const void *v_cache, const float *k_scales, const float *v_scales,
                                                    const int32_t *block_tables, int max_blocks_per_seq,
                                                    const int32_t *seq_lens, int max_seq_len, int num_seqs, int num_heads,
                                                    int num_kv_heads, int head_dim, int num_blocks, int block_size,
                                                    float scale, const int32_t *stale_seq_lens, void *workspace,
                                                    size_t workspace_bytes, pk_stream_t stream) {
    if (!stale_seq_lens) return PK_ERR_NULL;
    return attend(out, out_dtype, q, num_seqs, nullptr, 1, k_cache, v_cache, k_scales, v_scales, block_tables,
                  max_blocks_per_seq, seq_lens, max_seq_len, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks,
                  block_size, scale, workspace, workspace_bytes, stream, false, 0, 0, stale_seq_lens);
}

extern "C" int pk_paged_attention_multi_query_fp8(void *out, int out_dtype, const void *q, int total_q,
                                                  const int32_t *cu_q_lens, int max_q_len, const void *k_cache,
                                                  const void *v_cache, const float *k_scales, const float *v_scales,
                                                  const int32_t *block_tables, int max_blocks_per_seq,
                                                  const int32_t *seq_lens, int max_seq_len, int num_seqs,
                                                  int num_heads, int num_kv_heads, int head_dim, int num_blocks,
                                                  int block_size, float scale, void *workspace,
                                                  size_t workspace_bytes, pk_stream_t stream) {
    return attend(out, out_dtype, q, total_q, cu_q_lens, max_q_len, k_cache, v_cache, k_scales, v_scales,
                  block_tables, max_blocks_per_seq, seq_lens, max_seq_len, num_seqs, num_heads, num_kv_heads, head_dim,
                  num_blocks, block_size, scale, workspace, workspace_bytes, stream, true);
}
