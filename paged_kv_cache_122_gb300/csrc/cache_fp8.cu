// Byte movers of the 8-bit paged cache [num_blocks, num_kv_heads, block_size,
// head_dim]: block copies with their scales, and the gather that gives rows
// back as bf16.  The roofline of both is HBM bandwidth.
#include "../../include/pagedkv_fp8.h"
#include "fp8.cuh"

#include <algorithm>

namespace {

constexpr int kThreads = 256;
constexpr int kCopyVecsPerCta = kThreads * 4;

struct Pool {
    uint4 *k, *v;
    float *k_scales, *v_scales;
    int num_blocks;
};

// grid = (pairs, 2 [K, V], chunks of one block): each thread keeps four
// 16-byte reads in flight before it writes; chunk 0 moves the block's scales.
__global__ void __launch_bounds__(kThreads)
move_blocks_fp8_kernel(const Pool dst, const Pool src, const int64_t *pairs, int64_t block_vecs,
                       int num_kv_heads, unsigned int *err) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t pair = blockIdx.x;
    const int64_t from = pairs[2 * pair], to = pairs[2 * pair + 1];
    if (from < 0 || from >= src.num_blocks || to < 0 || to >= dst.num_blocks) {
        if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) pk::set_error(err, PK_DEVERR_PAIR);
        return;
    }
    const uint4 *s = (blockIdx.y ? src.v : src.k) + from * block_vecs;
    uint4 *d = (blockIdx.y ? dst.v : dst.k) + to * block_vecs;
    const int64_t lo = static_cast<int64_t>(blockIdx.z) * kCopyVecsPerCta;
    const int64_t hi = min(lo + kCopyVecsPerCta, block_vecs);
    uint4 buf[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t e = lo + u * kThreads + threadIdx.x;
        if (e < hi) buf[u] = s[e];
    }
    if (blockIdx.z == 0) {
        const float *ss = (blockIdx.y ? src.v_scales : src.k_scales) + from * num_kv_heads;
        float *ds = (blockIdx.y ? dst.v_scales : dst.k_scales) + to * num_kv_heads;
        for (int h = threadIdx.x; h < num_kv_heads; h += kThreads) ds[h] = ss[h];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t e = lo + u * kThreads + threadIdx.x;
        if (e < hi) d[e] = buf[u];
    }
}

// grid = (num_seqs, y): CTA y of a sequence takes its token chunks y, y +
// gridDim.y, ...; a thread turns 8 values (8 bytes) of one row into 8 bf16 (16
// bytes), so that a warp's reads and writes are whole 256- and 512-byte runs.
constexpr int kGatherTokens = 32;
constexpr int kGatherBatch = 4;

template <int D>
__global__ void __launch_bounds__(kThreads)
gather_kv_fp8_kernel(uint4 *out_k, uint4 *out_v, const uint2 *k_cache, const uint2 *v_cache, const float *k_scales,
                     const float *v_scales, const int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens,
                     const int64_t *cu_seq_lens, int64_t out_rows, int max_seq_len, int num_kv_heads, int num_blocks,
                     int log2_block, unsigned int *err) {
    // (No __restrict__: what the previous kernel wrote may not be read ahead of the wait.)
    constexpr int kVecs = D / 8;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int s = blockIdx.x;
    const int B = 1 << log2_block;
    int L = seq_lens[s];
    const int cap = static_cast<int>(min(static_cast<int64_t>(max_seq_len), static_cast<int64_t>(max_blocks_per_seq) * B));
    if (L < 0 || L > cap) {
        if (blockIdx.y == 0 && threadIdx.x == 0) pk::set_error(err, PK_DEVERR_SEQ_LEN);
        L = L < 0 ? 0 : cap;
    }
    const int64_t base = cu_seq_lens[s];
    if (base < 0 || base > out_rows - L) {        // rows outside the output: nothing of the sequence
        if (blockIdx.y == 0 && threadIdx.x == 0 && L > 0) pk::set_error(err, PK_DEVERR_SEQ_LEN);
        return;
    }
    const int32_t *table = block_tables + static_cast<int64_t>(s) * max_blocks_per_seq;
    const int row_vecs = num_kv_heads * kVecs;
    for (int64_t j0 = static_cast<int64_t>(blockIdx.y) * kGatherTokens; j0 < L;
         j0 += static_cast<int64_t>(gridDim.y) * kGatherTokens) {
        const int nj = static_cast<int>(min(static_cast<int64_t>(kGatherTokens), L - j0));
        const int total = nj * row_vecs;
        for (int i0 = 0; i0 < total; i0 += kThreads * kGatherBatch) {
            uint2 kw[kGatherBatch], vw[kGatherBatch];
            float ks[kGatherBatch], vs[kGatherBatch];
            int64_t dst[kGatherBatch];
#pragma unroll
            for (int u = 0; u < kGatherBatch; ++u) {
                const int i = i0 + u * kThreads + static_cast<int>(threadIdx.x);
                dst[u] = -1;
                if (i >= total) continue;
                const int jj = i / row_vecs, e = i - jj * row_vecs;
                const int h = e / kVecs;
                const int j = static_cast<int>(j0) + jj;
                const int blk = table[j >> log2_block];
                if (blk < 0 || blk >= num_blocks) {
                    if (e == 0) pk::set_error(err, PK_DEVERR_BLOCK_ID);
                    continue;
                }
                const int64_t cell = static_cast<int64_t>(blk) * num_kv_heads + h;
                const int64_t src = ((cell << log2_block) + (j & (B - 1))) * kVecs + (e % kVecs);
                kw[u] = __ldcs(k_cache + src);
                vw[u] = __ldcs(v_cache + src);
                ks[u] = k_scales[cell];
                vs[u] = v_scales[cell];
                dst[u] = (base + j) * row_vecs + e;
            }
#pragma unroll
            for (int u = 0; u < kGatherBatch; ++u) {
                if (dst[u] < 0) continue;
                if (!pk::scale_ok(ks[u]) || !pk::scale_ok(vs[u])) {
                    pk::set_error(err, PK_DEVERR_SCALE);
                    continue;
                }
                auto widen = [](const uint2 &w, float scale) {
                    float lo[4], hi[4];
                    pk::e4m3x4_to_float(w.x, lo);
                    pk::e4m3x4_to_float(w.y, hi);
                    return make_uint4(pk::pack_bf16x2(lo[0] * scale, lo[1] * scale),
                                      pk::pack_bf16x2(lo[2] * scale, lo[3] * scale),
                                      pk::pack_bf16x2(hi[0] * scale, hi[1] * scale),
                                      pk::pack_bf16x2(hi[2] * scale, hi[3] * scale));
                };
                out_k[dst[u]] = widen(kw[u], ks[u]);
                out_v[dst[u]] = widen(vw[u], vs[u]);
            }
        }
    }
}

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, cudaStream_t stream, Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

bool supported_geometry(int head_dim, int block_size) {
    return (head_dim == 64 || head_dim == 128) && (block_size == 8 || block_size == 16 || block_size == 32);
}

int move_blocks(const Pool &dst, const Pool &src, const int64_t *pairs, int num_pairs, int num_kv_heads, int head_dim,
                int block_size, pk_stream_t stream) {
    if (num_pairs < 0 || src.num_blocks < 0 || dst.num_blocks < 0 || num_kv_heads <= 0 || block_size <= 0)
        return PK_ERR_SHAPE;
    if (!supported_geometry(head_dim, block_size)) return PK_ERR_UNSUPPORTED;
    if (num_pairs == 0) return PK_OK;
    for (const Pool *p : {&dst, &src}) {
        if (!p->k || !p->v || !p->k_scales || !p->v_scales) return PK_ERR_NULL;
        if (!pk::aligned16(p->k) || !pk::aligned16(p->v)) return PK_ERR_ALIGNMENT;
    }
    if (!pairs) return PK_ERR_NULL;
    const int64_t block_vecs = static_cast<int64_t>(block_size) * num_kv_heads * head_dim / 16;
    const int64_t chunks = (block_vecs + kCopyVecsPerCta - 1) / kCopyVecsPerCta;
    if (chunks > 65535) return PK_ERR_SHAPE;
    unsigned int *err = pk::error_word_ptr();
    if (!err) return PK_ERR_NO_DEVICE;
    const dim3 grid(static_cast<unsigned>(num_pairs), 2, static_cast<unsigned>(chunks));
    return launch_dependent(move_blocks_fp8_kernel, grid, reinterpret_cast<cudaStream_t>(stream), dst, src, pairs,
                            block_vecs, num_kv_heads, err) == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

Pool pool_of(const void *k, const void *v, const float *k_scales, const float *v_scales, int num_blocks) {
    return Pool{const_cast<uint4 *>(static_cast<const uint4 *>(k)), const_cast<uint4 *>(static_cast<const uint4 *>(v)),
                const_cast<float *>(k_scales), const_cast<float *>(v_scales), num_blocks};
}

}  // namespace

extern "C" int pk_copy_blocks_fp8(void *k_cache, void *v_cache, float *k_scales, float *v_scales,
                                  const int64_t *src_dst_pairs, int num_pairs, int num_kv_heads, int head_dim,
                                  int num_blocks, int block_size, pk_stream_t stream) {
    const Pool pool = pool_of(k_cache, v_cache, k_scales, v_scales, num_blocks);
    return move_blocks(pool, pool, src_dst_pairs, num_pairs, num_kv_heads, head_dim, block_size, stream);
}

extern "C" int pk_swap_blocks_fp8(void *dst_k, void *dst_v, float *dst_k_scales, float *dst_v_scales,
                                  const void *src_k, const void *src_v, const float *src_k_scales,
                                  const float *src_v_scales, const int64_t *pairs, int num_pairs, int num_kv_heads,
                                  int head_dim, int block_size, int src_num_blocks, int dst_num_blocks,
                                  pk_stream_t stream) {
    return move_blocks(pool_of(dst_k, dst_v, dst_k_scales, dst_v_scales, dst_num_blocks),
                       pool_of(src_k, src_v, src_k_scales, src_v_scales, src_num_blocks), pairs, num_pairs,
                       num_kv_heads, head_dim, block_size, stream);
}

extern "C" int pk_gather_kv_fp8(void *out_k, void *out_v, const void *k_cache, const void *v_cache,
                                const float *k_scales, const float *v_scales, const int32_t *block_tables,
                                int max_blocks_per_seq, const int32_t *seq_lens, const int64_t *cu_seq_lens,
                                int64_t out_rows, int max_seq_len, int num_seqs, int num_kv_heads, int head_dim, int num_blocks,
                                int block_size, pk_stream_t stream) {
    if (num_seqs < 0 || num_blocks < 0 || max_blocks_per_seq < 0 || max_seq_len < 0 || num_kv_heads <= 0 ||
        block_size <= 0 || out_rows < 0)
        return PK_ERR_SHAPE;
    if (!supported_geometry(head_dim, block_size)) return PK_ERR_UNSUPPORTED;
    if (num_kv_heads > 32767) return PK_ERR_SHAPE;
    if (static_cast<int64_t>(max_seq_len) > static_cast<int64_t>(max_blocks_per_seq) * block_size)
        return PK_ERR_SHAPE;
    if (num_seqs == 0 || max_seq_len == 0 || out_rows == 0) return PK_OK;
    if (!out_k || !out_v || !k_cache || !v_cache || !k_scales || !v_scales || !block_tables || !seq_lens ||
        !cu_seq_lens)
        return PK_ERR_NULL;
    if (!pk::aligned16(out_k) || !pk::aligned16(out_v) || !pk::aligned16(k_cache) || !pk::aligned16(v_cache))
        return PK_ERR_ALIGNMENT;
    unsigned int *err = pk::error_word_ptr();
    const int sms = pk::sm_count();
    if (!err || sms <= 0) return PK_ERR_NO_DEVICE;
    // Enough CTAs for several rounds on every SM, however the tokens are
    // spread over the sequences; a CTA walks its sequence's chunks.
    const int64_t chunks = (static_cast<int64_t>(max_seq_len) + kGatherTokens - 1) / kGatherTokens;
    const int64_t most = std::max<int64_t>(1, 64ll * sms / num_seqs);
    const dim3 grid(static_cast<unsigned>(num_seqs),
                    static_cast<unsigned>(std::min<int64_t>(65535, std::min(chunks, most))));
    const int log2_block = block_size == 8 ? 3 : block_size == 16 ? 4 : 5;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    auto *kernel = head_dim == 64 ? gather_kv_fp8_kernel<64> : gather_kv_fp8_kernel<128>;
    return launch_dependent(kernel, grid, st, static_cast<uint4 *>(out_k), static_cast<uint4 *>(out_v),
                            static_cast<const uint2 *>(k_cache), static_cast<const uint2 *>(v_cache), k_scales,
                            v_scales, block_tables, max_blocks_per_seq, seq_lens, cu_seq_lens, out_rows, max_seq_len,
                            num_kv_heads, num_blocks, log2_block, err) == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}
