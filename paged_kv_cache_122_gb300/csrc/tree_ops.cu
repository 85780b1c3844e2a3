// The accepted path of each tree of drafted tokens, and the move of its K and V
// rows together in the paged cache.
#include "../../include/pagedkv_tree.h"
#include "common.cuh"

#include <algorithm>

namespace {

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                             Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// ------------------------------------------------------------------ accept_tree
// One CTA per sequence.  next[p], the lowest node c with parent p and the token
// that the target chose after p, is a minimum over the nodes, so all nodes are
// looked at side by side; the path is then a chain of shared-memory reads by one
// thread.  Bound by two dependent trips to memory (node -> its parent's target).
constexpr int kAcceptThreads = 128;
constexpr int kMaxTree = 8192;      // next[], which the path is written over, in 32 KB
constexpr int kNone = 0x7fffffff;

__global__ void __launch_bounds__(kAcceptThreads)
accept_tree_kernel(int32_t *accepted, int32_t *num_accepted, int64_t *next_tokens, int32_t *new_seq_lens,
                   const int64_t *draft_tokens, const int32_t *parents, const int64_t *target_tokens, int total_q,
                   const int32_t *cu_q_lens, int max_q_len, const int32_t *seq_lens, unsigned int *err) {
    extern __shared__ int32_t next[];
    __shared__ int path_len;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int s = blockIdx.x;
    const int L = seq_lens[s], q0 = cu_q_lens[s], q1 = cu_q_lens[s + 1];
    const bool bad = L < 0 || q0 < 0 || q1 < q0 || q1 > total_q || q1 - q0 > max_q_len || q1 - q0 > L;
    const int n = bad ? 0 : q1 - q0;
    if (bad && threadIdx.x == 0) pk::set_error(err, PK_DEVERR_SEQ_LEN);
    for (int i = threadIdx.x; i < n; i += kAcceptThreads) next[i] = kNone;
    __syncthreads();
    for (int c = 1 + threadIdx.x; c < n; c += kAcceptThreads) {
        const int p = parents[q0 + c];
        if (p < 0 || p >= c) continue;
        if (draft_tokens[q0 + c] == target_tokens[q0 + p]) atomicMin(&next[p], c);
    }
    __syncthreads();
    // The path in place: entry i of the path goes where next[] of a node before it
    // was (path nodes increase, so node i's entry has been read when i <= node).
    if (threadIdx.x == 0) {
        int len = 0, last = -1;
        for (int node = n > 0 ? 0 : kNone; node != kNone;) {
            const int following = next[node];
            next[len++] = node;
            last = node;
            node = following;
        }
        path_len = len;
        num_accepted[s] = len;
        next_tokens[s] = last >= 0 ? target_tokens[q0 + last] : -1;
        new_seq_lens[s] = L - n + len;
    }
    __syncthreads();
    const int len = path_len;
    int32_t *row = accepted + static_cast<size_t>(s) * max_q_len;
    for (int i = threadIdx.x; i < max_q_len; i += kAcceptThreads) row[i] = i < len ? next[i] : -1;
}

// ------------------------------------------------------------------ keep_tokens
// One CTA per sequence and group of layers.  It checks the list and looks up the rows'
// places once (a chunk of tokens at a time), then moves them in each of its layers' K
// and V.  A unit of a warp is 512 bytes of a row; a pass takes kKeepUnits a warp: all
// are read, then all are written.  Lists increase strictly, so accepted[i] >= i, tokens
// in their place are a prefix, and a row that a pass writes (i) comes before every row
// that a later pass reads (accepted[j] >= j > i).  Bound by memory: two rows moved for
// each kept token that is not in its place.  (A CTA per layer, K or V and sequence
// looked everything up 64 times for 32 layers: 25 us where this takes 17, for 128
// sequences.)
constexpr int kKeepThreads = 256;
constexpr int kKeepWarps = kKeepThreads / 32;
constexpr int kKeepUnits = 8;
constexpr int kKeepChunk = 256;      // tokens whose places are looked up together
constexpr int kKeepGroup = 64;       // layers of a CTA (at most)

struct KeepParams {
    uint4 *k_cache, *v_cache;                 // one layer, or
    uint4 *const *k_layers, *const *v_layers; // a device array of them
    const int32_t *block_tables;
    int max_blocks_per_seq;
    const int32_t *seq_lens, *cu_q_lens, *accepted;
    int accepted_stride;
    const int32_t *num_accepted;
    int row_vecs, num_blocks, log2_block;
    int num_layers, group;                    // layers; layers of a CTA
    unsigned int *err;
};

__global__ void __launch_bounds__(kKeepThreads)
keep_tokens_kernel(const KeepParams p) {
    __shared__ int64_t src[kKeepChunk], dst[kKeepChunk];
    __shared__ uint4 *caches[kKeepGroup][2];     // K and V of the layers; NULL for a layer to leave alone
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int s = blockIdx.x, layer0 = blockIdx.y * p.group, layers = min(p.group, p.num_layers - layer0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool reports = blockIdx.y == 0 && threadIdx.x == 0;
    const int L = p.seq_lens[s], q0 = p.cu_q_lens[s], q1 = p.cu_q_lens[s + 1];
    const int n = p.num_accepted[s];
    // The layers' pointers, a thread each: on their way while the list is checked.
    static_assert(kKeepGroup <= kKeepThreads, "a thread for each layer");
    const int mine = static_cast<int>(threadIdx.x) < layers ? layer0 + static_cast<int>(threadIdx.x) : -1;
    uint4 *own_k = p.k_cache, *own_v = p.v_cache;
    if (mine >= 0 && p.k_layers) {
        own_k = p.k_layers[mine];
        own_v = p.v_layers[mine];
    }
    const int32_t *list = p.accepted + static_cast<size_t>(s) * p.accepted_stride;
    const int64_t cap = static_cast<int64_t>(p.max_blocks_per_seq) << p.log2_block;
    // A layer of which K or V cannot be used is left alone, both of them: its rows have to
    // stay those of the same tokens.  (Reported by the first sequence's CTAs.)
    auto put_pointers = [&]() {
        if (mine < 0) return;
        const bool ok = own_k && own_v && !((reinterpret_cast<uintptr_t>(own_k) | reinterpret_cast<uintptr_t>(own_v)) & 15u);
        if (!ok && s == 0) pk::set_error(p.err, PK_DEVERR_POINTER);
        caches[threadIdx.x][0] = ok ? own_k : nullptr;
        caches[threadIdx.x][1] = ok ? own_v : nullptr;
    };
    if (L < 0 || L > cap || q0 < 0 || q1 < q0 || q1 - q0 > L) {
        if (reports) pk::set_error(p.err, PK_DEVERR_SEQ_LEN);
        put_pointers();
        return;
    }
    const int nodes = q1 - q0;
    bool bad = n < 0 || n > nodes || n > p.accepted_stride;
    int moved = 0;                               // tokens that are not in their place
    if (!bad)
        for (int i = threadIdx.x; i < n; i += kKeepThreads) {
            const int at = list[i];
            bad |= at >= nodes || at <= (i > 0 ? list[i - 1] : -1);
            moved += at != i;
        }
    put_pointers();
    if (__syncthreads_or(bad)) {
        if (reports) pk::set_error(p.err, PK_DEVERR_DRAFT);
        return;
    }
    __shared__ int total;
    if (threadIdx.x == 0) total = 0;
    __syncthreads();
    if (moved) atomicAdd(&total, moved);
    __syncthreads();
    const int first = n - total;                 // (integer sum: the order does not matter)
    const int32_t *table = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
    const int B1 = (1 << p.log2_block) - 1;
    const int base = L - nodes;
    const int segs = (p.row_vecs + 31) >> 5;     // units of a row
    for (int i0 = first; i0 < n; i0 += kKeepChunk) {
        const int count = min(kKeepChunk, n - i0);
        __syncthreads();                         // the last chunk's places have been used
        for (int j = threadIdx.x; j < count; j += kKeepThreads) {
            const int sp = base + list[i0 + j], dp = base + i0 + j;
            const int sb = table[sp >> p.log2_block], db = table[dp >> p.log2_block];
            const bool ok = sb >= 0 && sb < p.num_blocks && db >= 0 && db < p.num_blocks;
            if (!ok) pk::set_error(p.err, PK_DEVERR_BLOCK_ID);
            src[j] = ok ? ((static_cast<int64_t>(sb) << p.log2_block) + (sp & B1)) * p.row_vecs : -1;
            dst[j] = ((static_cast<int64_t>(db) << p.log2_block) + (dp & B1)) * p.row_vecs;
        }
        __syncthreads();
        // Units in the order (layer, K or V, token, piece of its row): of one cache, a
        // pass's tokens come before the next pass's.
        const uint32_t row_units = static_cast<uint32_t>(count) * segs;
        const uint32_t units = row_units * 2 * layers;          // (kKeepGroup keeps it within 32 bits)
        uint32_t per;
        for (uint32_t u0 = 0; u0 < units; u0 += kKeepWarps * per) {
            per = min(static_cast<uint32_t>(kKeepUnits), (units - u0 + kKeepWarps - 1) / kKeepWarps);
            uint4 buf[kKeepUnits];
            uint4 *to[kKeepUnits];
            // A warp's units of the pass lie one behind the other: one division a pass.
            uint32_t unit = u0 + warp * per;
            uint32_t lk = unit / row_units, j = unit % row_units / segs, seg = unit % row_units % segs;
#pragma unroll
            for (int u = 0; u < kKeepUnits; ++u, ++unit) {
                to[u] = nullptr;
                if (static_cast<uint32_t>(u) < per && unit < units) {
                    const uint32_t col = seg * 32 + lane;
                    uint4 *cache = caches[lk >> 1][lk & 1];
                    if (src[j] >= 0 && col < static_cast<uint32_t>(p.row_vecs) && cache) {
                        buf[u] = cache[src[j] + col];
                        to[u] = cache + dst[j] + col;
                    }
                }
                if (++seg == static_cast<uint32_t>(segs)) {
                    seg = 0;
                    if (++j == static_cast<uint32_t>(count)) {
                        j = 0;
                        ++lk;
                    }
                }
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kKeepUnits; ++u)
                if (to[u]) *to[u] = buf[u];
        }
    }
}

int keep(KeepParams &p, const void *const *ptrs, int num_seqs, int num_layers, int num_kv_heads, int head_dim,
         int block_size, bool check_alignment, pk_stream_t stream) {
    if (num_seqs < 0 || p.max_blocks_per_seq < 0 || p.accepted_stride < 0 || num_kv_heads <= 0 || p.num_blocks < 0 ||
        block_size <= 0 || num_layers < 0)
        return PK_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128) return PK_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PK_ERR_UNSUPPORTED;
    if (num_seqs > 65535 || num_layers > 32767 || num_kv_heads > 65535) return PK_ERR_SHAPE;
    if (num_seqs == 0 || num_layers == 0 || p.accepted_stride == 0 || p.max_blocks_per_seq == 0) return PK_OK;
    if (!ptrs[0] || !ptrs[1] || !p.block_tables || !p.seq_lens || !p.cu_q_lens || !p.accepted || !p.num_accepted)
        return PK_ERR_NULL;
    if (check_alignment && (!pk::aligned16(ptrs[0]) || !pk::aligned16(ptrs[1]))) return PK_ERR_ALIGNMENT;
    p.row_vecs = num_kv_heads * head_dim / 8;
    p.log2_block = block_size == 8 ? 3 : block_size == 16 ? 4 : 5;
    p.err = pk::error_word_ptr();
    const int sms = pk::sm_count();
    if (!p.err || sms <= 0) return PK_ERR_NO_DEVICE;
    // As many layers to a CTA as still leave eight CTAs for each SM (128 sequences, 32 layers: 17 us;
    // measured when eight took 18: four for each SM 20, two 23, one layer to a CTA 24).
    p.num_layers = num_layers;
    p.group = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kKeepGroup, static_cast<int64_t>(num_seqs) * num_layers / (8 * sms))));
    const dim3 grid(num_seqs, (num_layers + p.group - 1) / p.group);
    return launch_dependent(keep_tokens_kernel, grid, kKeepThreads, 0, reinterpret_cast<cudaStream_t>(stream), p) ==
                   cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

}  // namespace

extern "C" int pk_accept_tree(int32_t *accepted, int32_t *num_accepted, int64_t *next_tokens, int32_t *new_seq_lens,
                              const int64_t *draft_tokens, const int32_t *parents, const int64_t *target_tokens,
                              int total_q, const int32_t *cu_q_lens, int max_q_len, const int32_t *seq_lens,
                              int num_seqs, pk_stream_t stream) {
    if (total_q < 0 || max_q_len < 0 || num_seqs < 0) return PK_ERR_SHAPE;
    if (max_q_len > kMaxTree) return PK_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PK_OK;
    if (!num_accepted || !next_tokens || !new_seq_lens || !cu_q_lens || !seq_lens || (max_q_len > 0 && !accepted) ||
        (total_q > 0 && (!draft_tokens || !parents || !target_tokens)))
        return PK_ERR_NULL;
    unsigned int *err = pk::error_word_ptr();
    if (!err) return PK_ERR_NO_DEVICE;
    return launch_dependent(accept_tree_kernel, dim3(num_seqs), kAcceptThreads, max_q_len * sizeof(int32_t),
                            reinterpret_cast<cudaStream_t>(stream), accepted, num_accepted, next_tokens, new_seq_lens,
                            draft_tokens, parents, target_tokens, total_q, cu_q_lens, max_q_len, seq_lens, err) ==
                   cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

extern "C" int pk_keep_tokens(void *k_cache, void *v_cache, const int32_t *block_tables, int max_blocks_per_seq,
                              const int32_t *seq_lens, const int32_t *cu_q_lens, const int32_t *accepted,
                              int accepted_stride, const int32_t *num_accepted, int num_seqs, int num_kv_heads,
                              int head_dim, int num_blocks, int block_size, pk_stream_t stream) {
    const void *ptrs[2] = {k_cache, v_cache};
    KeepParams p{static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache), nullptr, nullptr, block_tables,
                 max_blocks_per_seq, seq_lens, cu_q_lens, accepted, accepted_stride, num_accepted, 0, num_blocks, 0,
                 0, 0, nullptr};
    return keep(p, ptrs, num_seqs, 1, num_kv_heads, head_dim, block_size, true, stream);
}

extern "C" int pk_keep_tokens_layers(void *const *k_cache_layers, void *const *v_cache_layers,
                                     const int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens,
                                     const int32_t *cu_q_lens, const int32_t *accepted, int accepted_stride,
                                     const int32_t *num_accepted, int num_seqs, int num_layers, int num_kv_heads,
                                     int head_dim, int num_blocks, int block_size, pk_stream_t stream) {
    const void *ptrs[2] = {k_cache_layers, v_cache_layers};
    KeepParams p{nullptr, nullptr, reinterpret_cast<uint4 *const *>(k_cache_layers),
                 reinterpret_cast<uint4 *const *>(v_cache_layers), block_tables, max_blocks_per_seq, seq_lens, cu_q_lens,
                 accepted, accepted_stride, num_accepted, 0, num_blocks, 0, 0, 0, nullptr};
    return keep(p, ptrs, num_seqs, num_layers, num_kv_heads, head_dim, block_size, false, stream);
}
