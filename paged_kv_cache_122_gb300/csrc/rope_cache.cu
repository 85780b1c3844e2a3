// Rotary positions and the append to the bf16 paged cache, in one pass.
//
// A byte mover: each new token's q, k and v are read once and written once
// (4 H D + 8 Hkv D bytes a token), with three multiply-adds an element in
// between, so the roofline is HBM bandwidth, and the launch for a few tokens.
// One CTA a token: its rot / 2 (cos, sin) pairs are computed once and kept in
// shared memory for all of its heads, while the token's vectors are already
// on their way.  The angles come from the position and the frequency (see
// rope.cuh), not from a table, so no position is out of range and no table is
// read.  8,192 tokens of 64 + 16 heads of 128 take 53.3 us (336 MB, 0.93 of a
// copy's rate), four tokens of 24 heads of 64 2.0 us back to back.
#include "rope.cuh"

namespace {

constexpr int kMaxThreads = 256;
// Eight CTAs an SM, one unit (2 x 16 bytes) of a thread in flight: 64 KiB an SM
// either way, but more CTAs cover one another's start and end (8,192 tokens of
// 64 + 16 heads: 53.3 us; four units a thread with four CTAs: 61 us).
constexpr int kCtasPerSm = 8;

struct RopeParams {
    uint16_t *q_out;
    const uint16_t *q, *k, *v;
    int64_t q_out_stride, q_stride, k_stride, v_stride;
    uint16_t *k_cache, *v_cache;
    const int64_t *slot_mapping, *positions;
    const float *inv_freq;
    int rot, num_heads, num_kv_heads;
    int64_t num_slots;
    float factor;
    unsigned int *err;
};

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kMaxThreads, kCtasPerSm)
rope_and_cache_kernel(const RopeParams p) {
    constexpr int kUnits = D / 16;                 // units a head
    __shared__ __align__(16) float cosines[D / 2], sines[D / 2];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t t = blockIdx.x;
    const int H = p.num_heads, Hkv = p.num_kv_heads;
    const int units = (H + 2 * Hkv) * kUnits;
    const int64_t slot = p.slot_mapping[t];
    const bool store_kv = slot >= 0 && slot < p.num_slots;      // a negative slot is padding
    if (slot >= p.num_slots && threadIdx.x == 0) pk::set_error(p.err, PK_DEVERR_SLOT);
    const int threads = blockDim.x;

    for (int base = 0; base < units; base += threads) {
        const int u = base + threadIdx.x;
        const bool active = u < units;
        const int head = u / kUnits, j = u % kUnits;
        const int2 o = pk::unit_offsets<kInterleaved>(j, head < H + Hkv ? p.rot : 0, D);
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (active) {
            const uint16_t *src = head < H        ? p.q + t * p.q_stride + head * D
                                  : head < H + Hkv ? p.k + t * p.k_stride + (head - H) * D
                                                   : p.v + t * p.v_stride + (head - H - Hkv) * D;
            a = pk::ld_stream(src + o.x);
            b = pk::ld_stream(src + o.y);
        }
        if (base == 0) {
            const int64_t pos = p.rot ? p.positions[t] : 0;
            for (int i = threadIdx.x; i < p.rot / 2; i += threads) {
                const float2 cs = pk::rotation(pos, pk::turns_per_position(p.inv_freq[i]), p.factor);
                cosines[i] = cs.x;
                sines[i] = cs.y;
            }
            __syncthreads();
        }
        if (!active) break;
        if (head < H + Hkv) pk::rotate_unit<kInterleaved>(a, b, cosines, sines, j, p.rot, D);
        uint16_t *dst;
        if (head < H) {
            dst = p.q_out + t * p.q_out_stride + head * D;
        } else {
            if (!store_kv) break;                  // every further unit is K or V too
            dst = head < H + Hkv ? p.k_cache + (slot * Hkv + (head - H)) * D
                                 : p.v_cache + (slot * Hkv + (head - H - Hkv)) * D;
        }
        *reinterpret_cast<uint4 *>(dst + o.x) = a;
        *reinterpret_cast<uint4 *>(dst + o.y) = b;
    }
}

template <int D, bool kInterleaved>
cudaError_t launch_rope(const RopeParams &p, int num_tokens, cudaStream_t stream) {
    // As many threads as spread the token's units evenly over the rounds.
    const int units = (p.num_heads + 2 * p.num_kv_heads) * (D / 16);
    const int rounds = (units + kMaxThreads - 1) / kMaxThreads;
    const int threads = ((units + rounds - 1) / rounds + 31) / 32 * 32;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_tokens));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_and_cache_kernel<D, kInterleaved>, p);
}

}  // namespace

extern "C" int pk_rope_and_cache(void *q_out, const void *q, const void *k, const void *v, int64_t q_out_stride,
                                 int64_t q_stride, int64_t k_stride, int64_t v_stride, void *k_cache, void *v_cache,
                                 const int64_t *slot_mapping, const int64_t *positions, const float *inv_freq,
                                 int rot_dim, int interleaved, float factor, int num_tokens, int num_heads,
                                 int num_kv_heads, int head_dim, int num_blocks, int block_size, pk_stream_t stream) {
    const int st = pk::check_rope_args(q_out_stride, q_stride, k_stride, v_stride, rot_dim, factor, num_tokens,
                                       num_heads, num_kv_heads, head_dim, num_blocks, block_size);
    if (st != PK_OK || num_tokens == 0) return st;
    if (!k || !v || !k_cache || !v_cache || !slot_mapping || (num_heads > 0 && (!q || !q_out)) ||
        (rot_dim > 0 && (!positions || !inv_freq)))
        return PK_ERR_NULL;
    if (!pk::aligned16(q_out) || !pk::aligned16(q) || !pk::aligned16(k) || !pk::aligned16(v) ||
        !pk::aligned16(k_cache) || !pk::aligned16(v_cache))
        return PK_ERR_ALIGNMENT;
    RopeParams p{};
    p.q_out = static_cast<uint16_t *>(q_out);
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_out_stride = q_out_stride;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.k_cache = static_cast<uint16_t *>(k_cache);
    p.v_cache = static_cast<uint16_t *>(v_cache);
    p.slot_mapping = slot_mapping;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.rot = rot_dim;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.num_slots = static_cast<int64_t>(num_blocks) * block_size;
    p.factor = factor;
    p.err = pk::error_word_ptr();
    if (!p.err) return PK_ERR_NO_DEVICE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (head_dim == 64)
        e = interleaved ? launch_rope<64, true>(p, num_tokens, s) : launch_rope<64, false>(p, num_tokens, s);
    else
        e = interleaved ? launch_rope<128, true>(p, num_tokens, s) : launch_rope<128, false>(p, num_tokens, s);
    return e == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}
