// Rotary positions and the append to the 8-bit paged cache, in one pass.
//
// A block's tokens share one scale for each KV head, so the unit of work is a
// cell: the part of one sequence's new tokens that falls into one block.  One
// warp owns a cell's K (or V) of one head: it keeps the new rows in registers,
// finds their largest magnitude, takes the scale from it and from the scale
// that the block's older tokens have, re-rounds those older rows if the scale
// grows, and rotates, divides, rounds and writes the new ones.  No two warps
// touch the same (block, head), so nothing is atomic and the result does not
// depend on any order.  The blocks to write come from the block tables and the
// lengths (as for the attention call), not from slots: the owner of a block
// has to know which of its tokens are new.
//
// Bound: HBM bytes for prompts (2 bytes an element read, 2 written for q and 1
// for K and V); for single tokens the chain of dependent loads (length, table
// entry, old scale).  The queries' rows are rotated by CTAs of their own
// (blockIdx.y >= kv_ctas), so that a step's K/V chain and its queries overlap.
// Measured back to back: 9 chunks, 6,689 tokens, of 32 + 16 heads of 128, half of
// a head rotated, in 25.0 us (151 MB, 0.89 of a copy's rate), of 64 + 16 in 44.0
// (0.87); one token of each of 256 sequences 6.8 us.
#include "../../include/pagedkv_fp8.h"
#include "fp8.cuh"
#include "rope.cuh"

#include <algorithm>

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// CTAs an SM and q units (2 x 16 bytes) a thread has in flight.  Blocks of 32
// tokens at head dim 128 keep 64 registers of rows (the 9 chunks above: 27.5 us
// so, 29.9 with the others' choice, which takes 24.9 on blocks of 16 where this
// one takes 24.7; two CTAs and 8 units take 25.9, but 256 decode tokens 9.5
// instead of 8.1).
template <int D, int B>
constexpr int ctas_per_sm() { return D * B >= 4096 ? 3 : 4; }
template <int D, int B>
constexpr int query_batch() { return D * B >= 4096 ? 4 : 3; }
constexpr int kQueryUnits = 2048;  // most q units of a CTA: 8 a thread

struct AppendParams {
    uint16_t *q_out;
    const uint16_t *q, *k, *v;
    int64_t q_out_stride, q_stride, k_stride, v_stride;
    uint8_t *k_cache, *v_cache;
    float *k_scales, *v_scales;
    const int32_t *block_tables, *seq_lens, *cu_q_lens;
    const int64_t *positions;
    const float *inv_freq;
    int rot, num_heads, num_kv_heads, max_blocks_per_seq, num_seqs, total_q, max_q_len, num_blocks;
    int cells_per_seq;       // > 0: cell x belongs to sequence x / cells_per_seq; 0: found by search
    int kv_ctas;             // CTAs (blockIdx.y) of a cell for K and V, kWarps heads each
    int q_heads_per_cta;
    float factor;
    unsigned int *err;
};

// First cell of sequence s when the cells are numbered by search: a sequence
// with n new tokens touches at most (n - 1) / B + 2 blocks, and
// floor((x + n) / B) + 2 - floor(x / B) is at least that.
template <int B>
__device__ __forceinline__ int first_cell(const AppendParams &p, int s) {
    return min(max(p.cu_q_lens[s], 0), p.total_q) / B + 2 * s;
}

// The sequence whose cells include x: the last s with first_cell(s) <= x, by
// two rounds of kThreads probes.  num_seqs <= 65535 = kThreads^2 - 1.
template <int B>
__device__ __forceinline__ int find_sequence(const AppendParams &p, int x) {
    const int step = (p.num_seqs + kThreads - 1) / kThreads;
    const int s0 = static_cast<int>(threadIdx.x) * step;
    const int coarse = __syncthreads_count(s0 < p.num_seqs && first_cell<B>(p, s0) <= x);
    const int lo = max(coarse - 1, 0) * step;
    const int s1 = lo + static_cast<int>(threadIdx.x);
    const int fine = __syncthreads_count(static_cast<int>(threadIdx.x) < step && s1 < p.num_seqs &&
                                         first_cell<B>(p, s1) <= x);
    return lo + max(fine - 1, 0);
}

// bf16 magnitudes in pairs: as integers they are ordered, with infinity and NaN
// above all others.
__device__ __forceinline__ uint32_t max_magnitude(uint32_t most, const uint4 &v) {
    most = __vmaxu2(most, v.x & 0x7fff7fffu);
    most = __vmaxu2(most, v.y & 0x7fff7fffu);
    most = __vmaxu2(most, v.z & 0x7fff7fffu);
    return __vmaxu2(most, v.w & 0x7fff7fffu);
}
constexpr uint32_t kHuge = 0x5e80;       // 2^62 as bf16: below, no square overflows

// The square of a magnitude for the scale: values that are not finite count
// as 0, finite ones whose square overflows as the largest float.
constexpr float kLargest = 3.402823466e38f;
__device__ __forceinline__ float capped(float m2, float x, float y) {
    if (m2 <= kLargest) return m2;
    return fabsf(x) <= kLargest && fabsf(y) <= kLargest ? kLargest : 0.f;
}

// The largest squared length of two pairs (kOdd: some value is huge or not finite).
template <bool kOdd>
__device__ __forceinline__ float longest(float x0, float x1, float y0, float y1) {
    const uint64_t x = pk::f2(x0, x1), y = pk::f2(y0, y1);
    const float2 m2 = pk::unf2(pk::fma2(x, x, pk::mul2(y, y)));      // all squares are exact in fp32
    return kOdd ? fmaxf(capped(m2.x, x0, y0), capped(m2.y, x1, y1)) : fmaxf(m2.x, m2.y);
}

// Of a unit's rotated pairs; 0 if it has none.
template <bool kInterleaved, bool kOdd>
__device__ __forceinline__ float longest_pair(const uint4 &a, const uint4 &b, pk::bool2 turned) {
    float fa[8], fb[8], m = 0.f;
    pk::unpack8(a, fa);
    pk::unpack8(b, fb);
    if constexpr (kInterleaved) {
        if (turned.x) {
#pragma unroll
            for (int i = 0; i < 8; i += 4) m = fmaxf(m, longest<kOdd>(fa[i], fa[i + 2], fa[i + 1], fa[i + 3]));
        }
        if (turned.y) {
#pragma unroll
            for (int i = 0; i < 8; i += 4) m = fmaxf(m, longest<kOdd>(fb[i], fb[i + 2], fb[i + 1], fb[i + 3]));
        }
    } else if (turned.x) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) m = fmaxf(m, longest<kOdd>(fa[i], fa[i + 1], fb[i], fb[i + 1]));
    }
    return m;
}

// The largest square of a vector where some value is huge or not finite.
__device__ __forceinline__ float largest_odd(const uint4 &v) {
    float f[8], m = 0.f;
    pk::unpack8(v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, capped(f[i] * f[i], f[i], 0.f));
    return m;
}

// Eight values to eight e4m3 bytes; where `odd`, what is not finite becomes NaN.
__device__ __forceinline__ uint2 quantise8(float (&f)[8], float inv, bool odd) {
    if (odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = fabsf(f[i]) <= kLargest ? f[i] : __int_as_float(0x7fffffff);
    }
    return make_uint2(pk::e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                      pk::e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}

template <int D, int B, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, (ctas_per_sm<D, B>()))
rope_and_cache_fp8_kernel(const AppendParams p) {
    constexpr int kBatch = query_batch<D, B>();
    constexpr int kUnits = D / 16;                 // units (two 8-element vectors) a row
    constexpr int kRows = 32 / kUnits;             // rows a warp handles at once
    constexpr int kIters = (B + kRows - 1) / kRows;
    __shared__ __align__(16) float cosines[B][D / 2], sines[B][D / 2];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- the cell ----------------------------------------------------------
    int s, j;
    if (p.cells_per_seq > 0) {
        s = blockIdx.x / p.cells_per_seq;
        j = blockIdx.x % p.cells_per_seq;
    } else {
        // The search may pass over a sequence whose rows run backwards: it is reported here.
        if (blockIdx.y == 0 && threadIdx.x == 0 && static_cast<int>(blockIdx.x) < p.num_seqs &&
            p.cu_q_lens[blockIdx.x + 1] < p.cu_q_lens[blockIdx.x])
            pk::set_error(p.err, PK_DEVERR_SEQ_LEN);
        s = find_sequence<B>(p, blockIdx.x);
        j = static_cast<int>(blockIdx.x) - first_cell<B>(p, s);
    }
    const int r0 = p.cu_q_lens ? p.cu_q_lens[s] : s;
    const int r1 = p.cu_q_lens ? p.cu_q_lens[s + 1] : s + 1;
    const int L = p.seq_lens[s];
    const int n = r1 - r0;
    if (r0 < 0 || n < 0 || r1 > p.total_q || L < 0 || L > static_cast<int64_t>(p.max_blocks_per_seq) * B || n > L ||
        n > p.max_q_len) {
        if (j == 0 && blockIdx.y == 0 && threadIdx.x == 0) pk::set_error(p.err, PK_DEVERR_SEQ_LEN);
        return;
    }
    const int start = L - n;                       // position of the first new token
    const int blk = start / B + j;
    if (n == 0 || j < 0 || static_cast<int64_t>(blk) * B >= L) return;
    const int tok0 = max(start, blk * B);
    const int tok1 = static_cast<int>(min(static_cast<int64_t>(L), (static_cast<int64_t>(blk) + 1) * B));
    const int nt = tok1 - tok0;                    // the cell's new tokens, 1 .. B
    const int64_t row0 = r0 + tok0 - start;        // their first row of q, k, v
    const int off0 = tok0 - blk * B;               // rows below are older tokens

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = p.num_heads, Hkv = p.num_kv_heads;
    const int half = p.rot / 2;

    // ---- (cos, sin) of the cell's tokens ------------------------------------
    auto angles = [&]() {
        if (half > 0) {
            const int per = kThreads / half;       // tokens at once (half <= 64)
            const int pair = threadIdx.x % half, t0 = threadIdx.x / half;
            if (t0 < per) {
                const uint64_t turns = pk::turns_per_position(p.inv_freq[pair]);
                for (int t = t0; t < nt; t += per) {
                    const int64_t pos = p.positions ? p.positions[row0 + t] : static_cast<int64_t>(tok0 + t);
                    const float2 cs = pk::rotation(pos, turns, p.factor);
                    cosines[t][pair] = cs.x;
                    sines[t][pair] = cs.y;
                }
            }
        }
        __syncthreads();
    };

    if (blockIdx.y >= p.kv_ctas) {
        // ---- queries: heads h0 .. h0 + nh - 1 of the cell's tokens ---------
        const int h0 = (blockIdx.y - p.kv_ctas) * p.q_heads_per_cta;
        const int nh = min(p.q_heads_per_cta, H - h0);
        const int per_token = nh * kUnits, units = nt * per_token;
        // u / per_token as a product: exact, since both are at most kQueryUnits.
        const uint32_t inv_per_token = 0xffffffffu / static_cast<uint32_t>(per_token) + 1u;
        for (int base = 0; base < units; base += kThreads * kBatch) {
            uint4 a[kBatch], b[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int u = base + i * kThreads + static_cast<int>(threadIdx.x);
                if (u >= units) break;
                const int t = static_cast<int>(__umulhi(u, inv_per_token)), w = u - t * per_token;
                const uint16_t *src = p.q + (row0 + t) * p.q_stride + (h0 + w / kUnits) * D;
                const int2 o = pk::unit_offsets<kInterleaved>(w % kUnits, p.rot, D);
                a[i] = pk::ld_stream(src + o.x);
                b[i] = pk::ld_stream(src + o.y);
            }
            if (base == 0) angles();
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int u = base + i * kThreads + static_cast<int>(threadIdx.x);
                if (u >= units) break;
                const int t = static_cast<int>(__umulhi(u, inv_per_token)), w = u - t * per_token;
                const int ju = w % kUnits;
                const int2 o = pk::unit_offsets<kInterleaved>(ju, p.rot, D);
                pk::rotate_unit<kInterleaved>(a[i], b[i], cosines[t], sines[t], ju, p.rot, D);
                uint16_t *dst = p.q_out + (row0 + t) * p.q_out_stride + (h0 + w / kUnits) * D;
                *reinterpret_cast<uint4 *>(dst + o.x) = a[i];
                *reinterpret_cast<uint4 *>(dst + o.y) = b[i];
            }
        }
        return;
    }

    // ---- K and V: one warp a (K or V, head) ---------------------------------
    const int phys = p.block_tables[static_cast<int64_t>(s) * p.max_blocks_per_seq + blk];
    if (phys < 0 || phys >= p.num_blocks) {
        if (threadIdx.x == 0 && blockIdx.y == 0) pk::set_error(p.err, PK_DEVERR_BLOCK_ID);
        return;
    }
    const int ju = lane % kUnits, lrow = lane / kUnits;
    const float f2 = p.factor * p.factor;
    // Task: K of head `task`, or V of head task - Hkv.
    const int task = blockIdx.y * kWarps + warp;
    const bool active = task < 2 * Hkv;
    const bool is_k = task < Hkv;
    const int h = is_k ? task : task - Hkv;
    const int rot = is_k ? p.rot : 0;
    const int2 o = pk::unit_offsets<kInterleaved>(ju, rot, D);
    const uint16_t *src = is_k ? p.k : p.v;
    const int64_t stride = is_k ? p.k_stride : p.v_stride;
    float *scale_at = (is_k ? p.k_scales : p.v_scales) + static_cast<int64_t>(phys) * Hkv + h;
    uint8_t *rows = (is_k ? p.k_cache : p.v_cache) + (static_cast<int64_t>(phys) * Hkv + h) * (B * D);
    uint4 a[kIters], b[kIters];
    float had = 0.f, most = 0.f;
    if (active) {
        if (off0 > 0) had = *scale_at;
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
            const int t = it * kRows + lrow;
            a[it] = b[it] = make_uint4(0, 0, 0, 0);
            if (t < nt) {
                a[it] = pk::ld_stream(src + (row0 + t) * stride + h * D + o.x);
                b[it] = pk::ld_stream(src + (row0 + t) * stride + h * D + o.y);
            }
        }
    }
    if (static_cast<int>(blockIdx.y) * kWarps < Hkv) angles();      // some warp has keys
    if (!active) return;
    // The largest magnitudes decide how the squares are taken: of vectors that
    // are not rotated they are all there is to know.
    const pk::bool2 turned = pk::unit_turned<kInterleaved>(ju, rot, D);
    uint32_t mag_a = 0, mag_b = 0;
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
        mag_a = max_magnitude(mag_a, a[it]);
        mag_b = max_magnitude(mag_b, b[it]);
    }
    mag_a = max(mag_a & 0xffffu, mag_a >> 16);
    mag_b = max(mag_b & 0xffffu, mag_b >> 16);
    const bool odd = __any_sync(0xffffffffu, max(mag_a, mag_b) >= kHuge);
    float plain = 0.f;                             // of elements that are not rotated
    if (odd) {
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
            if (it * kRows >= nt) break;
            most = fmaxf(most, longest_pair<kInterleaved, true>(a[it], b[it], turned));
            if (!turned.x) plain = fmaxf(plain, largest_odd(a[it]));
            if (!turned.y) plain = fmaxf(plain, largest_odd(b[it]));
        }
        if (most >= kLargest) plain = kLargest;    // overflowed: no factor brings that back
    } else {
        if (turned.x) {
#pragma unroll
            for (int it = 0; it < kIters; ++it) {
                if (it * kRows >= nt) break;
                most = fmaxf(most, longest_pair<kInterleaved, false>(a[it], b[it], turned));
            }
        }
        const float x = turned.x ? 0.f : pk::bf16_lo(mag_a), y = turned.y ? 0.f : pk::bf16_lo(mag_b);
        plain = fmaxf(x * x, y * y);
    }
    most = fmaxf(fminf(most * f2, kLargest), plain);
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
    float scale = pk::needed_scale(most);
    if (off0 > 0) {
        if (!pk::scale_ok(had)) {
            // Nothing says what the older rows stood for.  They become NaN: under the
            // new scale they would pass for values that nobody wrote.
            if (lane == 0) pk::set_error(p.err, PK_DEVERR_SCALE);
            const uint32_t nan = 0x7f7f7f7fu;
            for (int r = lrow; r < off0; r += kRows)
                *reinterpret_cast<uint4 *>(rows + r * D + ju * 16) = make_uint4(nan, nan, nan, nan);
        } else if (had >= scale) {
            scale = had;
        } else {
            // The scale grows: the older rows in the new one's steps.
            const float ratio = had / scale;       // exact: `scale` is a power of two
            for (int r = lrow; r < off0; r += kRows) {
                uint4 *at = reinterpret_cast<uint4 *>(rows + r * D + ju * 16);
                uint4 w = *at;
                uint32_t *e = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float f[4];
                    pk::e4m3x4_to_float(e[i], f);
                    e[i] = pk::e4m3x4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
                }
                *at = w;
            }
        }
    }
    __syncwarp();                                  // every lane has its copy of the old scale
    if (lane == 0) *scale_at = scale;
    const float inv = 1.f / scale;
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
        const int t = it * kRows + lrow;
        if (t >= nt) break;
        float fa[8], fb[8];
        pk::unpack8(a[it], fa);
        pk::unpack8(b[it], fb);
        pk::rotate_unit<kInterleaved>(fa, fb, cosines[t], sines[t], ju, rot, D);
        uint8_t *dst = rows + (off0 + t) * D;
        *reinterpret_cast<uint2 *>(dst + o.x) = quantise8(fa, inv, odd);
        *reinterpret_cast<uint2 *>(dst + o.y) = quantise8(fb, inv, odd);
    }
}

template <int D, int B, bool kInterleaved>
cudaError_t launch_append(AppendParams &p, cudaStream_t stream) {
    const int per_seq = (std::max(p.max_q_len, 1) - 1) / B + 2;
    // Cells: at most per_seq of every sequence, or at most total / B + 2 of
    // each by search (a batch of very unequal lengths).  The search costs two
    // block-wide counts, so it is used only where it saves CTAs.
    const int64_t direct = p.cu_q_lens ? static_cast<int64_t>(p.num_seqs) * per_seq : p.num_seqs;
    const int64_t searched = p.total_q / B + 2 * static_cast<int64_t>(p.num_seqs);
    p.cells_per_seq = 0;
    int64_t cells = searched;
    if (direct <= 2 * searched) {
        p.cells_per_seq = p.cu_q_lens ? per_seq : 1;
        cells = direct;
    }
    const int tokens = std::min(B, std::max(p.cu_q_lens ? p.max_q_len : 1, 1));   // of a cell, at most
    p.q_heads_per_cta = std::max(1, std::min(std::max(p.num_heads, 1), kQueryUnits / (tokens * (D / 16))));
    p.kv_ctas = (2 * p.num_kv_heads + kWarps - 1) / kWarps;
    const int q_ctas = (p.num_heads + p.q_heads_per_cta - 1) / p.q_heads_per_cta;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cells), static_cast<unsigned>(p.kv_ctas + q_ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_and_cache_fp8_kernel<D, B, kInterleaved>, static_cast<const AppendParams &>(p));
}

template <int D, int B>
cudaError_t launch_append_layout(AppendParams &p, bool interleaved, cudaStream_t stream) {
    return interleaved ? launch_append<D, B, true>(p, stream) : launch_append<D, B, false>(p, stream);
}

template <int D>
cudaError_t launch_append_block(AppendParams &p, int block_size, bool interleaved, cudaStream_t stream) {
    switch (block_size) {
        case 8: return launch_append_layout<D, 8>(p, interleaved, stream);
        case 16: return launch_append_layout<D, 16>(p, interleaved, stream);
        default: return launch_append_layout<D, 32>(p, interleaved, stream);
    }
}

}  // namespace

extern "C" int pk_rope_and_cache_fp8(void *q_out, const void *q, const void *k, const void *v, int64_t q_out_stride,
                                     int64_t q_stride, int64_t k_stride, int64_t v_stride, void *k_cache,
                                     void *v_cache, float *k_scales, float *v_scales, const int32_t *block_tables,
                                     int max_blocks_per_seq, const int32_t *seq_lens, const int32_t *cu_q_lens,
                                     int max_q_len, int num_seqs, const int64_t *positions, const float *inv_freq,
                                     int rot_dim, int interleaved, float factor, int num_tokens, int num_heads,
                                     int num_kv_heads, int head_dim, int num_blocks, int block_size,
                                     pk_stream_t stream) {
    const int st = pk::check_rope_args(q_out_stride, q_stride, k_stride, v_stride, rot_dim, factor, num_tokens,
                                       num_heads, num_kv_heads, head_dim, num_blocks, block_size);
    if (st != PK_OK) return st;
    if (num_seqs < 0 || num_seqs > 65535 || max_blocks_per_seq < 0 || max_q_len < 0) return PK_ERR_SHAPE;
    if (!cu_q_lens && num_tokens != num_seqs) return PK_ERR_SHAPE;     // one new token a sequence
    if (num_tokens == 0 || num_seqs == 0) return PK_OK;
    if (!k || !v || !k_cache || !v_cache || !k_scales || !v_scales || !block_tables || !seq_lens ||
        (num_heads > 0 && (!q || !q_out)) || (rot_dim > 0 && !inv_freq))
        return PK_ERR_NULL;
    if (!pk::aligned16(q_out) || !pk::aligned16(q) || !pk::aligned16(k) || !pk::aligned16(v) ||
        !pk::aligned16(k_cache) || !pk::aligned16(v_cache))
        return PK_ERR_ALIGNMENT;
    AppendParams p{};
    p.q_out = static_cast<uint16_t *>(q_out);
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_out_stride = q_out_stride;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.cu_q_lens = cu_q_lens;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.rot = rot_dim;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.total_q = num_tokens;
    p.max_q_len = cu_q_lens ? max_q_len : 1;
    p.num_blocks = num_blocks;
    p.factor = factor;
    p.err = pk::error_word_ptr();
    if (!p.err) return PK_ERR_NO_DEVICE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = head_dim == 64 ? launch_append_block<64>(p, block_size, interleaved != 0, s)
                                         : launch_append_block<128>(p, block_size, interleaved != 0, s);
    return e == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}
