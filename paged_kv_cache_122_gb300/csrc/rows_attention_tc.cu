// Attention of many query rows per sequence over its paged keys, split along
// the keys: a tree of drafted tokens (a bit mask among the drafts, the context
// in full) and cross attention (every key).
//
// Mathematics.  For a query row, scores s_j = c q.k_j (c holds log2 e) over the
// visible keys; weights 2^(s_j - m) against a reference m that starts above the row's
// first scores and moves only when a score exceeds it; O = sum of weights times v_j, l = sum of
// weights, result O / l.  Parts over disjoint keys join by M = max m, factors
// 2^(m - M): between the two groups of a CTA and between CTAs.
//
// Shapes.  A query tile is 128 rows -- 128 / G tokens x the G heads of one KV
// head -- on the M of both products, as in the prefill kernel:
//   S[128 x 64] = Q K_half^T,  O[128 x D] += P V_half   (tcgen05, fp32 in TMEM).
// A segment is one (sequence, KV head, block of query tiles) over all of the
// sequence's 128-key tiles.  A block is two query tiles that share every K and V
// tile, or one.  Two softmax groups of 128 threads: with two query tiles, each has
// its own; with one, each takes one half of every key tile, with an O and m of its
// own, and they join at the end of the part through tensor memory, where both see
// the same lanes.
//
// Jobs.  A group's job is 64 keys of a tile: S, weights, P.V.  Its S has two
// buffers, which the jobs take in turn, so that while the weights of one job are
// worked out the tensor core does P.V of the job before and S of the next: with one
// buffer of 128 keys a group's chain of S, weights and product took 2.4 us a tile
// however few instructions each had.  (The price: an S of 64 columns reads Q from
// shared memory twice as often.)
//
// Work.  The flattened (segment, key tile) space is cut into one range of equal
// cost for each persistent CTA, so few long sequences fill the GPU as many short
// ones do; a segment that is cut leaves (m, l, O) in a workspace slot, and a merge
// kernel joins its parts.
//
// Per CTA (384 threads): warps 0-3 and 4-7 the softmax groups (thread <-> query
// row = TMEM lane), warp 8 copies Q and K, 9 V, 10 and 11 issue the groups' MMAs.
#include "rows_attention.cuh"
#include "block_scan.cuh"
#include "sm100.cuh"
#include "tmem_wide.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

namespace pk {
namespace {

using namespace sm100;

constexpr int kRows = 128;                      // query rows per tile = MMA M
constexpr int kKeys = 128;                      // keys per tile
constexpr int kHalf = 64;                       // keys of a job = MMA N of S
constexpr int kThreads = 384;
constexpr uint32_t kChunk = 128 * 128;          // 128 rows x 128 bytes (64 bf16)
constexpr uint32_t kTmemCols = 512;             // S_0, S_1, O_0, O_1 (128 columns each)
constexpr uint32_t kTmemS = 0;                  // + x * 128 + buffer * 64; P over its first 32 columns
constexpr uint32_t kTmemO = 256;                // + x * 128
constexpr uint64_t kWaitLimitNs = 1000000000ull;
// A reference max is whole and this far above the scores that set it; it moves up when a
// score exceeds it, so that scores have to climb by 24 before a pass is made again.
// Weights of any size are exact to the same number of bits, and none is above 1: O stays
// within the number of keys times the largest value, as against the exact maximum.
constexpr float kHeadroomLog2 = 24.0f;
// A part starts from its row's reference of the part before, if no score of its first
// job is above it and the largest is not this far below: as far below the scores that set
// it as the headroom is above them.
constexpr float kGuessLog2 = -2.0f * kHeadroomLog2;

// What a part costs, in sixteenths of a key tile under one query tile: a segment's
// set-up and read-out, and a key tile under two query tiles.  From a least-squares fit
// of the CTAs' times to the tiles and segments of their ranges (eight batches): head dim
// 128, a tile 1.2-1.3 us, or 2.1 under two, a segment 2.3-3.9 us; head dim 64, 0.85-0.95,
// 1.6 and 2.6-2.8 us.  (With a segment as one tile, the last CTA of 152 ended 15-30 %
// after the mean on batches of short sequences.)
constexpr int64_t kTileCost1 = 16, kTileCost2 = 27;
template <int D>
constexpr int64_t kSegCost = D == 128 ? 38 : 40;
// A CTA is not given less than this: a cut costs a merge.  (The plan does not know what:
// one block of the merge joins all parts of a segment, one after the other.)
constexpr int64_t kMinCost = 32;

// Rings of 128-key tiles: what 224 KB hold.  TWO: segments may have two query
// tiles, both resident; otherwise one, or two of at most 64 rows.
template <int D, bool TWO>
struct Cfg {
    static constexpr uint32_t kTile = kChunk * (D / 64);     // Q, K or V of 128 rows
    static constexpr uint32_t kQRegion = (TWO ? 2 : 1) * kTile;
    static constexpr int kKS = D == 128 ? 3 : 6;
    static constexpr int kVS = D == 128 ? (TWO ? 2 : 3) : 6;
    static constexpr uint32_t kKOff = kQRegion;
    static constexpr uint32_t kVOff = kKOff + kKS * kTile;
    static constexpr uint32_t kEnd = kVOff + kVS * kTile;
    // Tile masks in flight: the K producer runs at most kKS + 1 tiles ahead of a
    // softmax group (a slot is free when both groups' S is done; the job two on waits
    // for its P).
    static constexpr int kMasks = D == 128 ? 8 : 16;
    static_assert(kMasks > kKS + 2, "masks in flight");
};

// A tile in the MMA warps' eyes: its block has two query tiles; the first and the last
// tile of its part; rows of the 16-key groups that hold no key; its keys.
constexpr uint32_t kMetaTwo = 1, kMetaFirst = 2, kMetaLast = 4, kMetaStale = 8;
constexpr int kMetaKeysShift = 8;

struct Pos {          // a place in the flattened (segment, key tile) space
    int64_t tile;     // index of the key tile
    int32_t s, h, j, t;
};

template <int KS, int VS, int MASKS>
struct Misc {
    uint64_t kfull[KS], kempty[KS], vfull[VS], vempty[VS];
    uint64_t qfull[2], qempty[2];
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];   // [group][buffer]
    uint64_t ml_ready[2], o_taken[2];   // the join of the groups' parts, by the group that arrives
    uint64_t drain[2];
    Pos pos[2];                   // start of this range and of the next one
    int32_t first_cta;            // the CTA in whose range this range's first segment starts
    uint32_t tmem_base;
    int abort;
    int never;
    uint32_t mask[MASKS][4];      // valid keys of a tile
    uint32_t meta[MASKS];         // of a tile, for the MMA warps: kMeta* bits
    union {
        struct {
            int64_t tiles[kThreads / 32 + 1], costs[kThreads / 32 + 1];
        } scan;                   // while planning
        struct {
            float m[kRows], l[kRows];
        } part;                   // what the groups tell each other of a part, one after the other
    };
};

// Slot of a cut part: slot 0 of a CTA for its first segment, slot 1 for its last.
struct SlotHead {
    int32_t flag;          // slot 0: the merge joins this segment at this CTA
    int32_t h, tok0;       // KV head, first token of the block's first tile
    int32_t ntiles;        // query tiles
    int32_t q0, qn;        // the sequence's query rows (the merge saves a trip to memory)
    int32_t first_cta;     // slot 0: the CTA in whose range the segment starts
    int32_t pad0;
    int64_t start_tile;    // slot 0: flattened index of the segment's key tile 0
    int64_t range_beg;     // slot 0: first tile of this CTA's range
    int64_t total_tiles;   // slot 0
    int64_t pad1;
};
static_assert(sizeof(SlotHead) == 64, "slot header");

template <int D>
constexpr size_t slot_bytes(int ntiles) {
    return sizeof(SlotHead) + static_cast<size_t>(ntiles) * (2 * kRows + D * kRows) * sizeof(float);
}
__device__ __forceinline__ char *slot_at(const RowsParams &p, size_t bytes, int cta, int which) {
    return static_cast<char *>(p.slots) + (2 * static_cast<size_t>(cta) + which) * bytes;
}
// m, l and O^T of query tile x of a slot.
__device__ __forceinline__ float *slot_m(char *slot, int x, int D) {
    return reinterpret_cast<float *>(slot + sizeof(SlotHead)) + static_cast<size_t>(x) * (2 + D) * kRows;
}

struct Seq {
    int L, q0, qn;      // keys; first query row; query rows (0 for a sequence to leave out)
    int nt, n2, n1;     // key tiles; blocks of two query tiles; blocks of one (0 or 1)
    bool bad;
};

// A load that bypasses L1: what is read before the programmatic wait and again after it
// cannot come back stale from there.
__device__ __forceinline__ int load_cg(const int32_t *p) {
    int v;
    asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// A sequence's length and first rows (its own and the next one's).
struct Raw {
    int L, q0, q1;
};
__device__ __forceinline__ Raw load_raw(const RowsParams &p, int s) {
    return {load_cg(p.seq_lens + s), load_cg(p.cu_q_lens + s), load_cg(p.cu_q_lens + s + 1)};
}

template <bool TWO>
__device__ __forceinline__ Seq seq_of(const RowsParams &p, const Raw &w, int lgG) {
    Seq r;
    r.L = w.L;
    r.q0 = w.q0;
    const int64_t cap = min(static_cast<int64_t>(p.max_seq_len),
                            static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size);
    r.bad = r.L < 0 || r.L > cap || r.q0 < 0 || w.q1 < r.q0 || w.q1 > p.total_q || w.q1 - r.q0 > p.max_q_len ||
            (p.tree_mask && w.q1 - r.q0 > r.L);
    r.qn = r.bad ? 0 : w.q1 - r.q0;
    r.nt = r.qn > 0 ? (r.L >> 7) + ((r.L & 127) != 0) : 0;
    const int lgqt = 7 - lgG;
    const int tiles = r.nt > 0 ? (r.qn + (1 << lgqt) - 1) >> lgqt : 0;
    r.n2 = TWO ? tiles >> 1 : 0;
    r.n1 = tiles - 2 * r.n2;
    return r;
}
template <bool TWO>
__device__ __forceinline__ Seq load_seq(const RowsParams &p, int s, int lgG) {
    return seq_of<TWO>(p, load_raw(p, s), lgG);
}

// A quotient of two numbers >= 0 and > 0, out of line (one copy of the code), by 32 bits
// where they fit: the plan divides a dozen times, and 64-bit divisions were half of its
// 3.6 us.
__device__ __noinline__ int64_t quotient(int64_t a, int64_t b) {
    if ((static_cast<uint64_t>(a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

template <int D>
__device__ __forceinline__ int64_t block_cost(const Seq &q, bool two) {
    return kSegCost<D> + (two ? kTileCost2 : kTileCost1) * q.nt;
}
template <int D>
__device__ __forceinline__ int64_t head_cost(const Seq &q) {
    return q.n2 * block_cost<D>(q, true) + q.n1 * block_cost<D>(q, false);
}

// One CTA's part of a segment, and the walk from part to part.
struct Part {
    int s, h, j;
    int t0, t1;          // key tiles
    int tok0;            // first query token of the block, in its sequence
    bool two;
};
template <bool TWO>
struct Walk {
    const RowsParams &p;
    int lgG;
    int64_t left;        // key tiles left in the range
    int s, h, j, t;
    Seq q;
    __device__ __forceinline__ Walk(const RowsParams &pp, int lg, const Pos &from, int64_t n)
        : p(pp), lgG(lg), left(n), s(from.s), h(from.h), j(from.j), t(from.t) {
        if (left > 0) q = load_seq<TWO>(p, s, lgG);
    }
    __device__ __forceinline__ bool next(Part &a) {
        if (left <= 0) return false;
        const int n = static_cast<int>(min(left, static_cast<int64_t>(q.nt - t)));
        a.s = s;
        a.h = h;
        a.j = j;
        a.t0 = t;
        a.t1 = t + n;
        a.two = TWO && j < q.n2;
        a.tok0 = j * (2 * (kRows >> lgG));
        left -= n;
        return true;
    }
    // To the part after the one that next() gave (its fields of q stay until here).
    __device__ __forceinline__ void advance() {
        if (left <= 0) return;
        t = 0;
        if (++j < q.n2 + q.n1) return;
        j = 0;
        if (++h < p.num_kv_heads) return;
        h = 0;
#pragma unroll 1
        do {
            ++s;                                  // (tiles are left, so there is such a sequence)
            q = load_seq<TWO>(p, s, lgG);
        } while (q.nt == 0);
    }
};

// Cuts the flattened space: CTA c of C takes the tiles whose cost starts in
// [c W / C, (c + 1) W / C), W the total cost, C no more than gives every CTA
// kMinCost.  A segment's tile 0 starts at its start, tile t at start + the segment's cost +
// t tiles.  The sequences (length, first row, next one's first row, kThreads apart) come
// from `copy` if there is one.  Every thread calls it; returns the total tile count, and in *odd whether
// a sequence is to be reported or to get zeros.
template <int D, bool TWO, typename M>
__device__ __forceinline__ int64_t plan(const RowsParams &p, M *misc, const int32_t *copy, int lgG, int c, int C,
                                        int *odd) {
    const int N = p.num_seqs, Hkv = p.num_kv_heads;
    auto seq = [&](int s) -> Seq {
        return seq_of<TWO>(p, copy ? Raw{copy[s], copy[kThreads + s], copy[2 * kThreads + s]} : load_raw(p, s), lgG);
    };
    const int per = (N + kThreads - 1) / kThreads;
    const int s_lo = min(N, static_cast<int>(threadIdx.x) * per), s_hi = min(N, s_lo + per);
    int64_t mine = 0, mine_w = 0;
    int strange = 0;
#pragma unroll 1
    for (int s = s_lo; s < s_hi; ++s) {
        const Seq q = seq(s);
        strange |= q.bad || (q.qn > 0 && q.L == 0);
        mine += static_cast<int64_t>(q.nt) * (q.n2 + q.n1) * Hkv;
        mine_w += head_cost<D>(q) * Hkv;
    }
    int64_t T, W;
    const int64_t off = block_exclusive_scan<kThreads>(mine, misc->scan.tiles, &T);
    const int64_t off_w = block_exclusive_scan<kThreads>(mine_w, misc->scan.costs, &W);
    const int64_t Ce = max(static_cast<int64_t>(1), min(static_cast<int64_t>(C), W / kMinCost));   // (kMinCost: 2^5)
    auto bound = [&](int64_t k) -> int64_t { return k >= Ce ? W : quotient(k * W, Ce); };
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        const int64_t P = bound(c + k);
        if (P >= W) {
            if (threadIdx.x == 0) misc->pos[k].tile = T;
            continue;
        }
        if (P < off_w || P >= off_w + mine_w) continue;
        int64_t at = off, at_w = off_w;
#pragma unroll 1
        for (int s = s_lo; s < s_hi; ++s) {
            const Seq q = seq(s);
            const int64_t hc = head_cost<D>(q);
            if (P >= at_w + hc * Hkv) {
                at += static_cast<int64_t>(q.nt) * (q.n2 + q.n1) * Hkv;
                at_w += hc * Hkv;
                continue;
            }
            int64_t r = P - at_w;
            int64_t h = quotient(r, hc);
            r -= h * hc;
            const int64_t b2 = block_cost<D>(q, true);
            int64_t j = min(quotient(r, b2), static_cast<int64_t>(q.n2));
            r -= j * b2;
            const int64_t tc = j < q.n2 ? kTileCost2 : kTileCost1;
            // The first tile that starts at or after r.
            int64_t t = r == 0 ? 0 : r <= kSegCost<D> ? 1 : quotient(r - kSegCost<D> + tc - 1, tc);
            int64_t a = P - r;                        // where the segment starts
            if (t >= q.nt) {                          // behind its last one: the next segment
                a += block_cost<D>(q, j < q.n2);
                t = 0;
                if (++j == q.n2 + q.n1) {
                    j = 0;
                    ++h;
                }
            }
            Pos &o = misc->pos[k];
            o.tile = at + (h * (q.n2 + q.n1) + j) * q.nt + t;
            if (h == Hkv) {                           // the first segment of a later sequence
                h = 0;
                int s2 = s;
#pragma unroll 1
                while (++s2 < N && seq(s2).nt == 0) {}
                o.s = s2;
            } else {
                o.s = s;
            }
            o.h = static_cast<int>(h);
            o.j = static_cast<int>(j);
            o.t = static_cast<int>(t);
            if (k == 0) {
                int64_t f = min(quotient(a * Ce, W), Ce - 1);
                while (f + 1 < Ce && bound(f + 1) <= a) ++f;
                while (f > 0 && bound(f) > a) --f;
                misc->first_cta = static_cast<int>(f);
            }
            break;
        }
    }
    *odd = __syncthreads_or(strange);
    return T;
}

__device__ __forceinline__ float ex2(float x) { return fast_exp2(x); }

// A warp's wait for a phase, one decision for all lanes; false on give-up.  What does
// not come at once is waited for out of line: the warps' different loops share one
// instruction cache, and a wait's code in every place is as long as the work.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int *abort, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, limit_ns));
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, int phase, volatile int *abort, uint64_t limit_ns) {
    const uint32_t b = smem_u32(bar);
    return __all_sync(0xffffffffu, mbar_try_wait(b, phase & 1)) || wait_on(b, phase & 1, abort, limit_ns);
}
// One lane of the warp, by the instruction whose predicate the compiler knows to be
// one lane's: the operands of what it issues stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}" : "=r"(p));
    return p != 0;
}

// Three-input max (NaN inputs are skipped, as by fmaxf).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// 32 bytes at once (a whole sector), where the output's alignment allows it.
__device__ __forceinline__ void store32(void *dst, const uint32_t (&w)[8], bool aligned) {
    if (aligned) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                     ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// N results of a row, to element idx of the output (idx and N multiples of 16).
template <int N>
__device__ __forceinline__ void store_row(const RowsParams &p, size_t idx, const float (&f)[N]) {
    const bool aligned = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
    if (p.out_fp32) {
        float *o = static_cast<float *>(p.out) + idx;
#pragma unroll
        for (int k = 0; k < N; k += 8) {
            uint32_t w[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) w[n] = __float_as_uint(f[k + n]);
            store32(o + k, w, aligned);
        }
    } else {
        uint16_t *o = static_cast<uint16_t *>(p.out) + idx;
#pragma unroll
        for (int k = 0; k < N; k += 16) {
            uint32_t w[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) w[n] = pack_bf16x2(f[k + 2 * n], f[k + 2 * n + 1]);
            store32(o + k, w, aligned);
        }
    }
}

// q_box: query tokens of a query copy (q_box * G rows, at most 128); q_slots: how
// many query buffers the region holds (1 or 2; always 2 with TWO).
template <int D, bool TWO>
__global__ void __launch_bounds__(kThreads, 1)
rows_attention_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ RowsParams p, int q_box,
                      int q_slots) {
    static_assert(D == 64 || D == 128, "head_dim");
    using C_ = Cfg<D, TWO>;
    using M_ = Misc<C_::kKS, C_::kVS, C_::kMasks>;
    constexpr int NCH = D / 64;
    constexpr int KS = C_::kKS, VS = C_::kVS;
    constexpr uint32_t kTile = C_::kTile;
    static_assert(1024 + C_::kEnd + sizeof(M_) <= 232448, "shared memory per CTA");
    // K and V of a key tile: each page in one TMA box as B / 8 blocks of 8 rows,
    // each block [half][8 rows][64], so the 8-row swizzle atoms of a half lie
    // kAtomStride apart whatever the block size.
    constexpr uint32_t kAtomStride = 1024u * NCH;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int Hkv = p.num_kv_heads, H = p.num_heads, B = p.block_size;
    const int G = H / Hkv, lgG = __ffs(G) - 1;
    const int QT = kRows >> lgG;                    // query tokens per tile
    const int c = blockIdx.x, C = gridDim.x;
    const uint64_t lim = p.wait_limit_ns ? p.wait_limit_ns : kWaitLimitNs;
    const size_t slot_sz = slot_bytes<D>(TWO ? 2 : 1);

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    M_ *misc = reinterpret_cast<M_ *>(smem + C_::kEnd);
    const uint32_t base = smem_u32(smem);

    if (threadIdx.x == 0) {
        for (int i = 0; i < KS; ++i) {
            mbar_init(smem_u32(&misc->kfull[i]), 1);
            mbar_init(smem_u32(&misc->kempty[i]), 2);
        }
        for (int i = 0; i < VS; ++i) {
            mbar_init(smem_u32(&misc->vfull[i]), 1);
            mbar_init(smem_u32(&misc->vempty[i]), 2);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&misc->qfull[x]), 1);
            mbar_init(smem_u32(&misc->qempty[x]), TWO ? 1 : 2);
            for (int u = 0; u < 2; ++u) {
                mbar_init(smem_u32(&misc->s_full[x][u]), 1);
                mbar_init(smem_u32(&misc->p_full[x][u]), 4);
                mbar_init(smem_u32(&misc->pv_done[x][u]), 1);
            }
            mbar_init(smem_u32(&misc->drain[x]), 1);
            mbar_init(smem_u32(&misc->ml_ready[x]), 4);
            mbar_init(smem_u32(&misc->o_taken[x]), 4);
        }
        misc->abort = 0;
        misc->never = 0;
        fence_mbar_init();
    }
    if (warp == 10) {
        tmem_alloc(smem_u32(&misc->tmem_base), kTmemCols);
        tmem_relinquish();
    }
    if (warp == 8 && lane == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        prefetch_tmap(&tm_q);
    }
    // A programmatic dependent of the previous kernel in the stream: what comes before the
    // wait overlaps that kernel's tail.  With a sequence a thread at most, the range is
    // planned before it, from a copy of the lengths in what will be the rings; afterwards
    // they are read again, and the plan is made again if one differs from the copy.  (From
    // the copy, not from memory: what is written there meanwhile, and written back, would
    // not show afterwards.)  Nothing else global is read before the wait, and nothing
    // written.
    auto wait_prev = [&]() {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    };
    bool ahead = p.num_seqs <= kThreads;
    int32_t *copy = ahead ? reinterpret_cast<int32_t *>(smem + C_::kKOff) : nullptr;
    static_assert(3 * kThreads * sizeof(int32_t) <= C_::kTile, "room for the copy");
    const bool owner = ahead && static_cast<int>(threadIdx.x) < p.num_seqs;     // (of a sequence)
    Raw seen{0, 0, 0};
    auto put = [&]() {
        copy[threadIdx.x] = seen.L;
        copy[kThreads + threadIdx.x] = seen.q0;
        copy[2 * kThreads + threadIdx.x] = seen.q1;
    };
    if (owner) {
        // (The self-test of the second look has the first one look elsewhere.)
        const int32_t *lens = p.lens_ahead ? p.lens_ahead : p.seq_lens, *cu = p.cu_ahead ? p.cu_ahead : p.cu_q_lens;
        seen = {load_cg(lens + threadIdx.x), load_cg(cu + threadIdx.x), load_cg(cu + threadIdx.x + 1)};
        put();
    }
    if (ahead) __syncthreads();
    else wait_prev();
    int odd;
    int64_t T;
#pragma unroll 1
    for (;;) {
        T = plan<D, TWO>(p, misc, copy, lgG, c, C, &odd);
        if (!ahead) break;
        ahead = false;
        wait_prev();
        bool changed = false;
        if (owner) {
            const Raw now = load_raw(p, threadIdx.x);
            changed = now.L != seen.L || now.q0 != seen.q0 || now.q1 != seen.q1;
            seen = now;
            put();
        }
        if (!__syncthreads_or(changed)) break;
    }
    fence_proxy_async_smem();                // the copy's place goes to the rings
    const Pos from = misc->pos[0];
    const int64_t n_tiles = misc->pos[1].tile - from.tile;
    if (threadIdx.x == 0 && p.slots) {
        SlotHead *hd = reinterpret_cast<SlotHead *>(slot_at(p, slot_sz, c, 0));
        hd->flag = 0;
        hd->range_beg = from.tile;
    }
    // Sequences out of range are reported, and rows without keys get zeros, by CTA s % C.
    if (odd) {
        for (int s = c; s < p.num_seqs; s += C) {
            const Seq q = load_seq<TWO>(p, s, lgG);
            if (q.bad && threadIdx.x == 0) set_error(p.err, PK_DEVERR_SEQ_LEN);
            if (q.qn == 0 || q.L != 0) continue;
            const float zero[16] = {};
            const size_t first = static_cast<size_t>(q.q0) * H * D;
            for (int64_t i = threadIdx.x; i < static_cast<int64_t>(q.qn) * H * (D / 16); i += kThreads)
                store_row<16>(p, first + 16 * i, zero);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc->tmem_base;

    Walk<TWO> walk(p, lgG, from, n_tiles);
    Part a;
    auto give_up = [&]() {
        misc->abort = 1;
        set_error(p.err, PK_DEVERR_TIMEOUT);
    };
    // Query buffers.  TWO: one for each group, whose query tile it holds (the same one in
    // both where the block has one).  Otherwise one of 128 rows, or two of at most 64
    // that the parts take in turn.
    const uint32_t q_chunk = static_cast<uint32_t>(max(8, q_box << lgG)) * 128u;
    const uint32_t q_slot = q_chunk * NCH;

    if (warp == 8 || warp == 9) {
        // ================= producers: warp 8 Q and K, warp 9 V =================
        const bool kprod = warp == 8;
        const int MB = p.max_blocks_per_seq;
        const int nst = kprod ? KS : VS;
        uint64_t *full = kprod ? misc->kfull : misc->vfull, *empty = kprod ? misc->kempty : misc->vempty;
        const uint32_t ring = base + (kprod ? C_::kKOff : C_::kVOff);
        const void *tm = kprod ? static_cast<const void *>(&tm_k) : static_cast<const void *>(&tm_v);
        int issued = 0, st = 0, q_issued = 0;
        uint32_t ph = 1;
        bool ok_run = true, stalled = false;
        int part = 0;
        while (ok_run && walk.next(a)) {
            if (kprod) {
                int got = 1;
                if (lane == 0) {
                    const uint32_t bytes = static_cast<uint32_t>(q_box << lgG) * 128u * NCH;
                    for (int x = 0; x < (TWO ? 2 : 1); ++x) {
                        const int sl = TWO ? x : (q_slots == 2 ? part & 1 : 0);
                        const int fill = TWO || q_slots == 1 ? part : part >> 1;
                        got = mbar_wait(smem_u32(&misc->qempty[sl]), (fill & 1) ^ 1, &misc->abort, lim);
                        if (!got) break;
                        const uint32_t bar = smem_u32(&misc->qfull[sl]);
                        mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
                        for (int ch = 0; ch < NCH; ++ch)
                            tma_load_3d(base + sl * q_slot + ch * q_chunk, &tm_q, bar, ch * 64, a.h * G,
                                        walk.q.q0 + a.tok0 + (a.two ? x * QT : 0));
                        ++q_issued;
                    }
                }
                if (!__shfl_sync(0xffffffffu, got, 0)) {
                    if (lane == 0) give_up();
                    break;
                }
            }
            const int L = walk.q.L;
            const int32_t *table = p.block_tables + static_cast<size_t>(a.s) * MB;
            // Block-table entries of a key tile, one page per lane; the next
            // tile's are fetched while the current tile's copies are issued.
            auto fetch = [&](int t) -> int {
                const int tok = t * kKeys;
                const int pg = (min(kKeys, L - tok) + B - 1) / B;
                return lane < pg ? table[tok / B + lane] : -1;
            };
            int phys_next = fetch(a.t0);
            for (int t = a.t0; t < a.t1; ++t) {
                // Self-test of the bounded waits: CTA 0 stops copying keys here.
                if (kprod && p.stall_tile > 0 && c == 0 && issued == p.stall_tile) {
                    stalled = true;
                    ok_run = false;
                    break;
                }
                const int phys = phys_next;
                int got = 1;
                if (lane == 0) got = mbar_wait(smem_u32(&empty[st]), ph, &misc->abort, lim);
                if (!__shfl_sync(0xffffffffu, got, 0)) {
                    if (lane == 0) give_up();
                    ok_run = false;
                    break;
                }
                const int vlen = min(kKeys, L - t * kKeys);
                const int r0 = lane * B;
                const bool in = r0 < vlen;
                const bool ok = in && phys >= 0 && phys < p.num_blocks;
                const uint32_t nok = __popc(__ballot_sync(0xffffffffu, ok));
                const uint32_t bar = smem_u32(&full[st]);
                if (kprod) {
                    if (in && !ok) set_error(p.err, PK_DEVERR_BLOCK_ID);
                    uint32_t bits = 0;
                    if (ok) {
                        const int nrows = min(B, vlen - r0);
                        bits = (nrows >= 32 ? 0xffffffffu : ((1u << nrows) - 1u)) << (r0 & 31);
                    }
                    const int word = r0 >> 5;
                    // Rows that P.V reads and that hold no key: the end of the last 16, and
                    // pages that are not there.
                    const bool stale = (vlen & 15) != 0 || nok * B < static_cast<uint32_t>(vlen);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t m = __reduce_or_sync(0xffffffffu, word == w ? bits : 0u);
                        if (lane == 0) misc->mask[issued & (C_::kMasks - 1)][w] = m;
                    }
                    if (lane == 0)
                        misc->meta[issued & (C_::kMasks - 1)] =
                            (a.two ? kMetaTwo : 0u) | (t == a.t0 ? kMetaFirst : 0u) | (t == a.t1 - 1 ? kMetaLast : 0u) |
                            (stale ? kMetaStale : 0u) | static_cast<uint32_t>(vlen) << kMetaKeysShift;
                }
                if (lane == 0) mbar_arrive_expect_tx(bar, nok * B * 128u * NCH);
                __syncwarp();
                // One box per page, at the page's place in the tile.
                if (ok) tma_load_5d(ring + st * kTile + r0 * 128 * NCH, tm, bar, 0, 0, 0, phys * (B >> 3), a.h);
                ++issued;
                if (++st == nst) {
                    st = 0;
                    ph ^= 1;
                }
                if (t + 1 < a.t1) phys_next = fetch(t + 1);
            }
            ++part;
            walk.advance();
        }
        if ((misc->abort || stalled) && lane == 0) {
            // Let the copies in flight land before the CTA can exit.
            for (int i = max(0, issued - nst); i < issued; ++i)
                mbar_wait(smem_u32(&full[i % nst]), (i / nst) & 1, &misc->never, lim);
            // (The last fill of each query buffer: fills come in turn.)
            const int bufs = TWO || q_slots == 2 ? 2 : 1;
            for (int i = max(0, q_issued - bufs); i < q_issued; ++i)
                mbar_wait(smem_u32(&misc->qfull[i % bufs]), (i / bufs) & 1, &misc->never, lim);
        }
    } else if (warp >= 10) {
        // ================= MMA issuers: warp 10 of group 0, 11 of group 1 =================
        // At job j, P.V of job j - 2 (whose P lies in the buffer that S is going to) and S of
        // job j.  Every tile is used by both groups, so both see every phase of the rings
        // in order.
        const int x = __shfl_sync(0xffffffffu, warp, 0) - 10;
        constexpr uint32_t kIdescO = idesc_bf16(kRows, D, 0, 1);           // A = P (TMEM), B = V (MN-major)
        // Descriptors of the rings' starts; an address moves on in 16-byte units.
        const uint64_t qdesc = smem_desc(base, 16, 1024, kLayoutSw128);
        const uint64_t kdesc = smem_desc(base + C_::kKOff, 16, kAtomStride, kLayoutSw128);
        const uint64_t vdesc = smem_desc(base + C_::kVOff, 1024, kAtomStride, kLayoutSw128);
        const uint32_t scol = __shfl_sync(0xffffffffu, tmem, 0) + kTmemS + x * 128, ocol = scol + kTmemO - kTmemS;
        auto wait = [&](uint64_t *bar, int phase) -> bool { return warp_wait(bar, phase, &misc->abort, lim); };
        auto there = [&](uint64_t *bar, int phase) -> bool {
            return __all_sync(0xffffffffu, mbar_test_wait(smem_u32(bar), phase & 1));
        };
        const int n_all = __shfl_sync(0xffffffffu, static_cast<int>(n_tiles), 0);
        bool alive = true;
        int kt = 0, kslot = 0, kpar = 0, vslot = 0, vpar = 0;
        bool vready = false;                   // the V tile at the ring's head has been waited for
        int s_jobs = 0, pv_jobs = 0;           // S and P.V issued
        // The jobs whose P.V is to come, by buffer: kMeta* bits (first and last as they are
        // for this job), keys (0-64) and half.
        uint32_t jinfo0 = 0, jinfo1 = 0;
        int jkt0 = 0, jkt1 = 0;
        int part = -1, half = 0, h_hi = 0;
        uint32_t mt = 0;                       // the current tile, once it has been opened
        bool opened = false;
        while (alive && (kt < n_all || pv_jobs < s_jobs)) {
            // What is next: the product of the job two before; or, where the next tile (or
            // the part's queries) is not there yet, that of a job before, so that its part
            // can end; or S.
            if (!opened && kt < n_all) {
                if (pv_jobs == s_jobs && !wait(&misc->kfull[kslot], kpar)) break;
                if (pv_jobs == s_jobs || there(&misc->kfull[kslot], kpar)) {
                    mt = __shfl_sync(0xffffffffu, misc->meta[kt & (C_::kMasks - 1)], 0);
                    opened = true;
                    if (mt & kMetaFirst) {
                        const int sl = TWO ? x : (q_slots == 2 ? (part + 1) & 1 : 0);
                        const int fill = TWO || q_slots == 1 ? part + 1 : (part + 1) >> 1;
                        if (pv_jobs == s_jobs && !wait(&misc->qfull[sl], fill)) break;
                        opened = pv_jobs == s_jobs || there(&misc->qfull[sl], fill);
                        part += opened;
                    }
                    half = mt & kMetaTwo ? 0 : x;
                    h_hi = mt & kMetaTwo ? 1 : x;
                }
            }
            if (pv_jobs < s_jobs && (!opened || s_jobs - pv_jobs == 2)) {
                const int u = pv_jobs & 1;
                const uint32_t info = u ? jinfo1 : jinfo0;
                const int n16 = (((info >> kMetaKeysShift) & 255) + 15) >> 4, hf = info >> 16;
                if (!wait(&misc->p_full[x][u], pv_jobs >> 1) || (!vready && !wait(&misc->vfull[vslot], vpar))) {
                    alive = false;
                    break;
                }
                vready = true;
                if (info & kMetaStale) {
                    // V rows of keys outside the sequence or behind a bad table entry may hold
                    // stale or non-finite bits, which weights of 0 do not cancel: zero those
                    // that the product reads.  (Both groups may do so, with the same zeros.)
                    const int pkt = u ? jkt1 : jkt0;
#pragma unroll 1
                    for (int q4 = 0; q4 < 2; ++q4) {
                        const int nrow = max(0, min(32, n16 * 16 - 32 * q4));
                        uint32_t gone = ~misc->mask[pkt & (C_::kMasks - 1)][2 * hf + q4];
                        if (nrow < 32) gone &= (1u << nrow) - 1u;
#pragma unroll 1
                        while (gone) {
                            const int r = 64 * hf + 32 * q4 + __ffs(gone) - 1;
                            gone &= gone - 1;
                            if (lane < 8 * NCH)
                                *reinterpret_cast<uint4 *>(smem + C_::kVOff + vslot * kTile + (r >> 3) * kAtomStride +
                                                           (lane >> 3) * 1024 + (r & 7) * 128 + (lane & 7) * 16) =
                                    make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                tc_fence_after();
                if (elect_one()) {
                    // Keys 16kk .. 16kk+15: 8-row blocks 2kk and 2kk + 1; the two 64-element
                    // halves of the head 1,024 bytes apart.
                    const uint64_t vd = vdesc + static_cast<uint32_t>(vslot) * (kTile >> 4) + hf * (8 * kAtomStride >> 4);
                    const uint32_t acol = scol + u * kHalf;
#pragma unroll
                    for (int kk = 0; kk < kHalf / 16; ++kk)
                        if (kk < n16)
                            mma_bf16_tmem_a(ocol, acol + kk * 8, vd + kk * (2 * kAtomStride >> 4), kIdescO,
                                            kk > 0 || !(info & kMetaFirst) ? 1u : 0u);
                    mma_commit(smem_u32(&misc->pv_done[x][u]));
                    if (info & kMetaLast) mma_commit(smem_u32(&misc->vempty[vslot]));   // the group's last of this tile
                }
                __syncwarp();
                if (info & kMetaLast) {
                    vready = false;
                    if (++vslot == VS) {
                        vslot = 0;
                        vpar ^= 1;
                    }
                }
                ++pv_jobs;
                continue;
            }
            if (!opened) continue;
            const int u = s_jobs & 1;
            const int sl = TWO ? x : (q_slots == 2 ? part & 1 : 0);
            const int n = max(0, min(kHalf, static_cast<int>(mt >> kMetaKeysShift) - half * kHalf));
            const bool done = half == h_hi;        // the group's last S of this tile
            tc_fence_after();
            if (elect_one()) {
                const uint64_t kd = kdesc + static_cast<uint32_t>(kslot) * (kTile >> 4) + half * (8 * kAtomStride >> 4);
                const uint64_t qd = qdesc + ((static_cast<uint32_t>(sl) * q_slot) >> 4);
                const uint32_t idesc = idesc_bf16(kRows, (n + 15) & ~15, 0, 0);   // A = Q, B = K, both K-major
                if (n > 0) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_bf16(scol + u * kHalf, qd + (((kk >> 2) * q_chunk + (kk & 3) * 32) >> 4),
                                 kd + (((kk >> 2) * 1024u + (kk & 3) * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
                }
                mma_commit(smem_u32(&misc->s_full[x][u]));
                if (done) {
                    mma_commit(smem_u32(&misc->kempty[kslot]));
                    if (mt & kMetaLast) mma_commit(smem_u32(&misc->qempty[sl]));   // the part's last scores
                }
            }
            __syncwarp();
            const uint32_t info = (mt & kMetaStale) | ((mt & kMetaFirst) && (half == 0 || !(mt & kMetaTwo)) ? kMetaFirst : 0u) |
                                  (done ? kMetaLast : 0u) | static_cast<uint32_t>(n) << kMetaKeysShift |
                                  static_cast<uint32_t>(half) << 16;
            if (u) {
                jinfo1 = info;
                jkt1 = kt;
            } else {
                jinfo0 = info;
                jkt0 = kt;
            }
            ++s_jobs;
            ++half;
            if (done) {
                opened = false;
                ++kt;
                if (++kslot == KS) {
                    kslot = 0;
                    kpar ^= 1;
                }
            }
        }
        if ((!alive || kt < n_all || pv_jobs < s_jobs) && lane == 0) give_up();
        // Let every issued MMA finish before the CTA can release TMEM.
        if (elect_one()) mma_commit(smem_u32(&misc->drain[x]));
        __syncwarp();
        wait_on(smem_u32(&misc->drain[x]), 0, &misc->never, lim);
    } else {
        // ================= softmax: warps 0-3 group 0, 4-7 group 1; thread <-> query row =================
        const int x = warp >> 2;
        const int quad = warp & 3;                      // TMEM lanes 32 * (warp % 4) ..
        const int row = quad * 32 + lane;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const uint32_t o_col = lane_addr + kTmemO + x * 128;
        const uint32_t o_other = lane_addr + kTmemO + (1 - x) * 128;
        const int half_d = x * (D / 2);                 // of a joined part, a group gives out half of each row
        const int rr = row >> lgG;                      // query token of this row in its tile
        const float cs = p.scale_log2;
        const uint64_t c2 = f2(cs, cs);
        const uint32_t unseen = __float_as_uint(cs > 0.f ? -INFINITY : INFINITY);
        int ktile = 0;                                  // key tile (of the CTA's range) at the part's start
        int jobs = 0;                                   // jobs so far (both groups have as many)
        int joins = 0;                                  // joins of two groups so far
        float m_ref = -INFINITY;                        // the row's reference max
        bool owe = false;                               // the other group still reads this group's O
        bool alive = true;
        auto wait = [&](uint64_t *bar, int phase) -> bool { return warp_wait(bar, phase, &misc->abort, lim); };
        while (alive && walk.next(a)) {
            const Seq q = walk.q;
            const int per = a.two ? 2 : 1;
            const int njobs = (a.t1 - a.t0) * per;
            const int tok0 = a.tok0 + (a.two ? x * QT : 0);   // first query token of this tile
            const int ntok = min(q.qn - tok0, QT);
            const bool busy = (quad * 32) >> lgG < ntok;      // this warp has a row in use
            const bool idle_row = rr >= ntok;
            const int base_pos = q.L - q.qn;                  // position of the tree's node 0
            const uint32_t *mrow_bits = p.tree_mask && busy
                ? p.tree_mask + static_cast<size_t>(q.q0 + tok0 + min(rr, ntok - 1)) * p.mask_words : nullptr;
            // The first key of job i of the part.
            auto job_key = [&](int i) -> int {
                return a.two ? a.t0 * kKeys + i * kHalf : (a.t0 + i) * kKeys + x * kHalf;
            };
            // The mask words that the 64 keys of a job can touch, read a job ahead: all
            // ones before node 0 (the context), zeros behind the row's words.
            uint32_t mw[3];
            auto fetch_mask = [&](int i) {
                const int at = (job_key(i) - base_pos) >> 5;         // (rounds down)
                if (!mrow_bits || i >= njobs || at <= -3) return;    // (-3: nothing of the tree in these keys)
#pragma unroll
                for (int w = 0; w < 3; ++w)
                    mw[w] = at + w < 0 ? 0xffffffffu : (at + w < p.mask_words ? mrow_bits[at + w] : 0u);
            };
            if (!(fabsf(m_ref) < 1e30f)) m_ref = -INFINITY;    // (the part before's, as a guess)
            float l_run = 0.f;
            fetch_mask(0);
            for (int i = 0; i < njobs; ++i, ++jobs) {
                const int u = jobs & 1;
                const int key0 = job_key(i);
                const int kt = ktile + (key0 >> 7) - a.t0;
                if (!wait(&misc->s_full[x][u], jobs >> 1)) {
                    alive = false;
                    break;
                }
                tc_fence_after();
                const uint32_t s_col = lane_addr + kTmemS + x * 128 + u * kHalf;
                if (busy) {
                    uint32_t sc[64];
                    tmemw::ld64(s_col, sc);
                    const uint32_t *valid = &misc->mask[kt & (C_::kMasks - 1)][(key0 >> 5) & 2];
                    uint32_t v0 = valid[0], v1 = valid[1];
                    const int off = key0 - base_pos;
                    if (mrow_bits && (off >> 5) > -3) {
                        v0 &= __funnelshift_r(mw[0], mw[1], off & 31);
                        v1 &= __funnelshift_r(mw[1], mw[2], off & 31);
                    }
                    fetch_mask(i + 1);
                    // One pass over the row: weights against the reference max as it is,
                    // and the largest score beside them.  Only where that moves the
                    // reference (the first part's first job, seldom later) is the pass made again.
                    // P is bf16 pairs over the first half of S (the A operand of P.V): half
                    // the tensor work of fp32 weights at an error of 2^-8 of each; the
                    // denominator sums the rounded weights, so that their mean stays one.
                    uint32_t packed[32];
                    float lsum;
                    tmemw::wait_ld(sc);
                    // Scores of keys that the row does not see become the one that weighs
                    // nothing (c is not 0), unless every row in use sees all of them.
                    if (!__all_sync(0xffffffffu, idle_row || (v0 & v1) == 0xffffffffu)) {
#pragma unroll
                        for (int n = 0; n < 64; ++n)
                            sc[n] = ((n < 32 ? v0 : v1) >> (n & 31)) & 1u ? sc[n] : unseen;
                    }
                    // (Two moves at most: scores whose rounding exceeds the threshold would
                    // ask for ever.)
                    for (int pass = 0;; ++pass) {
                        const float nm = m_ref == -INFINITY ? 0.f : -m_ref;
                        const uint64_t nm2 = f2(nm, nm);
                        uint64_t lacc[2] = {0ull, 0ull};
                        // The largest c s - m_ref (c s where there is no m_ref yet).
                        float e[4];
#pragma unroll
                        for (int n = 0; n < 4; ++n) e[n] = -INFINITY;
#pragma unroll
                        for (int n = 0; n < 64; n += 2) {
                            const float2 arg = unf2(fma2(f2(__uint_as_float(sc[n]), __uint_as_float(sc[n + 1])), c2, nm2));
                            e[(n >> 1) & 3] = max3(e[(n >> 1) & 3], arg.x, arg.y);
                            const uint32_t w = pack_bf16x2(ex2(arg.x), ex2(arg.y));
                            packed[n / 2] = w;
                            lacc[(n >> 1) & 1] = add2(lacc[(n >> 1) & 1], f2(bf16_lo(w), bf16_hi(w)));
                        }
                        const float tmax = fmaxf(max3(e[0], e[1], e[2]), e[3]);
                        const float2 la = unf2(lacc[0]), lb = unf2(lacc[1]);
                        lsum = (la.x + la.y) + (lb.x + lb.y);
                        bool need = m_ref == -INFINITY ? tmax > -INFINITY : tmax > 0.f;
                        if (i == 0) {
                            if (tmax == -INFINITY) m_ref = -INFINITY;      // nothing seen: no reference
                            else need |= tmax < kGuessLog2;
                        }
                        need &= !idle_row;
                        if (pass == 2 || !__any_sync(0xffffffffu, need)) break;
                        // Move this row's reference max and rescale its O (of the jobs so
                        // far) and denominator.
                        const float mn = need ? ceilf(m_ref == -INFINITY ? tmax : m_ref + tmax) + kHeadroomLog2 : m_ref;
                        const float f = rescale(m_ref, mn);
                        if (i > 0) {
                            if (!wait(&misc->pv_done[x][u ^ 1], (jobs - 1) >> 1)) {
                                alive = false;
                                break;
                            }
                            tc_fence_after();
#pragma unroll 1
                            for (int cc = 0; cc < D / 8; ++cc) {
                                float ov[8];
                                tmem_ld<8>(o_col + cc * 8, ov);
#pragma unroll
                                for (int n = 0; n < 8; ++n) ov[n] *= f;
                                tmem_st8(o_col + cc * 8, ov);
                            }
                        }
                        l_run *= f;
                        m_ref = mn;
                    }
                    if (!alive) break;
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        uint32_t pk16[16];
#pragma unroll
                        for (int n = 0; n < 16; ++n) pk16[n] = packed[cc * 16 + n];
                        tmem_st16(s_col + cc * 16, pk16);      // keys 32cc .. 32cc+31 of this row
                    }
                    l_run += lsum;
                }
                // The first product of a part overwrites O: the other group has to have
                // read its half of it, where they joined the last part.
                if (owe) {
                    if (!wait(&misc->o_taken[1 - x], joins - 1)) {
                        alive = false;
                        break;
                    }
                    owe = false;
                }
                tmem_wait_st();                     // P is in TMEM before the MMA may read it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&misc->p_full[x][u]));
            }
            if (!alive) break;
            // ---- the part's end ----
            // P.V of the last jobs done.  (Probes of a phase are exact when the one before is
            // known to be over: S of the last job followed P.V of the one before in its
            // buffer; the other group has left m and l after its last S.)
            const bool joined = !a.two;
            const int last = jobs - 1;                      // both groups' last job
            const bool complete = a.t0 == 0 && a.t1 == q.nt;
            float f_own = 1.f, f_other = 0.f;
            if (joined) {
                // m and l of both groups, through one place: group 0's, then group 1's.
                if (x == 0) {
                    misc->part.m[row] = m_ref;
                    misc->part.l[row] = l_run;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&misc->ml_ready[0]));
                }
                if (!wait(&misc->ml_ready[1 - x], joins)) {
                    alive = false;
                    break;
                }
                const float m2 = misc->part.m[row], l2 = misc->part.l[row];
                if (x == 1) {
                    misc->part.m[row] = m_ref;
                    misc->part.l[row] = l_run;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&misc->ml_ready[1]));
                }
                const float mm = fmaxf(m_ref, m2);
                f_own = rescale(m_ref, mm);
                f_other = rescale(m2, mm);
                l_run = l_run * f_own + l2 * f_other;
                m_ref = mm;
            }
            if (!wait(&misc->pv_done[x][last & 1], last >> 1) ||
                (joined && !wait(&misc->pv_done[1 - x][last & 1], last >> 1))) {
                alive = false;
                break;
            }
            tc_fence_after();
            if (complete) {
                const float inv = l_run > 0.f ? 1.f / l_run : (l_run == 0.f ? 0.f : l_run);
                f_own *= inv;
                f_other *= inv;
            }
            const int tile_x = a.two ? x : 0;
            const bool first_part = a.s == from.s && a.h == from.h && a.j == from.j;
            char *slot = complete ? nullptr : slot_at(p, slot_sz, c, first_part ? 0 : 1);
            if (busy) {
                const bool use = rr < ntok;
                const size_t oidx = (static_cast<size_t>(q.q0 + tok0 + rr) * H + a.h * G + (row & (G - 1))) *
                                    static_cast<size_t>(D);
                // (A group whose halves held no key has written no O at all.)
                auto part_of = [](uint32_t v, float g) -> float { return g == 0.f ? 0.f : __uint_as_float(v) * g; };
                const int lo = joined ? half_d : 0, hi = joined ? half_d + D / 2 : D;
#pragma unroll 1
                for (int d = lo; d < hi; d += 32) {
                    float f[32];
                    uint32_t ov[32];
                    tmemw::ld32(o_col + d, ov);
                    if (joined) {
                        uint32_t ow[32];
                        tmemw::ld32(o_other + d, ow);
                        tmemw::wait_ld(ov);
                        tmemw::wait_ld(ow);
#pragma unroll
                        for (int n = 0; n < 32; ++n) f[n] = part_of(ov[n], f_own) + part_of(ow[n], f_other);
                    } else {
                        tmemw::wait_ld(ov);
#pragma unroll
                        for (int n = 0; n < 32; ++n) f[n] = __uint_as_float(ov[n]) * f_own;
                    }
                    // (The last reads of O: the other group may overwrite its own before the
                    // stores, slow while the copies fill the memory, are out.)
                    if (joined && d + 32 == hi) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&misc->o_taken[x]));
                    }
                    if (!complete) {
                        float *so = slot_m(slot, tile_x, D) + 2 * kRows + static_cast<size_t>(d) * kRows + row;
#pragma unroll
                        for (int n = 0; n < 32; ++n) so[n * kRows] = f[n];
                    } else if (use) {
                        store_row<32>(p, oidx + d, f);
                    }
                }
            } else if (joined && lane == 0) {
                mbar_arrive(smem_u32(&misc->o_taken[x]));
            }
            if (!complete && (a.two || x == 0)) {
                float *sm = slot_m(slot, tile_x, D);
                sm[row] = m_ref;
                sm[kRows + row] = l_run;
                if (row == 0 && tile_x == 0) {
                    SlotHead *hd = reinterpret_cast<SlotHead *>(slot);
                    hd->h = a.h;
                    hd->tok0 = a.tok0;
                    hd->ntiles = per;
                    hd->q0 = q.q0;
                    hd->qn = q.qn;
                    if (first_part) {
                        // Cut at its start and finished here: this CTA's merge joins it.
                        hd->start_tile = from.tile - a.t0;
                        hd->total_tiles = T;
                        hd->first_cta = misc->first_cta;
                        hd->flag = a.t0 > 0 && a.t1 == q.nt ? 1 : 0;
                    }
                }
            }
            if (joined) {
                owe = true;
                ++joins;
            }
            ktile += a.t1 - a.t0;
            walk.advance();
        }
        if (!alive) give_up();
        tc_fence_before();
    }

    __syncthreads();
    if (warp == 10) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// One block per CTA c of the attention grid: where c's first segment was cut at its
// start and ends in c, join its parts.  A thread has a query row and 16 elements of the
// head (O^T in the slots makes the reads whole lines); the parts come two at a time,
// their loads in flight together.  Few large blocks: 152 of them are launched in 1.5 us,
// 2,432 of 128 threads in 3.8 us.
constexpr int kMergeThreads = 1024;

template <int D>
__global__ void __launch_bounds__(kMergeThreads)
rows_merge_kernel(const __grid_constant__ RowsParams p, int C, int slot_tiles) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const size_t slot_sz = slot_bytes<D>(slot_tiles);
    const int c = blockIdx.x, row = threadIdx.x & (kRows - 1);
    auto head = [&](int cc) -> const SlotHead * {
        return reinterpret_cast<const SlotHead *>(slot_at(p, slot_sz, cc, 0));
    };
    const SlotHead hd = *head(c);
    const int64_t before = head(c > 0 ? c - 1 : 0)->range_beg;     // (the usual first part's)
    if (hd.flag != 1) return;
    const int lgG = __ffs(p.num_heads / p.num_kv_heads) - 1, G = 1 << lgG;
    const int q0 = hd.q0, qn = hd.qn;
    // A header of another call (one on another stream that was given the same workspace)
    // leads nowhere outside the slots and the output.
    if (hd.first_cta < 0 || hd.first_cta > c || hd.ntiles < 1 || hd.ntiles > slot_tiles || hd.h < 0 ||
        hd.h >= p.num_kv_heads || hd.tok0 < 0 || hd.tok0 >= qn || q0 < 0 || q0 > p.total_q - qn) {
        if (threadIdx.x == 0) set_error(p.err, PK_DEVERR_WORKSPACE);
        return;
    }
    // CTA cc's part, from its slot 0 if the segment is the first of its range, else 1; a
    // range may be empty (more CTAs than tiles) and then has none.
    auto range_beg = [&](int cc) -> int64_t { return cc == c ? hd.range_beg : cc == c - 1 ? before : head(cc)->range_beg; };
    for (int unit = threadIdx.x / kRows; unit < hd.ntiles * (D / 16); unit += kMergeThreads / kRows) {
        const int x = unit / (D / 16), d0 = unit % (D / 16) * 16;
        const int tok = hd.tok0 + x * (kRows >> lgG) + (row >> lgG);
        if (tok >= qn) continue;
        float M = -INFINITY, l = 0.f, o[16];
#pragma unroll
        for (int n = 0; n < 16; ++n) o[n] = 0.f;
        int64_t rb = range_beg(hd.first_cta);
#pragma unroll 1
        for (int cc = hd.first_cta; cc <= c; cc += 2) {
            const bool two = cc + 1 <= c;
            const int64_t r1 = two ? range_beg(cc + 1) : hd.total_tiles, r2 = cc + 2 <= c ? range_beg(cc + 2) : hd.total_tiles;
            float m[2], lp[2], v[2][16];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bool some = u == 0 ? cc == c || r1 > rb : two && (cc + 1 == c || r2 > r1);
                const float *sm = slot_m(slot_at(p, slot_sz, two ? cc + u : cc, (u ? r1 : rb) >= hd.start_tile ? 0 : 1), x, D) + row;
                m[u] = some ? sm[0] : -INFINITY;
                lp[u] = some ? sm[kRows] : 0.f;
#pragma unroll
                for (int n = 0; n < 16; ++n) v[u][n] = some ? sm[(2 + d0 + n) * kRows] : 0.f;
            }
            rb = r2;
            const float mm = max3(M, m[0], m[1]);
            const float f = rescale(M, mm), f0 = rescale(m[0], mm), f1 = rescale(m[1], mm);
            l = l * f + (lp[0] * f0 + lp[1] * f1);
#pragma unroll
            for (int n = 0; n < 16; ++n) o[n] = o[n] * f + (v[0][n] * f0 + v[1][n] * f1);
            M = mm;
        }
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
        for (int n = 0; n < 16; ++n) o[n] *= inv;
        store_row<16>(p, (static_cast<size_t>(q0 + tok) * p.num_heads + hd.h * G + (row & (G - 1))) * static_cast<size_t>(D) + d0,
                      o);
    }
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        else
            cudaGetLastError();
    });
    return fn;
}

// A tiled bf16 map with the 128-byte swizzle the MMA descriptors expect.
bool encode(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
            const cuuint32_t *box) {
    auto enc = encoder();
    if (!enc) return false;
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks of two query tiles exist where a sequence can have more rows than one holds.
bool two_tiles(int num_heads, int num_kv_heads, int max_q_len) {
    return max_q_len > kRows / (num_heads / num_kv_heads);
}

template <int D, bool TWO>
cudaError_t launch(const RowsParams &p, cudaStream_t stream) {
    using C_ = Cfg<D, TWO>;
    const cuuint64_t Dd = D, Hkv = p.num_kv_heads, B = p.block_size;
    const cuuint64_t P = p.num_blocks > 0 ? p.num_blocks : 1;
    const int G = p.num_heads / p.num_kv_heads;
    // K and V: one box per (page, KV head) holding its B rows as B / 8 blocks of
    // [half][8 rows][64] (dimensions: 64 elements; row within the block; half, 128
    // bytes apart; 8-row block, page * B / 8 + block; KV head).
    const cuuint64_t pdims[5] = {64, 8, Dd / 64, P * (B / 8), Hkv};
    const cuuint64_t pstr[4] = {Hkv * Dd * 2, 128, 8 * Hkv * Dd * 2, Dd * 2};
    const cuuint32_t pbox[5] = {64, 8, static_cast<cuuint32_t>(Dd / 64), static_cast<cuuint32_t>(B / 8), 1};
    // Queries [total_q, H, D]: box (64 elements, G heads, q_box tokens), row =
    // token * G + head; no more tokens than a sequence has, rounded up to a power of
    // two.
    int q_box = kRows / G;
    if (!TWO)
        while (q_box > 1 && q_box / 2 >= p.max_q_len) q_box /= 2;
    const int q_slots = TWO || q_box * G <= kRows / 2 ? 2 : 1;
    const cuuint64_t qdims[3] = {Dd, static_cast<cuuint64_t>(p.num_heads), static_cast<cuuint64_t>(p.total_q)};
    const cuuint64_t qstr[2] = {Dd * 2, Dd * p.num_heads * 2};
    const cuuint32_t qbox[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(q_box)};
    CUtensorMap mk, mv, mq;
    if (!encode(&mq, p.q, 3, qdims, qstr, qbox)) return cudaErrorInvalidValue;
    if (p.k_cache) {
        if (!encode(&mk, p.k_cache, 5, pdims, pstr, pbox) || !encode(&mv, p.v_cache, 5, pdims, pstr, pbox))
            return cudaErrorInvalidValue;
    } else {
        mk = mv = mq;                    // no sequence can have keys: never read
    }
    constexpr int smem = static_cast<int>(1024 + C_::kEnd + sizeof(Misc<C_::kKS, C_::kVS, C_::kMasks>));
    {
        const cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(rows_attention_kernel<D, TWO>), smem);
        if (e != cudaSuccess) return e;
    }
    // No more CTAs than the longest sequences could have key tiles.
    int C = std::min(sm_count(), kRowsMaxCtas);
    if (C <= 0) return cudaErrorNoDevice;
    const int64_t qt = kRows / G;
    const int64_t tiles = static_cast<int64_t>(p.num_seqs) * p.num_kv_heads * ((p.max_q_len + qt - 1) / qt) *
                          ((static_cast<int64_t>(p.max_seq_len) + kKeys - 1) / kKeys);
    C = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(C, tiles)));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, rows_attention_kernel<D, TWO>, mk, mv, mq, p, q_box, q_slots);
    if (e != cudaSuccess || !p.slots) return e;          // without slots nothing is cut
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, rows_merge_kernel<D>, p, C, TWO ? 2 : 1);
}

}  // namespace

size_t rows_workspace_bytes(int num_heads, int num_kv_heads, int head_dim, int max_q_len) {
    const int tiles = two_tiles(num_heads, num_kv_heads, max_q_len) ? 2 : 1;
    return 2 * kRowsMaxCtas * (head_dim == 64 ? slot_bytes<64>(tiles) : slot_bytes<128>(tiles));
}

cudaError_t launch_rows_attention(const RowsParams &p, cudaStream_t stream) {
    const bool two = two_tiles(p.num_heads, p.num_kv_heads, p.max_q_len);
    if (p.head_dim == 64) return two ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
    return two ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
}

}  // namespace pk
