// Attention over the 8-bit paged cache on the 5th-generation tensor cores.
//
// Mathematics.  With ks, vs the scales of a token's block and KV head,
//   s_j = scale * ks_j * (q . k_j),  out = sum_j 2^(t_j - m) v_j / sum_j 2^(t_j - m) / vs_j,
//   t_j = s_j log2(e) + log2(vs_j),
// k_j and v_j the stored e4m3 rows.  Both contractions run on kind::f8f6f4
// MMAs straight from the pages as TMA lands them: nothing widens K or V.  The
// other operands are split into 8-bit terms that each take columns of their own:
//   q * 2^k = h + l / 32, 2^k bringing the row's largest to [128, 256): two e4m3
//     terms hold a bf16 value exactly down to 2^-13 of the row's largest, and
//     what is smaller to 2^-22 of it.
//   u = 2^(t - m) = h1 + h2 + h3, e5m2 terms of u rounded to fp16, u <= 2^15: three
//     hold an fp16 value exactly down to 2^-6, so u to 2^-11 of itself, and below
//     to 2^-17, which is 2^-24 of the largest weight: that is 2^7 or more (m moves
//     when a u exceeds 2^15).  bf16 weights are to 2^-8.  e4m3 terms with scales
//     between them have a bit more each but 2^-20 of the largest weight for small
//     ones: a tail of 16,000 tokens 2^-16 below one peak was off by 6 % (a tail's
//     weights are alike, so their rounding does not average out).
// The extra columns cost MMA time only: the tensor pipe is active 7 % of
// the time.
//
// Bound: HBM bytes of the cache, 2 D a token and KV head.  The work split, the
// reference maximum that moves rarely and the bounded waits are those of the
// bf16 kernel (decode_tc.cu, decode_split.cuh).  What half the bytes a token
// changed: a tile's bytes take 0.75 us of HBM time, less than one warp's chain
// through it (scores in, exponentials, terms, weights out: 1,100 cycles) and
// less than one dependent read, so
//   - two CTAs an SM (three stages of 32 KiB each) where 128 registers do;
//   - table entries are read four tiles ahead, through shared memory;
//   - the code is kept small (rolled loops, waits and divisions out of line):
//     the roles run different code side by side and missed the instruction
//     cache a quarter of the time at 100 KB, 2 % at 65 KB;
//   - whole warps wait, so that none runs on split.
// Measured (back to back, 8 KV heads, head dim 128, block 16; 6,787 GB/s is a
// copy): 8 sequences of 32k to 128k tokens 172 us at 4 query heads a KV head
// (1.15 GB, 0.99 of the copy), 256 sequences of 16 to 8,192 tokens 88 us at 8
// (0.52 GB, 0.87), 16 query columns 197 and 132 us; 512 tokens each of 256
// sequences 49 us, of 257 (no lengths in shared memory) 51.  The first form
// took 307 and 151 us, one CTA an SM with table entries ahead 245 and 145.
//
// Per 128-token tile, inside a CTA:
//   producers block-table entries (a lane per page), one box of K and one of V
//             per page and KV head -- B D contiguous bytes -- into the ring of
//             stages, and the pages' scales by cp.async beside them;
//   MMA       one warp, event loop: scores as soon as K is in, up to three
//             tiles ahead; P.V as soon as the weights are;
//   softmax   four warps a group, thread <-> token (TMEM lane);
//   queries   two warps take the (sequence, head) segments in turn, split their
//             rows into h and l and write them in the MMA's layout, ahead of
//             the tiles.
// Up to 8 query columns (per tile): 8 warps, two CTAs an SM.  16: two groups of
// softmax warps, eight columns each, and four producers, one CTA an SM.
// At head dim 64 a tile holds two adjacent KV heads (HP = 2) where their number
// is even and the group small enough, so that its bytes are those of head dim 128.
#include "decode_fp8.cuh"
#include "decode_split.cuh"
#include "fp8.cuh"
#include "sm100.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

namespace pk {
namespace {

using namespace sm100;

constexpr int kTables = 5;                                   // ring of their entries, above kAhead
constexpr int kAhead = 4;                                    // tiles whose table entries are on their way
constexpr int kScores = 3;                                   // score buffers: two tiles ahead of the weights
constexpr int kQRing = 6;                                    // query scales kept, by segment
constexpr uint64_t kWaitLimitNs = 1000000000ull;             // 1 s: far beyond any legal wait
constexpr float kLevel2 = 1.f / 32;                          // what the second term of a query stands for
constexpr float kHeadroom = 15.f;                            // u <= 2^15: e5m2 holds 57344
constexpr float kNoReference = 3.0e38f;                      // minus the reference of a segment's start
constexpr float kStart = 7.f;                                // the largest u when the reference moves: 2^7
// The denominator adds (u * 2^60) * (2^-60 / vs).  Accepted scales span 2^128, so at
// equal scores u can be 2^-128 where 1 / vs makes it a whole share, and 2^x is 0
// below 2^-126.  With 2^60 only a u below 2^-186 is lost, a share of at most 2^-122
// where the token of the largest u alone adds 2^-57; both factors are normal numbers.
// (Added to the exponent after the reference is taken off: scores of 2^30 would
// swallow it.)  Costs two packed instructions a pair of columns, 1 to 2 % at 16
// columns; a second case for small scales, behind a vote, cost 3 %.
constexpr float kLift = 60.f, kUnlift = 0x1p-60f;

constexpr uint32_t kLayoutSw64 = 4;

// Instruction descriptor for kind::f8f6f4: fp32 accumulator, A of e4m3, B of e4m3 or e5m2.
__host__ __device__ constexpr uint32_t idesc_fp8(uint32_t m, uint32_t n, uint32_t a_mn_major, uint32_t b_mn_major,
                                                 bool b_e5m2) {
    return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | (a_mn_major << 15) | (b_mn_major << 16) | ((n >> 3) << 17) |
           ((m >> 4) << 24);
}

SM100_DEV void mma_fp8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// True in one lane of the (converged) warp.
SM100_DEV bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

SM100_DEV void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// One arrival on `bar` when this thread's cp.async so far have landed.
SM100_DEV void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
SM100_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most N of this thread's groups are on their way.
template <int N>
SM100_DEV void cp_async_wait_group() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
SM100_DEV void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// mbar_wait with its loop out of line: the kernel's warps run different code
// side by side, so its size is instruction-cache traffic.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int *abort, uint64_t limit_ns) {
    return mbar_wait(bar, parity, abort, limit_ns);
}
SM100_DEV bool wait_for(uint32_t bar, uint32_t parity, volatile int *abort, uint64_t limit_ns) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort, limit_ns);
}

template <int kThreads, int kStages, int kLenCache, int kHeadsPerTile, int kProducers>
struct MiscT {
    uint64_t full[kStages];       // K rows of a stage landed
    uint64_t vfull[kStages];      // V rows of a stage landed
    uint64_t sfull[kStages];      // its pages' scales landed
    uint64_t empty[kStages];
    uint64_t qfull[kQRing];       // a segment's queries written (by buffer)
    uint64_t qempty[kQRing];
    uint64_t s_full[kScores];     // scores of a tile complete
    uint64_t p_full[2];
    uint64_t o_full[2];       // P.V of a tile complete (per tile parity)
    uint64_t o_free[2];       // a segment's O buffer has been read out
    uint64_t drain;
    int64_t scan[kThreads / 32 + 1];
    int64_t scan_w[kThreads / 32 + 1];
    int64_t bnd[2];
    int64_t rem0;
    int32_t s0;
    int32_t first_cta;
    uint32_t tmem_base;
    int abort;
    int never;
    int2 held[kStages];            // (tokens, a bit for each page that was read) of a stage's tile
    int4 meta[kStages];            // (sequence, KV head group, tile, tiles in segment) of a stage's tile
    int4 qmeta[kStages];           // (first query row, query tokens, first query position, 0) of it
    float scales[kStages][16][2][kHeadsPerTile];   // [page][K, V][head]
    float qscale[kQRing][kNPad];   // by segment: what the stored query values of a column stand for
    int table[kProducers][kTables][16];  // table entries of the tiles ahead, a ring a producer
    float red[4][kNPad];
    float lsum[2][4][kNPad];       // a segment's denominators by warp (segment parity)
    float mref[2][kNPad];          // its references
    int lens[kLenCache];          // the raw sequence lengths, when there are at most kLenCache
};

// N consecutive columns of this thread's TMEM lane, on their way: r may be used
// after tmem_wait_ld(r), which takes it as an operand to say so.
template <int N>
SM100_DEV void tmem_ld_start(uint32_t taddr, uint32_t *r) {
    static_assert(N == 8 || N == 16, "columns");
    if constexpr (N == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr)
                     : "memory");
    } else {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                     "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                       "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                     : "r"(taddr)
                     : "memory");
    }
}
template <int N>
SM100_DEV void tmem_wait_ld(uint32_t (&r)[N]) {
    static_assert(N % 8 == 0, "columns");
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                       "+r"(r[i + 6]), "+r"(r[i + 7])
                     ::"memory");
}

// The three terms of two weights u <= 2^15, two e5m2 bytes each.  u is first
// rounded to fp16 (11 bits), in which the remainders after each term are exact:
// each takes off three bits and leaves half a step with its sign, so nothing is
// left after the third but below e5m2's smallest steps of 2^-16.
SM100_DEV void split_weights(float u0, float u1, uint32_t &h1, uint32_t &h2, uint32_t &h3) {
    asm("{\n\t.reg .b32 u, b, r;\n\t.reg .b16 a;\n\t"
        "cvt.rn.f16x2.f32 u, %4, %3;\n\t"
        "cvt.rn.satfinite.e5m2x2.f16x2 a, u;\n\t"
        "cvt.u32.u16 %0, a;\n\t"
        "cvt.rn.f16x2.e5m2x2 b, a;\n\t"
        "sub.rn.f16x2 r, u, b;\n\t"
        "cvt.rn.satfinite.e5m2x2.f16x2 a, r;\n\t"
        "cvt.u32.u16 %1, a;\n\t"
        "cvt.rn.f16x2.e5m2x2 b, a;\n\t"
        "sub.rn.f16x2 r, r, b;\n\t"
        "cvt.rn.satfinite.e5m2x2.f16x2 a, r;\n\t"
        "cvt.u32.u16 %2, a;\n\t}"
        : "=r"(h1), "=r"(h2), "=r"(h3)
        : "f"(u0), "f"(u1));
}

// The two terms of two query values below 256, which fp16 holds exactly down
// to 2^-14 (and to 2^-25 below): h, and 32 times what is left.
SM100_DEV void split_query(float q0, float q1, uint32_t &h, uint32_t &l) {
    asm("{\n\t.reg .b32 u, b;\n\t.reg .b16 a;\n\t"
        "cvt.rn.f16x2.f32 u, %3, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 a, u;\n\t"
        "cvt.u32.u16 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 b, a;\n\t"
        "sub.rn.f16x2 u, u, b;\n\t"
        "mul.rn.f16x2 u, u, %4;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 a, u;\n\t"
        "cvt.u32.u16 %1, a;\n\t}"
        : "=r"(h), "=r"(l) : "f"(q0), "f"(q1), "r"(0x50005000u));
}

// Nearly 1 / v for a scale (relative error 2^-23).
SM100_DEV float fast_rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The weights of the cut (see decode_tc.cu): a full tile 272; a segment (its
// read-out, first reference and queries) by sweeps over 256 sequences of 16 to
// 8,192 tokens.  Head dim 128, 16 columns: 132 us at 780, 130 at 500 to 680, 134
// at 300; 8 columns: 88 at 80 to 160, 89 at 240.  Head pairs, 16 columns: 74 at
// 780, 69 at 300 to 500; 8 columns: 54.7 at 80, 56 at 160.  (Swept before the
// denominators reached over the whole scale range; with these weights 132, 88, 70
// and 56 us now.)
constexpr int64_t kTileCost = 400;
constexpr int kTokCost = 1;
template <int NUSED, int HP>
constexpr int64_t seg_cost() { return NUSED > 8 ? (HP == 2 ? 400 : 600) : (HP == 2 ? 10 : 20) * NUSED; }

// What follows from (head dim, query columns per KV head, KV heads per tile).
template <int D, int NC, int HP>
struct Shape {
    static_assert(D == 64 || D == 128, "head_dim");
    static_assert(NC >= 1 && NC <= kNPad, "query columns");
    static_assert(HP == 1 || (HP == 2 && D == 64 && NC <= 8), "head pairs: head dim 64, at most 8 columns each");
    static constexpr int CW = HP == 2 ? 8 : kNPad;          // columns per head in slots and lsum
    static constexpr int HL = NC <= 8 ? 8 : 16;             // rows of h (and of l) in a query buffer
    static constexpr int NS = 2 * HL;                       // MMA N of S^T per head: h columns, then l columns
    static constexpr int PW = HP * NC > 8 ? 16 : 8;         // columns of one term of u
    static constexpr int PC = PW / HP;                      // of them, one head's
    static constexpr int NP = PW == 8 ? 32 : 48;            // MMA N of O^T: three terms (and padding to 16)
    static constexpr uint32_t HeadBytes = kTile * D;        // one head's rows of a tile
    static constexpr uint32_t StageBytes = 2 * HP * HeadBytes;
    static constexpr uint32_t VOff = HP * HeadBytes;
    static constexpr uint32_t QHeadBytes = NS * D;
    static constexpr uint32_t QBufBytes = HP * QHeadBytes;
    // Two CTAs an SM where their shared memory and 128 registers a thread do:
    // one CTA's warps wait for one another most of the time (a tile is a chain
    // of copies, scores, weights and products), and a second one fills that.
    static constexpr int CtasPerSm = NP == 32 ? 2 : 1;
    static constexpr int Stages = CtasPerSm == 2 ? 3 * 32768 / StageBytes : 6;
    static constexpr int LenCache = CtasPerSm == 2 ? 256 : 2048;
    static constexpr int QBufs = 2;
    // The one CTA of an SM splits its work over more warps instead: two groups
    // of softmax warps, eight columns each, and four producers (the even and
    // the odd pages of K and of V: issuing a box takes a warp 70 to 100 cycles).
    static constexpr int Groups = CtasPerSm == 2 ? 1 : 2;
    static constexpr int GPairs = Groups == 2 ? 4 : (HP == 2 ? NC + NC % 2 : (NC + 1) / 2);   // pairs of columns of a group
    static constexpr int QueryWarp = 2 + 4 * Groups;        // the first of two
    static constexpr int Producers = CtasPerSm == 2 ? 1 : 4;   // warp 0 and those behind the query warps
    static constexpr int Threads = 32 * (QueryWarp + 1 + Producers);
    static constexpr uint32_t PBytes = kTile * NP;
    static constexpr uint32_t SCols = HP * NS;
    static constexpr uint32_t tS = 0, tO = kScores * SCols;
    static constexpr uint32_t TmemCols = tO + 2 * NP <= 128 ? 128 : 256;
    using Misc = MiscT<Threads, Stages, LenCache, HP, Producers>;
    static constexpr size_t SmemBytes = 1024 + Stages * StageBytes + QBufs * QBufBytes + 2 * PBytes + sizeof(Misc);
    // The queries run at most QBufs segments ahead of the scores, and those kScores - 1 tiles of the weights.
    static_assert(QBufs >= 2 && QBufs + kScores - 1 < kQRing, "query scales outlive their buffers");
    static_assert(tO + 2 * NP <= 256, "TMEM");
    static_assert(SmemBytes <= 227 * 1024, "shared memory");
    static_assert(CtasPerSm * (SmemBytes + 1024) <= 228 * 1024, "CTAs per SM");
    static_assert(CtasPerSm * TmemCols <= 512, "TMEM");
};

template <int D, int NC, bool MQ, int HP>
__global__ void __launch_bounds__(Shape<D, NC, HP>::Threads, Shape<D, NC, HP>::CtasPerSm)
decode_fp8_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const DecodeFp8Params p) {
    using C_ = Shape<D, NC, HP>;
    using Misc = typename C_::Misc;
    constexpr int kThreads = C_::Threads, kStages = C_::Stages, kLenCache = C_::LenCache, kGroups = C_::Groups;
    constexpr int kProducers = C_::Producers, kPerOperand = kProducers == 4 ? 2 : 1;
    constexpr int CW = C_::CW, HL = C_::HL, NS = C_::NS, PW = C_::PW, PC = C_::PC, NP = C_::NP;
    constexpr uint32_t kLayout = D == 128 ? kLayoutSw128 : kLayoutSw64;
    constexpr uint32_t kAtom = 8 * D;                 // eight rows: the swizzle's atom
    constexpr uint32_t kIdescQK = idesc_fp8(kTile, NS, 0, 0, false);   // A = K (K-major), B = Q (K-major)
    constexpr uint32_t kIdescPV = idesc_fp8(128, NP, 1, 1, true);      // A = V^T (MN-major), B = P^T (MN-major)
    constexpr int64_t kSegCost = seg_cost<HP * NC, HP>();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    uint8_t *stage_ptr = smem;
    uint8_t *q_ptr = smem + kStages * C_::StageBytes;
    uint8_t *p_ptr = q_ptr + C_::QBufs * C_::QBufBytes;
    Misc *misc = reinterpret_cast<Misc *>(p_ptr + 2 * C_::PBytes);
    const uint32_t stage_addr = smem_u32(stage_ptr);
    const uint32_t q_addr = smem_u32(q_ptr);
    const uint32_t p_addr = smem_u32(p_ptr);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x, C = gridDim.x;
    // Hkv counts the tile's KV head groups (segments per sequence).
    const int N = p.num_seqs, Hkv = p.num_kv_heads / HP, H = p.num_heads, B = p.block_size;
    const int lgB = __ffs(B) - 1;
    const int cap = p.max_seq_len;                    // at most max_blocks_per_seq * B (checked on the host)
    const int Gq = H / p.num_kv_heads, lgG = __ffs(Gq) - 1;     // query heads per KV head (a power of two)
    Slot *slots = static_cast<Slot *>(p.tc_slots);
    const uint64_t lim = p.wait_limit_ns ? p.wait_limit_ns : kWaitLimitNs;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&misc->full[i]), kPerOperand);
            mbar_init(smem_u32(&misc->vfull[i]), kPerOperand);
            mbar_init(smem_u32(&misc->sfull[i]), 32 * kProducers);   // the lanes of every producer
            mbar_init(smem_u32(&misc->empty[i]), 1);
        }
        for (int i = 0; i < C_::QBufs; ++i) {
            mbar_init(smem_u32(&misc->qfull[i]), 1);
            mbar_init(smem_u32(&misc->qempty[i]), 1);
        }
        for (int i = 0; i < kScores; ++i) mbar_init(smem_u32(&misc->s_full[i]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&misc->p_full[i]), 4 * kGroups);
            mbar_init(smem_u32(&misc->o_full[i]), 1);
            mbar_init(smem_u32(&misc->o_free[i]), 4 * kGroups);
        }
        mbar_init(smem_u32(&misc->drain), 1);
        misc->abort = 0;
        misc->never = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&misc->tmem_base), C_::TmemCols);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    // ---- this CTA's range of the flattened tile space, as in decode_tc_kernel:
    // planned before the wait on the previous grid, checked after it.
    const bool cached = N <= kLenCache;
    const LenSrc lens{cached ? misc->lens : nullptr, p.seq_lens, cap};
    int64_t T = 0;
    int odd = 0;
    auto first_tile = [&]() -> Walk {
        Walk w{};
        w.nh = Hkv;
        w.ns = N;
        w.s = misc->s0;
        w.load(lens);
        w.h = static_cast<int>(quotient(misc->rem0, w.nt));
        w.t = static_cast<int>(misc->rem0 - static_cast<int64_t>(w.h) * w.nt);
        return w;
    };
    auto wait_prev = [&]() {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (threadIdx.x == 0 && slots) slots[2 * c].flag = 0;
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    };
    bool ahead = cached;
    if (cached) {
        const int32_t *first_read = p.lens_ahead ? p.lens_ahead : p.seq_lens;
#pragma unroll 1
        for (int s = threadIdx.x; s < N; s += kThreads) misc->lens[s] = ld_cg(first_read + s);
        __syncthreads();
    } else {
        wait_prev();
    }
    for (;;) {
        T = plan_range<kThreads>(lens, misc, N, Hkv, c, C, kSegCost, kTileCost, kTokCost, &odd);
        if (!ahead) break;
        ahead = false;
        wait_prev();
        int changed = 0;
#pragma unroll 1
        for (int s = threadIdx.x; s < N; s += kThreads) changed |= ld_cg(p.seq_lens + s) != misc->lens[s];
        if (!__syncthreads_or(changed)) break;
#pragma unroll 1
        for (int s = threadIdx.x; s < N; s += kThreads) misc->lens[s] = ld_cg(p.seq_lens + s);
        __syncthreads();
    }
    const int64_t beg = misc->bnd[0], end = misc->bnd[1];
    if (threadIdx.x == 0 && slots) slots[2 * c].range_beg = beg;
    const int n_tiles = static_cast<int>(end - beg);
    // Lengths outside [0, cap] are reported, and empty sequences get zeros,
    // by CTA s % C.
    if (odd || MQ) {
#pragma unroll 1
        for (int s = c; s < N; s += C) {
            const int raw = lens.raw(s);
            if ((raw < 0 || raw > cap) && threadIdx.x == 0) set_error(p.err, PK_DEVERR_SEQ_LEN);
            const int L = lens(s);
            if constexpr (MQ) {
                // A sequence has at most L query tokens (they are its newest tokens).
                const int r0 = p.cu_q_lens[s], r1 = p.cu_q_lens[s + 1];
                const bool bad = r0 < 0 || r1 < r0 || r1 > p.total_q || r1 - r0 > p.q_len;
                if ((bad || r1 - r0 > L) && threadIdx.x == 0) set_error(p.err, PK_DEVERR_SEQ_LEN);
                if (L != 0 || bad) continue;
#pragma unroll 1
                for (int64_t i = threadIdx.x; i < static_cast<int64_t>(r1 - r0) * H * D; i += kThreads)
                    store_out(p, static_cast<size_t>(r0) * H * D + i, 0.f);
            } else {
                if (L != 0) continue;
#pragma unroll 1
                for (int i = threadIdx.x; i < H * D; i += kThreads) store_out(p, static_cast<size_t>(s) * H * D + i, 0.f);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc->tmem_base;

    Walk w0{};
    w0.nh = Hkv;
    w0.ns = N;
    if (n_tiles > 0) w0 = first_tile();

    // The sequence's query rows (first, number): its newest tokens.  Rows that
    // are not within the queries given, or more than the columns hold, are
    // none (reported above).
    auto query_rows = [&](int s) -> int2 {
        if constexpr (MQ) {
            const int r0 = p.cu_q_lens[s], r1 = p.cu_q_lens[s + 1];
            if (r0 < 0 || r1 < r0 || r1 > p.total_q || r1 - r0 > p.q_len) return make_int2(0, 0);
            return make_int2(r0, r1 - r0);
        } else {
            return make_int2(s, 1);
        }
    };

    if (warp == 0 || warp >= C_::QueryWarp + 2) {
        // ================= producer =================
        // One of K and V, or four: K and V of the even pages, K and V of the odd ones.
        const int pi = warp == 0 ? 0 : warp - (C_::QueryWarp + 1);
        const bool do_k = (pi & 1) == 0, do_v = kProducers == 1 || (pi & 1);
        const bool my_page = kProducers == 1 || (lane & 1) == (pi >> 1);
        Walk w = w0;
        int2 qr = make_int2(0, 0);
        int qr_of = -1;
        const int MB = p.max_blocks_per_seq;
        int issued = 0;
        bool stalled = false;
        // Table entries (a lane per page) are read kAhead tiles before their tile:
        // a tile's bytes take less time than one read does, so one tile ahead would
        // bound the copies by that read's latency.  They go through shared memory
        // (registers that move up would wait for the reads on their way), each
        // lane reading what it copied itself.
        int (*ring)[16] = misc->table[pi];
        Walk wf = w;
        auto fetch_tile = [&](int i) {
            if (i < n_tiles) {
                const int fp = wf.t * (kTile >> lgB);
                if (lane < (kTile >> lgB) && fp + lane < MB)
                    cp_async4(smem_u32(&ring[i % kTables][lane]), p.block_tables + static_cast<size_t>(wf.s) * MB + fp + lane);
                wf.next(lens);
            }
            cp_async_commit();
        };
#pragma unroll 1
        for (int i = 0; i < kAhead; ++i) fetch_tile(i);
#pragma unroll 1
        for (int i = 0; i < n_tiles; ++i) {
            // Self-test: CTA 0 stops issuing copies, so the barriers of this tile
            // never complete.
            if (p.stall_tile > 0 && c == 0 && i == p.stall_tile) {
                stalled = true;
                break;
            }
            const int st = i % kStages;
            fetch_tile(i + kAhead);
            cp_async_wait_group<kAhead>();
            const int phys = lane < 16 ? ring[i % kTables][lane] : -1;
            // What the tile needs is worked out before the wait for its stage.
            const int vlen = min(kTile, w.L - w.t * kTile);
            const int pages = (vlen + B - 1) >> lgB;
            bool ok = false;
            if (lane < pages) {
                ok = phys >= 0 && phys < p.num_blocks;
                if (!ok && pi == 0) set_error(p.err, PK_DEVERR_BLOCK_ID);
            }
            const uint32_t oks = __ballot_sync(0xffffffffu, ok);
            ok = ok && my_page;
            const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, ok))) * (HP * D) << lgB;
            const uint32_t full = smem_u32(&misc->full[st]);
            const uint32_t vfull = smem_u32(&misc->vfull[st]);
            const uint32_t sbase = stage_addr + st * C_::StageBytes;
            if constexpr (MQ) {
                if (w.s != qr_of) qr = query_rows(qr_of = w.s);
            }
            const int piece = phys * p.num_kv_heads + w.h * HP;
            // Every lane waits (a lane that waited alone would leave the warp split
            // for what follows); one decision for the whole warp.
            if (!__all_sync(0xffffffffu, wait_for(smem_u32(&misc->empty[st]), ((i / kStages) & 1) ^ 1, &misc->abort, lim))) {
                misc->abort = 1;
                set_error(p.err, PK_DEVERR_TIMEOUT);
                break;
            }
            if (lane == 0 && do_v) mbar_arrive_expect_tx(vfull, bytes);
            if (lane == 0 && do_k) {
                if (pi == 0) {
                    misc->meta[st] = make_int4(w.s, w.h, w.t, w.nt);
                    misc->held[st] = make_int2(vlen, static_cast<int>(oks));
                    if constexpr (MQ) misc->qmeta[st] = make_int4(qr.x, qr.y, w.L - qr.y, 0);
                }
                mbar_arrive_expect_tx(full, bytes);
            }
            __syncwarp();
            if (ok) {
                // The (block, head) piece: B rows of D bytes, at the page's place in each head's tile.
                const uint32_t at = sbase + (static_cast<uint32_t>(lane) << lgB) * D;
                if (do_k) {
#pragma unroll
                    for (int hd = 0; hd < HP; ++hd)
                        tma_load_3d(at + hd * C_::HeadBytes, &tm_k, full, 0, 0, piece + hd);
                }
                if (do_v) {
#pragma unroll
                    for (int hd = 0; hd < HP; ++hd)
                        tma_load_3d(at + C_::VOff + hd * C_::HeadBytes, &tm_v, vfull, 0, 0, piece + hd);
                }
#pragma unroll
                for (int hd = 0; hd < HP; ++hd) {
                    if (do_k) cp_async4(smem_u32(&misc->scales[st][lane][0][hd]), p.k_scales + piece + hd);
                    if (do_v) cp_async4(smem_u32(&misc->scales[st][lane][1][hd]), p.v_scales + piece + hd);
                }
            }
            cp_async_arrive(smem_u32(&misc->sfull[st]));
            ++issued;
            w.next(lens);
        }
        cp_async_wait_all();
        // On abort (or a self-test's stall), let this warp's copies land before the
        // CTA can exit.
        if ((misc->abort || stalled) && lane == 0) {
            for (int i = max(0, issued - kStages); i < issued; ++i) {
                if (do_k) wait_for(smem_u32(&misc->full[i % kStages]), (i / kStages) & 1, &misc->never, lim);
                if (do_v) wait_for(smem_u32(&misc->vfull[i % kStages]), (i / kStages) & 1, &misc->never, lim);
            }
        }
    } else if (warp == 1) {
        // ================= MMA issuer =================
        // The whole warp runs the loop and one lane issues: what an MMA takes then
        // stays in uniform registers (one lane alone took 100 cycles an MMA, and
        // this warp bounded the tile).
        const bool leader = elect_one();
        const uint64_t k_desc = smem_desc(stage_addr, 16, kAtom, kLayout);
        // Head dim 64: the second 64 rows of O^T come from the pair's second head
        // (HP == 2) or are not used.
        const uint64_t v_desc = smem_desc(stage_addr + C_::VOff, HP == 2 ? C_::HeadBytes : kAtom, kAtom, kLayout);
        const uint64_t q_desc = smem_desc(q_addr, 16, kAtom, kLayout);
        const uint64_t p_desc = smem_desc(p_addr, 8 * NP, 128, kLayoutNone);
        int pv_seg = -1, qk_seg = -1;
        auto pv = [&](int j, int st, bool first, int sg) {
            const int pb = j & 1;
            tc_fence_after();
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < kTile / 32; ++kk) {
                    // Tokens 32 kk .. 32 kk + 31: four 8-row atoms of V.
                    mma_fp8(tmem + C_::tO + (sg & 1) * NP, v_desc + ((st * C_::StageBytes + kk * 4 * kAtom) >> 4),
                             p_desc + ((pb * C_::PBytes + kk * 32 * NP) >> 4), kIdescPV, (first && kk == 0) ? 0u : 1u);
                }
                mma_commit(smem_u32(&misc->o_full[pb]));
                mma_commit(smem_u32(&misc->empty[st]));
            }
            __syncwarp();
        };
        auto qk = [&](int sb, int st, int sg, bool last) {
            const uint32_t qb = sg % C_::QBufs;
            tc_fence_after();
            if (leader) {
#pragma unroll
                for (int hd = 0; hd < HP; ++hd) {
#pragma unroll
                    for (int kk = 0; kk < D / 32; ++kk) {
                        mma_fp8(tmem + C_::tS + sb * C_::SCols + hd * NS,
                                 k_desc + ((st * C_::StageBytes + hd * C_::HeadBytes + kk * 32) >> 4),
                                 q_desc + ((qb * C_::QBufBytes + hd * C_::QHeadBytes + kk * 32) >> 4), kIdescQK, kk > 0 ? 1u : 0u);
                    }
                }
                mma_commit(smem_u32(&misc->s_full[sb]));
                if (last) mma_commit(smem_u32(&misc->qempty[qb]));
            }
            __syncwarp();
        };
        auto done = [&](uint64_t &bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_test_wait(smem_u32(&bar), parity));
        };
        // Event loop, as in decode_tc_kernel; the scores of a segment's first tile
        // also wait for its queries.
        int nq = 0, np = 0;
        int st_q = 0, st_p = 0, sb = 0;                  // stages of tiles nq and np, score buffer of nq
        uint32_t ph_q = 0, ph_p = 0;                     // and the parities of their rounds
        uint64_t t_idle = 0;
        uint32_t spins = 0;
#pragma unroll 1
        while (np < n_tiles) {
            bool prog = false;
            if (np < nq && done(misc->p_full[np & 1], (np >> 1) & 1) && done(misc->vfull[st_p], ph_p)) {
                const bool first = np == 0 || misc->meta[st_p].z == 0;
                const int sg = pv_seg + (first ? 1 : 0);
                // A new segment's O buffer must have been read out (segment sg - 2).
                if (!first || done(misc->o_free[sg & 1], ((sg >> 1) & 1) ^ 1)) {
                    pv(np, st_p, first, sg);
                    pv_seg = sg;
                    ++np;
                    if (++st_p == kStages) {
                        st_p = 0;
                        ph_p ^= 1;
                    }
                    prog = true;
                }
            }
            if (nq < n_tiles && nq < np + kScores && done(misc->full[st_q], ph_q)) {
                const int4 mt = misc->meta[st_q];
                const bool first = nq == 0 || mt.z == 0;
                const int sg = qk_seg + (first ? 1 : 0);
                if (!first || done(misc->qfull[sg % C_::QBufs], (sg / C_::QBufs) & 1)) {
                    qk(sb, st_q, sg, nq == n_tiles - 1 || mt.z == mt.w - 1);
                    qk_seg = sg;
                    ++nq;
                    if (++st_q == kStages) {
                        st_q = 0;
                        ph_q ^= 1;
                    }
                    if (++sb == kScores) sb = 0;
                    prog = true;
                }
            }
            if (prog) {
                spins = 0;
            } else if ((++spins & 255u) == 0) {
                const uint64_t now = globaltimer_ns();
                if (spins == 256) t_idle = now;
                else if (__any_sync(0xffffffffu, misc->abort || now - t_idle > lim)) {
                    misc->abort = 1;
                    set_error(p.err, PK_DEVERR_TIMEOUT);
                    break;
                }
            }
        }
        // Let every issued MMA finish before the CTA can release TMEM.
        if (leader) mma_commit(smem_u32(&misc->drain));
        __syncwarp();
        wait_for(smem_u32(&misc->drain), 0, &misc->never, lim);
        __syncwarp();
    } else if (warp >= C_::QueryWarp) {
        // ================= queries =================
        // One warp takes the even segments, the other the odd ones.
        // A row is D / 8 lanes of 8 elements; a warp does kRows rows at once.
        constexpr int kLanes = D / 8, kRows = 32 / kLanes, kIters = (HP * NC + kRows - 1) / kRows;
        const int part = lane % kLanes, sub = lane / kLanes;
        Walk w = w0;
        int i = 0;
#pragma unroll 1
        for (int sg = 0; i < n_tiles; ++sg) {
            const int left = min(w.nt - w.t, n_tiles - i);
            if ((sg & 1) == warp - C_::QueryWarp) {
                const int2 qr = query_rows(w.s);
                // Row x of the buffer: query column x % NC of head x / NC of the pair;
                // column cq: query token cq / G, query head cq % G.  For one token
                // (NC == G) the rows are consecutive.
                uint4 raw[kIters];
                const uint16_t *rows = p.q + (static_cast<size_t>(qr.x) * H + w.h * HP * Gq) * D + part * 8;
#pragma unroll
                for (int y = 0; y < kIters; ++y) {
                    const int x = y * kRows + sub, cq = x % NC;
                    raw[y] = make_uint4(0, 0, 0, 0);
                    if (x < HP * NC && (cq >> lgG) < qr.y) {
                        const int at = MQ ? ((cq >> lgG) * H + x / NC * Gq + (cq & (Gq - 1))) * D : x * D;
                        raw[y] = ldg_stream(rows + at);      // volatile: stays ahead of the wait
                    }
                }
                const int qb = sg % C_::QBufs;
                if (!__all_sync(0xffffffffu, wait_for(smem_u32(&misc->qempty[qb]), ((sg / C_::QBufs) & 1) ^ 1, &misc->abort, lim))) {
                    misc->abort = 1;
                    set_error(p.err, PK_DEVERR_TIMEOUT);
                    break;
                }
                uint8_t *buf = q_ptr + qb * C_::QBufBytes;
                // Not unrolled (the code of every warp's part shares the instruction
                // cache): the rows move up in their registers instead.
#pragma unroll 1
                for (int y = 0; y < kIters; ++y) {
                    const int x = y * kRows + sub, hd = x / NC, cq = x % NC;
                    // The row's largest magnitude: bf16 bits without the sign order as integers.
                    uint32_t top = 0;
                    const uint32_t words[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
                    for (int e = 0; e + 1 < kIters; ++e) raw[e] = raw[e + 1];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t v = words[e] & 0x7fff7fffu;
                        top = max(top, max(v & 0xffffu, v >> 16));
                    }
#pragma unroll
                    for (int o = kLanes / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    // 2^k brings it to [128, 256); |k| <= 120 keeps 2^k and 2^-k normal.
                    const bool finite = top < 0x7f80u;
                    const int k = finite ? min(7 - (max(static_cast<int>(top >> 7), 1) - 127), 120) : 0;
                    const float up = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
                    if (part == 0 && x < HP * NC)
                        misc->qscale[sg % kQRing][hd * CW + cq] =
                            finite ? __uint_as_float(static_cast<uint32_t>(127 - k) << 23) : __int_as_float(0x7fffffff);
                    uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t h2, l2;
                        split_query(bf16_lo(words[e]) * up, bf16_hi(words[e]) * up, h2, l2);
                        hi[e >> 1] |= h2 << (16 * (e & 1));
                        lo[e >> 1] |= l2 << (16 * (e & 1));
                    }
                    // K-major rows of D bytes, swizzled as TMA swizzles K: the 16-byte
                    // piece of a row is exchanged by the row (128 bytes: row % 8; 64: row / 2 % 4).
                    const int r = cq, piece = (part >> 1) ^ (D == 128 ? r & 7 : (r >> 1) & 3);
                    uint8_t *dst = buf + hd * C_::QHeadBytes + r * D + piece * 16 + (part & 1) * 8;
                    if (x < HP * NC) {
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(hi[0], hi[1]);
                        *reinterpret_cast<uint2 *>(dst + HL * D) = make_uint2(lo[0], lo[1]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&misc->qfull[qb]));
            }
            i += left;
            w.t += left - 1;
            w.next(lens);
        }
    } else {
        // ================= softmax: thread <-> tile row =================
        // Group g has columns 8 g to 8 g + 7 (two groups), or all of them.
        const int grp = kGroups == 2 ? (warp - 2) >> 2 : 0;
        const uint32_t bar = 1 + grp;                   // its named barrier
        const int quad = warp & 3;
        const int row = quad * 32 + lane;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        // Columns: HP == 1, query column j; HP == 2, 0-7 the pair's first head's and 8-15 the second's.
        // They are kept in pairs, for the packed fp32 instructions: pair x holds
        // columns col(x) and col(x) + 1 of head hd_of(x) (a single column's
        // partner is unused), which are pc(x) and pc(x) + 1 of a term of u and
        // of O^T.  With two groups col(x) = pc(x), and the head is the group's.
        constexpr int kPairs = C_::GPairs, kPerHead = kGroups == 2 ? 4 : (NC + 1) / 2;
        auto local = [](int x) { return x / kPerHead * PC + 2 * (x % kPerHead); };     // pc(x) less 8 grp
        auto col = [&](int x) { return kGroups == 2 ? 8 * grp + 2 * x : x / kPerHead * 8 + 2 * (x % kPerHead); };
        auto hd_of = [](int x) { return kGroups == 1 ? x / kPerHead : 0; };   // index into this group's heads
        constexpr int kHeads = HP == 2 && kGroups == 1 ? 2 : 1;               // heads a group has
        const int hd0 = HP == 2 && kGroups == 2 ? grp : 0;                    // its first head
        constexpr int kCols = kGroups == 2 ? 8 : HP * NC;                     // its columns
        constexpr int kGW = kGroups == 2 ? 8 : PW;                            // and with padding, in a term of u
        uint64_t qf[kPairs], l_run[kPairs];
        uint64_t neg_m[kPairs];                          // minus the references
#pragma unroll
        for (int x = 0; x < kPairs; ++x) qf[x] = l_run[x] = neg_m[x] = 0;
        const int hr = HP == 2 ? row >> 6 : 0;          // head of the pair of this O^T row
        const int dd = HP == 2 ? (row & 63) : row;      // its element
        const bool row_ok = HP == 2 || row < D;
        int seg = -1, seg_t0 = 0, seg_i0 = 0;
        bool pending = false;            // a finished segment awaits its read-out
        int pend_seg = 0, pend_s = 0, pend_h = 0, pend_i = 0, pend_t0 = 0, pend_i0 = 0, pend_q0 = 0, pend_qn = 1;
        bool pend_complete = false, pend_cut_end = false;
        auto finalize = [&]() -> bool {
            // P.V of the segment's last tile (pend_i) complete.
            if (!__all_sync(0xffffffffu, wait_for(smem_u32(&misc->o_full[pend_i & 1]), (pend_i >> 1) & 1,
                                                   &misc->never, lim)))
                return false;
            tc_fence_after();
            // The three terms, smallest first.
            float ov[kGW];
            {
                const uint32_t oaddr = lane_addr + C_::tO + (pend_seg & 1) * NP + 8 * grp;
                float o1[kGW], o2[kGW], o3[kGW];
                tmem_ld<kGW>(oaddr, o1);
                tmem_ld<kGW>(oaddr + PW, o2);
                tmem_ld<kGW>(oaddr + 2 * PW, o3);
#pragma unroll
                for (int j = 0; j < kGW; ++j) ov[j] = (o3[j] + o2[j]) + o1[j];
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&misc->o_free[pend_seg & 1]));
            // This row's columns: of one head, first_col .. first_col + kMine - 1.
            constexpr int kMine = kGroups == 2 ? 8 : NC;
            const int first_col = kGroups == 2 ? 8 * grp : hr * 8;
            if constexpr (kHeads == 2) {
#pragma unroll
                for (int x = 0; x < kMine; ++x) ov[x] = hr ? ov[PC + x] : ov[x];
            }
            // Lane x sums column x's denominator for the warp.
            float l = 0.f;
            if (lane < kMine) {
                const float *ls = &misc->lsum[pend_seg & 1][0][first_col + lane];
                l = ls[0] + ls[kNPad] + ls[2 * kNPad] + ls[3 * kNPad];
            }
            // A cut part goes to slot 0 if the segment is this CTA's first, 1 if not.
            Slot *sl = slots + 2 * c + (pend_i0 == 0 ? 0 : 1);
            const bool mine = row_ok && (HP == 1 || kGroups == 1 || hr == grp);
            if (pend_complete) {
                // Query column cq: token cq / G of the sequence, head cq % G of the KV head.
                const int cq0 = HP == 1 ? first_col : 0;
                const size_t base = (static_cast<size_t>(MQ ? pend_q0 : pend_s) * H + (pend_h * HP + hr) * Gq) * D + dd;
                const int used = MQ ? min(NC, pend_qn << lgG) - cq0 : NC - cq0;     // the rest are padding
                const float inv = l != 0.f ? __fdividef(1.f, l) : 0.f;
#pragma unroll
                for (int x = 0; x < kMine; ++x) {
                    const float o = ov[x] * __shfl_sync(0xffffffffu, inv, x);
                    const int cq = cq0 + x;
                    const size_t at = MQ ? base + static_cast<size_t>(cq >> lgG) * H * D + (cq & (Gq - 1)) * D : base + cq * D;
                    if (mine && x < used) store_out(p, at, o);
                }
            } else {
                if (mine) {
#pragma unroll
                    for (int x = 0; x < kMine; ++x) sl->o[(first_col + x) * 128 + row] = ov[x];
                }
                // The warp with element 0 of the head's rows writes its columns' sums.
                if ((quad == 0 || (HP == 2 && quad == 2)) && (HP == 1 || kGroups == 1 || hr == grp) && lane < kMine) {
                    sl->l[first_col + lane] = l;
                    sl->m[first_col + lane] = misc->mref[pend_seg & 1][first_col + lane];
                }
            }
            if (!pend_complete && row == 0 && grp == 0) {
                sl->s = pend_s;
                sl->h = pend_h;
                sl->start_tile = beg + pend_i0 - pend_t0;
                sl->total_tiles = T;
                // Cut at its start and finished here: this CTA merges it.
                if (pend_i0 == 0) {
                    sl->flag = (pend_t0 > 0 && pend_cut_end) ? 1 : 0;
                    sl->first_cta = misc->first_cta;
                }
            }
            pending = false;
            return true;
        };
        // A finished segment's denominators and references, for finalize (which
        // follows at least one barrier of the group later).
        auto close_segment = [&]() {
            // Sums over the warp: halves of the columns are exchanged until a
            // lane holds one column's (n - 1 + log2(32 / n) shuffles for n
            // columns instead of 5 n).
            constexpr int n = kCols;
            float v[n];
#pragma unroll
            for (int x = 0; x < kPairs; ++x) {
                const float2 lp = unf2(l_run[x]);
                const int at = kGroups == 2 ? 2 * x : hd_of(x) * NC + 2 * (x % kPerHead);
                v[at] = lp.x;
                if constexpr (NC > 1) v[at + 1] = lp.y;
            }
            int off = 16;
#pragma unroll
            for (int m = n; m > 1; m >>= 1, off >>= 1) {
                const bool upper = lane & off;
#pragma unroll
                for (int x = 0; x < m / 2; ++x) {
                    const float keep = upper ? v[x + m / 2] : v[x], give = upper ? v[x] : v[x + m / 2];
                    v[x] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                }
            }
#pragma unroll
            for (; off >= 1; off >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
            if (lane % (32 / n) == 0) {
                const int at = lane / (32 / n);
                misc->lsum[seg & 1][quad][kGroups == 2 ? 8 * grp + at : (HP == 2 ? at / NC * 8 : 0) + at % NC] = v[0];
            }
            if (row == 0) {
#pragma unroll
                for (int x = 0; x < kPairs; ++x) {
                    const float2 m = unf2(neg_m[x]);
                    misc->mref[seg & 1][col(x)] = -m.x;
                    if constexpr (NC > 1) misc->mref[seg & 1][col(x) + 1] = -m.y;
                }
            }
        };
        // Round n_tiles only reads out the last segment.  A warp that gives up leaves
        // with i the first round whose barriers it has not met.
        int i = 0;
#pragma unroll 1
        for (; i <= n_tiles; ++i) {
            int4 mt = make_int4(0, 0, 0, 0);             // (s, h, t, nt), written with the stage
            int4 qm = make_int4(0, 1, 0, 0);             // (first query row, query tokens, first query position)
            bool seg_last = false;
            if (i == n_tiles) named_bar_sync(bar, 128);
            if (i < n_tiles) {
                const int st = i % kStages;
                const int sb = i & 1;
                // Three barriers asked side by side: the scores, the scales, and whether
                // P buffer sb is free (P.V of tile i - 2 is done).
                const bool scores_in = mbar_try_wait(smem_u32(&misc->s_full[i % kScores]), (i / kScores) & 1);
                const bool scales_in = mbar_test_wait(smem_u32(&misc->sfull[st]), (i / kStages) & 1);
                const bool p_free = mbar_test_wait(smem_u32(&misc->o_full[sb]), ((i >> 1) & 1) ^ 1);
                if (!__all_sync(0xffffffffu,
                                (scores_in || wait_slow(smem_u32(&misc->s_full[i % kScores]), (i / kScores) & 1, &misc->never, lim)) &&
                                (scales_in || wait_slow(smem_u32(&misc->sfull[st]), (i / kStages) & 1, &misc->never, lim)))) {
                    misc->abort = 1;
                    set_error(p.err, PK_DEVERR_TIMEOUT);
                    break;
                }
                mt = misc->meta[st];
                if constexpr (MQ) qm = misc->qmeta[st];
                const bool seg_first = (i == 0) || (mt.z == 0);
                seg_last = (i == n_tiles - 1) || (mt.z == mt.w - 1);
                if (seg_first) {
                    ++seg;
                    seg_t0 = mt.z;
                    seg_i0 = i;
#pragma unroll
                    for (int x = 0; x < kPairs; ++x) {
                        neg_m[x] = f2(kNoReference, kNoReference);
                        l_run[x] = 0;
                        const float *qs = &misc->qscale[seg % kQRing][col(x)];
                        qf[x] = f2(qs[0] * p.scale_log2, NC > 1 ? qs[1] * p.scale_log2 : 0.f);
                    }
                }
                tc_fence_after();
                // Scores: h columns plus 1/32 of the l columns (of this group), on their
                // way while the token's scales are looked at.
                uint64_t t2[kPairs];
                constexpr int kWide = kHeads * 16;
                uint32_t sr[kWide];
                const uint32_t saddr = lane_addr + C_::tS + (i % kScores) * C_::SCols;
                __syncwarp();
                if constexpr (kGroups == 2 && HP == 1) {
                    tmem_ld_start<8>(saddr + 8 * grp, sr);
                    tmem_ld_start<8>(saddr + HL + 8 * grp, sr + 8);
                } else {
                    tmem_ld_start<16>(saddr + hd0 * NS, sr);
                    if constexpr (kWide == 32) tmem_ld_start<16>(saddr + 16, sr + 16);
                }
                // The token's scales; one that is out of range hides the token's head.
                const int2 held = misc->held[st];
                const bool in_page = row < held.x && ((held.y >> (row >> lgB)) & 1);
                bool valid[kHeads];
                float ks[kHeads], lv[kHeads], ivs[kHeads];
#pragma unroll
                for (int hd = 0; hd < kHeads; ++hd) {
                    float k1 = misc->scales[st][row >> lgB][0][hd0 + hd], v1 = misc->scales[st][row >> lgB][1][hd0 + hd];
                    valid[hd] = in_page && scale_ok(k1) && scale_ok(v1);
                    if (in_page && !valid[hd]) set_error(p.err, PK_DEVERR_SCALE);
                    if (!valid[hd]) k1 = v1 = 1.f;         // a weight of zero times its scale stays zero
                    ks[hd] = k1;
                    const uint32_t b = __float_as_uint(v1);
                    lv[hd] = static_cast<float>(static_cast<int>(b >> 23) - 127);
                    if (b & 0x7fffffu) lv[hd] = __log2f(v1);
                    ivs[hd] = fast_rcp(v1) * kUnlift;
                }
                tmem_wait_ld(sr);
#pragma unroll
                for (int y = 0; y < kPairs; ++y) {
                    const int h = hd_of(y) * 16 + 2 * (y % kPerHead);
                    t2[y] = fma2(f2(__uint_as_float(sr[h + 8]), NC > 1 ? __uint_as_float(sr[h + 9]) : 0.f), f2(kLevel2, kLevel2),
                                 f2(__uint_as_float(sr[h]), NC > 1 ? __uint_as_float(sr[h + 1]) : 0.f));
                }
#pragma unroll
                for (int x = 0; x < kPairs; ++x) {
                    const int hd = hd_of(x);
                    t2[x] = fma2(t2[x], mul2(qf[x], f2(ks[hd], ks[hd])), f2(lv[hd], lv[hd]));
                }
                const bool hide = !valid[0] || !valid[kHeads - 1];
                const bool any_hidden = __any_sync(0xffffffffu, hide);
                if (MQ || any_hidden) {
                    // Query column y of a head is query token y / G, which sees positions <= its own.
                    const int ahead = mt.z * kTile + row - qm.z;      // of the first query token
#pragma unroll
                    for (int x = 0; x < kPairs; ++x) {
                        float2 t = unf2(t2[x]);
                        const int y = (HP == 1 ? 8 * grp : 0) + 2 * (x % kPerHead);
                        if (!valid[hd_of(x)] || (MQ && ahead > (y >> lgG))) t.x = -INFINITY;
                        if (!valid[hd_of(x)] || (MQ && ahead > ((y + 1) >> lgG))) t.y = -INFINITY;
                        t2[x] = f2(t.x, t.y);
                    }
                }
                // Exponents t - m; a reference moves when one exceeds kHeadroom.
                uint64_t d[kPairs];
                float top = -INFINITY;
#pragma unroll
                for (int x = 0; x < kPairs; ++x) {
                    d[x] = add2(t2[x], neg_m[x]);
                    const float2 v = unf2(d[x]);
                    top = fmaxf(top, NC > 1 ? fmaxf(v.x, v.y) : v.x);
                }
                if (named_bar_or(bar, 128, top > kHeadroom)) {
                    // Rare: move the references to the running maxima less kStart.
#pragma unroll
                    for (int x = 0; x < kPairs; ++x) {
                        const float2 t = unf2(t2[x]);
                        const float m0 = warp_max_redux(t.x), m1 = NC > 1 ? warp_max_redux(t.y) : m0;
                        if (lane == 0) {
                            misc->red[quad][col(x)] = m0;
                            misc->red[quad][col(x) + 1] = m1;
                        }
                    }
                    named_bar_sync(bar, 128);
                    float a[kGW];
#pragma unroll
                    for (int j = 0; j < kGW; ++j) a[j] = 1.f;
#pragma unroll
                    for (int x = 0; x < kPairs; ++x) {
                        const float2 nm = unf2(neg_m[x]);
                        float n2[2] = {nm.x, nm.y};
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int j = col(x) + y;
                            const float t = fmaxf(fmaxf(misc->red[0][j], misc->red[1][j]),
                                                  fmaxf(misc->red[2][j], misc->red[3][j]));
                            const float moved = fminf(n2[y], kStart - t);
                            a[local(x) + y] = fast_exp2(moved - n2[y] + kLift);
                            n2[y] = moved;
                        }
                        neg_m[x] = f2(n2[0], n2[1]);
                        // The denominator's factor with its 2^60 (as for u), O's without.
                        l_run[x] = mul2(mul2(l_run[x], f2(kUnlift, kUnlift)), f2(a[local(x)], a[local(x) + 1]));
                        a[local(x)] *= kUnlift;
                        a[local(x) + 1] *= kUnlift;
                        d[x] = add2(t2[x], neg_m[x]);
                    }
                    if (!seg_first) {
                        // O through tile i-1, in TMEM (thread <-> head-dim row).
                        if (!__all_sync(0xffffffffu, wait_for(smem_u32(&misc->o_full[(i - 1) & 1]), ((i - 1) >> 1) & 1,
                                                               &misc->never, lim))) {
                            misc->abort = 1;
                            set_error(p.err, PK_DEVERR_TIMEOUT);
                            ++i;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t oaddr = lane_addr + C_::tO + (seg & 1) * NP + 8 * grp;
#pragma unroll 1
                        for (int term = 0; term < 3; ++term) {
                            float o8[kGW];
                            tmem_ld<kGW>(oaddr + term * PW, o8);
#pragma unroll
                            for (int x = 0; x < kGW; ++x) o8[x] *= a[x];
                            static_assert(kGW == 8, "one store");
                            tmem_st8(oaddr + term * PW, o8);
                        }
                    }
                    // red[] is rewritten only in a later rare path, after the next vote.
                }
                // Weights in their three terms: words[term][4 columns of the group].
                static_assert(kGW == 8, "two words a term");
                uint32_t words[3][2] = {};
#pragma unroll
                for (int x = 0; x < kPairs; ++x) {
                    const float2 e = unf2(add2(d[x], f2(kLift, kLift)));
                    const uint64_t u = f2(fast_exp2(e.x), NC > 1 ? fast_exp2(e.y) : 0.f);
                    const float iv = ivs[hd_of(x)];
                    l_run[x] = fma2(u, f2(iv, iv), l_run[x]);
                    uint32_t h1, h2, h3;
                    const float2 w = unf2(mul2(u, f2(kUnlift, kUnlift)));
                    split_weights(w.x, w.y, h1, h2, h3);
                    const int j = local(x), sh = (j & 2) * 8;
                    words[0][j >> 2] |= h1 << sh;
                    words[1][j >> 2] |= h2 << sh;
                    words[2][j >> 2] |= h3 << sh;
                }
                if (!__all_sync(0xffffffffu, p_free || wait_slow(smem_u32(&misc->o_full[sb]), ((i >> 1) & 1) ^ 1,
                                                                 &misc->never, lim))) {
                    misc->abort = 1;
                    set_error(p.err, PK_DEVERR_TIMEOUT);
                    ++i;
                    break;
                }
                // Rows of hidden tokens are zeroed once this tile's V has landed: the
                // MMA multiplies every V row by its weight, and theirs may hold stale
                // bytes or NaN.
                if (any_hidden &&
                    !__all_sync(0xffffffffu, wait_for(smem_u32(&misc->vfull[st]), (i / kStages) & 1, &misc->never,
                                                       lim))) {
                    misc->abort = 1;
                    set_error(p.err, PK_DEVERR_TIMEOUT);
                    ++i;
                    break;
                }
                if (hide && (HP == 2 || grp == 0)) {
#pragma unroll
                    for (int hd = 0; hd < kHeads; ++hd) {
                        if (valid[hd]) continue;
                        uint4 *vrow = reinterpret_cast<uint4 *>(stage_ptr + st * C_::StageBytes + C_::VOff +
                                                                (hd0 + hd) * C_::HeadBytes + row * D);
#pragma unroll
                        for (int x = 0; x < D / 16; ++x) vrow[x] = make_uint4(0, 0, 0, 0);
                    }
                }
                // MN-major, no swizzle: 16 columns side by side, 8 tokens 16 bytes
                // apart, 128 bytes to the next 16 columns, 8 NP to the next 8 tokens.
                uint8_t *prow = p_ptr + sb * C_::PBytes + (row >> 3) * (8 * NP) + (row & 7) * 16;
                if constexpr (PW == 8) {
                    *reinterpret_cast<uint4 *>(prow) = make_uint4(words[0][0], words[0][1], words[1][0], words[1][1]);
                    *reinterpret_cast<uint4 *>(prow + 128) = make_uint4(words[2][0], words[2][1], 0, 0);
                } else {
#pragma unroll
                    for (int x = 0; x < 3; ++x)
                        *reinterpret_cast<uint2 *>(prow + 128 * x + 8 * grp) = make_uint2(words[x][0], words[x][1]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&misc->p_full[sb]));
            }

            // The previous segment's read-out, one tile late.
            if (pending && !finalize()) {
                misc->abort = 1;
                set_error(p.err, PK_DEVERR_TIMEOUT);
                ++i;
                break;
            }
            if (seg_last) {
                pending = true;
                pend_seg = seg;
                pend_s = mt.x;
                pend_q0 = qm.x;
                pend_qn = qm.y;
                pend_h = mt.y;
                pend_i = i;
                pend_t0 = seg_t0;
                pend_i0 = seg_i0;
                pend_complete = seg_t0 == 0 && mt.z == mt.w - 1;
                pend_cut_end = mt.z == mt.w - 1;
                close_segment();
            }
        }
        // Its group may be further on (a wait can end for one warp just after another
        // gave up): it meets them at the barriers that are left, or they would wait for ever.
#pragma unroll 1
        for (; i <= n_tiles; ++i) {
            if (i == n_tiles || named_bar_or(bar, 128, false)) named_bar_sync(bar, 128);
        }
        tc_fence_before();
    }

    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C_::TmemCols);
    }
}

// Merge of cut segments.  CTA (c, y) combines query columns 2 y and 2 y + 1 of
// the segment that was cut at the start of CTA c's range and ends in it, from
// every CTA it spans; thread r handles O^T row r.  Two parts are one round
// trip.  A segment of a long context spans dozens of CTAs (at one sequence of
// 131,072 tokens, 38): their headers are read side by side by the threads, the
// weights follow in shared memory, and the rows are added with kMergeAhead
// reads on their way -- part after part, the chain of reads took longer than
// the attention.  The order of the sum is the parts' order in any case.
constexpr int kMergeAhead = 8;

template <int D, int NC, int HP>
__global__ void __launch_bounds__(128)
decode_fp8_merge_kernel(const DecodeParams p, int C) {
    constexpr int CW = HP == 2 ? 8 : kNPad;
    constexpr int kCols = NC < 2 ? 1 : 2;                   // columns per head of this CTA
    constexpr int kAll = HP * kCols;
    __shared__ int part_slot[kTcMaxCtas];                   // slot of a part, -1 for an empty range
    __shared__ float part_m[kTcMaxCtas][kAll], part_l[kTcMaxCtas][kAll], den_all[kAll];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Slot *slots = static_cast<const Slot *>(p.tc_slots);
    const int c = blockIdx.x, y = blockIdx.y;
    const int row = threadIdx.x;
    const int hr = HP == 2 ? row >> 6 : 0;
    const int dd = HP == 2 ? (row & 63) : row;
    const bool row_ok = HP == 2 || row < D;
    const int orow = row_ok ? row : 0;
    const int j0 = hr * CW + 2 * y;                         // this row's first column in the slots
    const Slot *mine = slots + 2 * c;
    // Everything two parts need is read at once, before the flag is known.
    const Slot *q0 = slots + 2 * (c > 0 ? c - 1 : c);
    const Slot *q1 = q0 + 1;
    const int flag = mine->flag;
    const int s = mine->s, h = mine->h;
    const int64_t start = mine->start_tile, T = mine->total_tiles;
    const int ca = mine->first_cta;
    const int64_t beg_prev = q0->range_beg;
    float mm[kCols], ml[kCols], mo[kCols], am[kCols], al[kCols], ao[kCols], bm[kCols], bl[kCols], bo[kCols];
#pragma unroll
    for (int x = 0; x < kCols; ++x) {
        const int j = j0 + x;
        mm[x] = mine->m[j];
        ml[x] = mine->l[j];
        mo[x] = mine->o[j * 128 + orow];
        am[x] = q0->m[j];
        al[x] = q0->l[j];
        ao[x] = q0->o[j * 128 + orow];
        bm[x] = q1->m[j];
        bl[x] = q1->l[j];
        bo[x] = q1->o[j * 128 + orow];
    }
    if (flag != 1) return;                                  // the same for the whole CTA
    float num[kCols], den[kCols];
    if (ca == c - 1) {
        const bool first_of_prev = beg_prev >= start;
#pragma unroll
        for (int x = 0; x < kCols; ++x) {
            const float pm = first_of_prev ? am[x] : bm[x];
            const float pl = first_of_prev ? al[x] : bl[x];
            const float po = first_of_prev ? ao[x] : bo[x];
            const float M = fmaxf(pm, mm[x]);
            // 2^60 too large for the denominators (see kLift), which are made as much smaller first.
            const float a0 = fast_exp2(pm - M + kLift), a1 = fast_exp2(mm[x] - M + kLift);
            den[x] = a0 * (pl * kUnlift) + a1 * (ml[x] * kUnlift);
            num[x] = (a0 * kUnlift) * po + (a1 * kUnlift) * mo[x];
        }
    } else {
        const int parts = c - ca + 1;
#pragma unroll 1
        for (int i = threadIdx.x; i < parts; i += 128) {
            const int cc = ca + i;
            const int64_t b0 = slots[2 * cc].range_beg, b1 = cc + 1 < C ? slots[2 * (cc + 1)].range_beg : T;
            const int at = 2 * cc + (b0 >= start ? 0 : 1);
            part_slot[i] = b0 == b1 ? -1 : at;
#pragma unroll
            for (int x = 0; x < kAll; ++x) {
                const int j = x / kCols * CW + 2 * y + x % kCols;
                part_m[i][x] = b0 == b1 ? -INFINITY : slots[at].m[j];
                part_l[i][x] = b0 == b1 ? 0.f : slots[at].l[j];
            }
        }
        __syncthreads();
        // One warp a column: the largest reference, the weights, the denominator.
        const int x = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (x < kAll) {
            float M = -INFINITY, sum = 0.f;
            for (int i = lane; i < parts; i += 32) M = fmaxf(M, part_m[i][x]);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            for (int i = lane; i < parts; i += 32) {
                const float a = fast_exp2(part_m[i][x] - M + kLift);      // (an empty part's -inf: 0)
                part_m[i][x] = a * kUnlift;
                sum = fmaf(a, part_l[i][x] * kUnlift, sum);
            }
            sum = warp_sum(sum);
            if (lane == 0) den_all[x] = sum;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kCols; ++k) {
            num[k] = 0.f;
            den[k] = den_all[hr * kCols + k];
        }
        for (int i0 = 0; i0 < parts; i0 += kMergeAhead) {
            float o[kMergeAhead][kCols];
#pragma unroll
            for (int i = 0; i < kMergeAhead; ++i) {
                const int at = i0 + i < parts ? part_slot[i0 + i] : -1;
#pragma unroll
                for (int k = 0; k < kCols; ++k) o[i][k] = at >= 0 ? slots[at].o[(j0 + k) * 128 + orow] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kMergeAhead; ++i) {
                if (i0 + i < parts) {
#pragma unroll
                    for (int k = 0; k < kCols; ++k) num[k] = fmaf(part_m[i0 + i][hr * kCols + k], o[i][k], num[k]);
                }
            }
        }
    }
    if (!row_ok) return;
    // Column cq: query token cq / G of the sequence, query head cq % G of this
    // row's KV head; a sequence whose rows are not within the queries given has none.
    const int Gq = p.num_heads / p.num_kv_heads, lgG = __ffs(Gq) - 1;
    int row0 = s, qn = 1;
    if (p.cu_q_lens) {
        row0 = p.cu_q_lens[s];
        const int row1 = p.cu_q_lens[s + 1];
        qn = row1 - row0;
        if (row0 < 0 || qn < 0 || row1 > p.total_q || qn > p.q_len) return;
    }
#pragma unroll
    for (int x = 0; x < kCols; ++x) {
        const int cq = 2 * y + x;
        if ((cq >> lgG) >= qn) continue;
        const int qh = (h * HP + hr) * Gq + (cq & (Gq - 1));
        store_out(p, (static_cast<size_t>(row0 + (cq >> lgG)) * p.num_heads + qh) * D + dd,
                  den[x] != 0.f ? num[x] / den[x] : 0.f);
    }
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 get_encoder() {
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

// [P Hkv] pieces of B rows of D bytes, one piece a box.
bool encode_piece_map(CUtensorMap *m, const void *base, const DecodeFp8Params &p) {
    auto enc = get_encoder();
    if (!enc) return false;
    const cuuint64_t D = p.head_dim, B = p.block_size;
    const cuuint64_t pieces = static_cast<cuuint64_t>(p.num_blocks > 0 ? p.num_blocks : 1) * p.num_kv_heads;
    cuuint64_t dims[3] = {D, B, pieces};
    cuuint64_t strides[2] = {D, B * D};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(B), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NC, int HP>
cudaError_t launch_shape(const DecodeFp8Params &p, int sms, cudaStream_t stream) {
    const int C = std::min(sms * Shape<D, NC, HP>::CtasPerSm, static_cast<int>(kMaxCtas));
    CUtensorMap mk, mv;
    if (!encode_piece_map(&mk, p.k8, p) || !encode_piece_map(&mv, p.v8, p)) return cudaErrorInvalidValue;
    auto *kernel = p.cu_q_lens ? decode_fp8_tc_kernel<D, NC, true, HP> : decode_fp8_tc_kernel<D, NC, false, HP>;
    constexpr size_t smem = Shape<D, NC, HP>::SmemBytes;
    cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(Shape<D, NC, HP>::Threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, mk, mv, p);
    if (e != cudaSuccess) return e;
    if (!p.tc_slots) return cudaSuccess;   // no sequence longer than one tile: nothing is cut
    cfg.gridDim = dim3(C, (NC + 1) / 2);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, decode_fp8_merge_kernel<D, NC, HP>, static_cast<const DecodeParams &>(p), C);
}

template <int NC>
cudaError_t launch_dim(const DecodeFp8Params &p, int C, cudaStream_t stream) {
    if (p.head_dim == 128) return launch_shape<128, NC, 1>(p, C, stream);
    if constexpr (NC <= 8) {
        if (p.num_kv_heads % 2 == 0) return launch_shape<64, NC, 2>(p, C, stream);
    }
    return launch_shape<64, NC, 1>(p, C, stream);
}

}  // namespace

cudaError_t launch_decode_fp8_tensor_core(const DecodeFp8Params &p, cudaStream_t stream) {
    const int C = sm_count();
    if (C <= 0) return cudaErrorNoDevice;
    // MMA columns: the group's query heads times the query tokens per sequence.
    switch ((p.num_heads / p.num_kv_heads) * (p.cu_q_lens ? p.q_len : 1)) {
        case 1: return launch_dim<1>(p, C, stream);
        case 2: return launch_dim<2>(p, C, stream);
        case 4: return launch_dim<4>(p, C, stream);
        case 8: return launch_dim<8>(p, C, stream);
        case 16: return launch_dim<16>(p, C, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pk
