// What the persistent decode kernels share: the flattened (sequence, KV head
// group, tile) space, its cut into one range of equal cost for each CTA, the
// workspace slots of cut segments and the kernel that merges them.
#pragma once

#include "decode.cuh"
#include "block_scan.cuh"

namespace pk {
namespace {

constexpr int kTile = 128;                                   // tokens per tile = MMA M of S^T
constexpr int kNPad = 16;                                    // query columns of a slot (at most)

// Workspace slot of a cut segment's part: slot 0 of a CTA holds the part of
// its first segment, slot 1 the part of its last one.
struct Slot {
    int32_t flag;          // slot 0 only: 1 = the merge kernel's CTA c combines this segment
    int32_t s, h;
    int32_t first_cta;     // slot 0 only: the CTA in whose range the segment starts
    int64_t start_tile;    // flattened index of the segment's (s, h) tile 0
    int64_t total_tiles;
    int64_t range_beg;     // slot 0 only: first tile of this CTA's range
    int64_t pad2[3];
    float m[kNPad];        // reference max per column (base 2)
    float l[kNPad];        // denominator per column
    float o[kNPad * 128];  // unnormalised output, [column][O^T row]
};
constexpr size_t kMaxCtas = kTcMaxCtas;

// A 32-bit load that bypasses L1: L2 is coherent with writes of other
// grids, so a value read before the programmatic wait and read again after
// it cannot come back stale from L1.
__device__ __forceinline__ int ld_cg(const int *p) {
    int v;
    asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// The sequence lengths, from the shared-memory copy when there is one;
// operator() clamps to [0, cap] (values outside are reported separately).
struct LenSrc {
    const int *cache;   // shared memory, or null
    const int *glob;
    int cap;
    __device__ __forceinline__ int raw(int s) const { return cache ? cache[s] : glob[s]; }
    __device__ __forceinline__ int operator()(int s) const {
        const int r = raw(s);
        return r < 0 ? 0 : (r > cap ? cap : r);
    }
};

// Walks the flattened (sequence, KV head group, tile) space in order.
struct Walk {
    int s, h, t, nt, L, nh, ns;      // nh: KV head groups per sequence; ns: sequences
    __device__ __forceinline__ void load(const LenSrc &len) {
        L = len(s);
        nt = (L + kTile - 1) / kTile;
    }
    __device__ __forceinline__ void next(const LenSrc &len) {
        if (++t < nt) return;
        t = 0;
        if (++h < nh) return;
        h = 0;
#pragma unroll 1
        do {
            if (++s >= ns) return;
            load(len);
        } while (nt == 0);
    }
};

// 64-bit division, out of line: each copy of its code is as long as the rest
// of the plan, and the warps' different loops share one instruction cache.
__device__ __noinline__ int64_t quotient(int64_t a, int64_t b) { return a / b; }

// This CTA's range of the flattened tile space.  Tile x, whose cost interval
// starts at a_x (a segment's tile 0 at its start, tile t >= 1 at start +
// seg_cost + full * t, full the cost of a full tile), belongs to CTA k when
// P_k <= a_x < P_{k+1}, P_k = k * W / C, W the total cost.  Writes misc->bnd (the first tile of this range and of the next),
// misc->s0 / rem0 (where the range starts) and misc->first_cta (the CTA in
// whose range a segment cut at this range's start begins); returns the
// total tile count and, in *odd, whether some length is zero or outside
// [0, cap] (the same for every thread).  Every thread of the CTA calls it.
template <int kThreadsT, typename MiscT>
__device__ __forceinline__ int64_t plan_range(const LenSrc lens, MiscT *misc, int N, int Hkv, int c, int C,
                                           int64_t seg_cost, int tile_cost, int tok_cost, int *odd) {
    // A segment of L tokens in nt tiles costs seg_cost + tile_cost * nt -
    // tok_cost * L: a full tile costs full = tile_cost - tok_cost * kTile, and
    // only a segment's last tile can be partial, so tile t >= 1 starts at
    // seg_cost + full * t.
    const int64_t full = tile_cost - static_cast<int64_t>(tok_cost) * kTile;
    auto seg_total = [&](int64_t nt, int L) -> int64_t {
        return nt > 0 ? seg_cost + tile_cost * nt - static_cast<int64_t>(tok_cost) * L : 0;
    };
    const int per = (N + kThreadsT - 1) / kThreadsT;
    const int s_lo = min(N, static_cast<int>(threadIdx.x) * per), s_hi = min(N, s_lo + per);
    const int cap = lens.cap;
    int64_t mine = 0, mine_w = 0;
    int bad = 0;
#pragma unroll 1
    for (int s = s_lo; s < s_hi; ++s) {
        const int raw = lens.raw(s);
        bad |= raw <= 0 || raw > cap;
        const int L = lens(s);
        const int64_t nt = (L + kTile - 1) / kTile;
        mine += nt * Hkv;
        mine_w += seg_total(nt, L) * Hkv;
    }
    int64_t T, W;
    const int64_t my_off = block_exclusive_scan<kThreadsT>(mine, misc->scan, &T);
    const int64_t my_off_w = block_exclusive_scan<kThreadsT>(mine_w, misc->scan_w, &W);
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        const int64_t P = quotient(static_cast<int64_t>(c + k) * W, C);
        if (P >= W) {
            if (threadIdx.x == 0) misc->bnd[k] = T;
            continue;
        }
        if (my_off_w <= P && P < my_off_w + mine_w) {
            int64_t acc_t = my_off, acc_w = my_off_w;
        #pragma unroll 1
    for (int s = s_lo; s < s_hi; ++s) {
                const int L = lens(s);
                const int64_t nt = (L + kTile - 1) / kTile;
                const int64_t segc = seg_total(nt, L);
                const int64_t cw = segc * Hkv;
                if (P < acc_w + cw) {
                    const int64_t q = P - acc_w;
                    int64_t h = quotient(q, segc);
                    const int64_t r = q - h * segc;
                    // The first tile of the segment that starts at or after r.
                    int64_t t = r == 0 ? 0 : quotient(r - seg_cost + full - 1, full);
                    if (r > 0 && t < 1) t = 1;
                    if (t >= nt) {
                        ++h;
                        t = 0;
                    }
                    misc->bnd[k] = acc_t + h * nt + t;
                    break;
                }
                acc_t += nt * Hkv;
                acc_w += cw;
            }
        }
    }
    __syncthreads();
    const int64_t b0 = misc->bnd[0];
    if (misc->bnd[1] > b0) {
        int64_t acc = my_off, acc_w = my_off_w;
        if (acc <= b0 && b0 < acc + mine) {
        #pragma unroll 1
    for (int s = s_lo; s < s_hi; ++s) {
                const int L = lens(s);
                const int64_t nt = (L + kTile - 1) / kTile;
                const int64_t w = nt * Hkv;
                if (b0 < acc + w) {
                    misc->s0 = s;
                    misc->rem0 = b0 - acc;
                    // If the range starts inside a segment, the CTA where that
                    // segment starts (the owner of its tile 0's cost start).
                    const int64_t h0 = quotient(b0 - acc, nt);
                    const int64_t a = acc_w + h0 * seg_total(nt, L);
                    int64_t k = W > 0 ? quotient(a * C, W) : 0;
                    while (k + 1 < C && quotient((k + 1) * W, C) <= a) ++k;
                    while (k > 0 && quotient(k * W, C) > a) --k;
                    misc->first_cta = static_cast<int32_t>(k);
                    break;
                }
                acc += w;
                acc_w += seg_total(nt, L) * Hkv;
            }
        }
    }
    *odd = __syncthreads_or(bad);
    return T;
}

// Warp max of a float in one integer reduction: the bits are mapped to an
// unsigned key with the same order (a non-negative float gets its sign bit
// set, a negative one all bits flipped), reduced, and mapped back.
__device__ __forceinline__ float warp_max_redux(float v) {
    const uint32_t b = __float_as_uint(v);
    const uint32_t key = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    const uint32_t m = __reduce_max_sync(0xffffffffu, key);
    return __uint_as_float((m & 0x80000000u) ? (m & 0x7fffffffu) : ~m);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void store_out(const DecodeParams &p, size_t idx, float v) {
    if (p.out_fp32) static_cast<float *>(p.out)[idx] = v;
    else static_cast<uint16_t *>(p.out)[idx] = static_cast<uint16_t>(pack_bf16x2(v, 0.f) & 0xffffu);
}

// One CTA per decode CTA c: if c's first segment was cut at its start and
// ends in c, combine the parts of that segment from every CTA it spans.
// Thread r handles O^T row r (as the decode kernel's TMEM lanes).
template <int D, int NC, int HP>
__global__ void __launch_bounds__(128)
decode_tc_merge_kernel(const DecodeParams p, int C) {
    constexpr int CW = HP == 2 ? 8 : kNPad;
    // A decode grid launched next in the stream as this grid's programmatic
    // dependent may begin its set-up (before this grid completes it reads
    // only the sequence lengths, and reads them again afterwards).  Its CTAs
    // find room only as this decode grid's CTAs leave their SMs.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // Launched as a programmatic dependent of the decode grid: wait for it
    // to finish and its writes to be visible.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Slot *slots = static_cast<const Slot *>(p.tc_slots);
    const int c = blockIdx.x;
    const int row = threadIdx.x;
    const int hr = HP == 2 ? row >> 6 : 0;           // head of the pair (HP == 2)
    const int dd = HP == 2 ? (row & 63) : row;       // head-dim element
    const bool row_ok = HP == 2 || row < D;
    const int orow = row_ok ? row : 0;
    const Slot *mine = slots + 2 * c;
    // Everything the common case needs (this CTA's slot 0 and both slots of
    // CTA c - 1) is loaded at once, before the flag is known.
    const Slot *q0 = slots + 2 * (c > 0 ? c - 1 : c);
    const Slot *q1 = q0 + 1;
    const int flag = mine->flag;
    const int s = mine->s, h = mine->h;
    const int64_t start = mine->start_tile, T = mine->total_tiles;
    const int ca = mine->first_cta;
    const int64_t beg_prev = q0->range_beg;
    float mm[NC], ml[NC], mo[NC], am[NC], al[NC], ao[NC], bm[NC], bl[NC], bo[NC];
#pragma unroll
    for (int cq = 0; cq < NC; ++cq) {
        const int j = hr * CW + cq;
        mm[cq] = mine->m[j];
        ml[cq] = mine->l[j];
        mo[cq] = mine->o[j * 128 + orow];
        am[cq] = q0->m[j];
        al[cq] = q0->l[j];
        ao[cq] = q0->o[j * 128 + orow];
        bm[cq] = q1->m[j];
        bl[cq] = q1->l[j];
        bo[cq] = q1->o[j * 128 + orow];
    }
    if (flag != 1 || !row_ok) return;
    // First tile of CTA cc's range (the decode grid wrote it into slot 0).
    auto range_beg = [&](int cc) -> int64_t { return cc < C ? slots[2 * cc].range_beg : T; };
    float num[NC], den[NC];
    if (ca == c - 1) {
        // Two parts: CTA c - 1 (slot 0 if the segment is its first, else 1) and this CTA.
        const bool first_of_prev = beg_prev >= start;
#pragma unroll
        for (int cq = 0; cq < NC; ++cq) {
            const float pm = first_of_prev ? am[cq] : bm[cq];
            const float pl = first_of_prev ? al[cq] : bl[cq];
            const float po = first_of_prev ? ao[cq] : bo[cq];
            const float M = fmaxf(pm, mm[cq]);
            const float a0 = rescale(pm, M), a1 = rescale(mm[cq], M);
            den[cq] = a0 * pl + a1 * ml[cq];
            num[cq] = a0 * po + a1 * mo[cq];
        }
    } else {
        // Contributors are the CTAs from ca to c with a non-empty range (when
        // the grid has more CTAs than tiles, some ranges are empty and hold
        // no slot).
        float M[NC];
#pragma unroll
        for (int cq = 0; cq < NC; ++cq) M[cq] = -INFINITY;
        for (int cc = ca; cc <= c; ++cc) {
            if (range_beg(cc) == range_beg(cc + 1)) continue;
            const Slot *sl = slots + 2 * cc + (range_beg(cc) >= start ? 0 : 1);
#pragma unroll
            for (int cq = 0; cq < NC; ++cq) M[cq] = fmaxf(M[cq], sl->m[hr * CW + cq]);
        }
#pragma unroll
        for (int cq = 0; cq < NC; ++cq) num[cq] = den[cq] = 0.f;
        for (int cc = ca; cc <= c; ++cc) {
            if (range_beg(cc) == range_beg(cc + 1)) continue;
            const Slot *sl = slots + 2 * cc + (range_beg(cc) >= start ? 0 : 1);
#pragma unroll
            for (int cq = 0; cq < NC; ++cq) {
                const int j = hr * CW + cq;
                const float a = rescale(sl->m[j], M[cq]);
                den[cq] = fmaf(a, sl->l[j], den[cq]);
                num[cq] = fmaf(a, sl->o[j * 128 + row], num[cq]);
            }
        }
    }
    // Column cq: query token cq / G of the sequence, query head cq % G of
    // this row's KV head (as in the decode kernel).
    const int Gq = p.num_heads / p.num_kv_heads, lgG = __ffs(Gq) - 1;
    const int q0row = p.cu_q_lens ? p.cu_q_lens[s] : s;
    const int qn = p.cu_q_lens ? p.cu_q_lens[s + 1] - q0row : 1;
#pragma unroll
    for (int cq = 0; cq < NC; ++cq) {
        if ((cq >> lgG) >= qn) continue;
        const int qh = (h * HP + hr) * Gq + (cq & (Gq - 1));
        store_out(p, (static_cast<size_t>(q0row + (cq >> lgG)) * p.num_heads + qh) * D + dd,
                  den[cq] > 0.f ? num[cq] / den[cq] : 0.f);
    }
}

}  // namespace
}  // namespace pk
