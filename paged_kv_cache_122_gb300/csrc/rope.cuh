// Rotary position angles (sm_103a) and what the two rotary appends share.
#pragma once

#include "common.cuh"

namespace pk {

struct bool2 {
    bool x, y;
};

// A frequency f (radians a position) in turns a position, as a 64-bit binary
// fraction: the integer nearest below f / (2 pi) * 2^64, modulo 2^64 (whole
// turns do not matter, since positions are integers).
//
// Why fixed point: at position 100,000 an angle in fp32 is off by 0.004
// radians (its spacing there), and what a rotation needs is the angle modulo
// a turn.  position * turns in 64-bit integers is exact modulo a turn, so the
// error is that of the fraction alone, 2^-64 turns a position: below 2^-33
// turns for every 31-bit position, at the price of two integer multiplies.
//
// f = m 2^e with m < 2^24, and 1 / (2 pi) = K 2^-96 (from the series of pi),
// so the fraction is (m K) >> (32 - e); m K has at most 118 bits.  A
// frequency that is not finite or not below 2^32 gives 0 (no rotation).
PK_DEV uint64_t turns_per_position(float f) {
    const uint32_t b = __float_as_uint(f);
    const int field = static_cast<int>((b >> 23) & 0xffu);
    if (field == 0 || field >= 127 + 32) return 0;      // zero, below 2^-126, or too large
    const uint64_t m = (b & 0x7fffffu) | 0x800000u;
    const int shift = 32 - (field - 150);               // 24 .. 181
    if (shift >= 128) return 0;
    constexpr uint64_t kHi = 0x28be60dbull, kLo = 0x9391054a7f09d5f4ull;   // K = kHi 2^64 + kLo
    const unsigned __int128 prod = static_cast<unsigned __int128>(m) * kLo +
                                   (static_cast<unsigned __int128>(m * kHi) << 64);
    const uint64_t t = static_cast<uint64_t>(prod >> shift);
    return (b & 0x80000000u) ? 0ull - t : t;
}

// cos and sin of position * frequency, times `factor`.  The nearest quarter
// turn is taken off in integers; the rest, at most an eighth of a turn, is x
// below pi / 4, where the Taylor series to x^9 and x^8 are within 2^-25 of sine
// and cosine (the next terms are x^11 / 11! and x^10 / 10!).
PK_DEV float2 rotation(int64_t position, uint64_t turns, float factor) {
    const uint64_t a = static_cast<uint64_t>(position) * turns;
    const uint32_t quarter = static_cast<uint32_t>((a + (1ull << 61)) >> 62);
    const int64_t rest = static_cast<int64_t>(a - (static_cast<uint64_t>(quarter) << 62));
    constexpr float kUnit = 3.65729520e-10f;                    // 2 pi / 2^34: of rest >> 30
    const float x = static_cast<float>(static_cast<int32_t>(rest >> 30)) * kUnit, x2 = x * x;
    float s = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), 1.f) * x;
    float c = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.f / 40320, -1.f / 720), 1.f / 24), -0.5f), 1.f);
    if (quarter & 1) {
        const float t = c;
        c = -s;
        s = t;
    }
    if (quarter & 2) {
        c = -c;
        s = -s;
    }
    return make_float2(c * factor, s * factor);
}

// 16-byte load of data that the same call may write elsewhere (a rotation in
// place): no read-only path, no place in L1.
PK_DEV uint4 ld_stream(const void *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    return r;
}

PK_DEV uint4 pack8(const float f[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// A head's D elements are handled in units of two 8-element vectors, so that
// neighbouring lanes touch neighbouring vectors.  Interleaved layout: unit j has
// those at 8 j and D / 2 + 8 j (a warp's rows are whole 128-byte lines, and with
// half of a head rotated every lane rotates its first vector, none its second).
// Half layout: of the first `rot` elements, unit j < rot / 16 has those at 8 j
// and rot / 2 + 8 j, each other's partners; of the others those at
// rot + 8 (j - rot / 16) and half of the rest further on.
template <bool kInterleaved>
PK_DEV int2 unit_offsets(int j, int rot, int D) {
    if constexpr (kInterleaved) return make_int2(8 * j, (D >> 1) + 8 * j);
    const int n = rot >> 4;
    if (j < n) return make_int2(8 * j, (rot >> 1) + 8 * j);
    const int a = rot + 8 * (j - n);
    return make_int2(a, a + ((D - rot) >> 1));
}

// Whether unit j's vectors are rotated (x: the first, y: the second).
template <bool kInterleaved>
PK_DEV bool2 unit_turned(int j, int rot, int D) {
    if constexpr (kInterleaved) return {8 * j < rot, (D >> 1) + 8 * j < rot};
    return {16 * j < rot, 16 * j < rot};
}

// Two pairs (x, y) at once, in packed instructions.
PK_DEV void turn_pairs(float &x0, float &x1, float &y0, float &y1, const float *cosines, const float *sines) {
    const uint64_t c = f2(cosines[0], cosines[1]), s = f2(sines[0], sines[1]);
    const uint64_t x = f2(x0, x1), y = f2(y0, y1);
    const float2 ys = unf2(mul2(y, s));
    const float2 u = unf2(fma2(x, c, f2(-ys.x, -ys.y))), v = unf2(fma2(y, c, mul2(x, s)));
    x0 = u.x;
    x1 = u.y;
    y0 = v.x;
    y1 = v.y;
}

// Interleaved layout: a vector is four pairs, the first of which is number 0 here.
PK_DEV void rotate_vector(float (&f)[8], const float *cosines, const float *sines) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) turn_pairs(f[2 * i], f[2 * i + 2], f[2 * i + 1], f[2 * i + 3], cosines + i, sines + i);
}

// Rotate unit j: `a` and `b` are its two vectors, `cosines` and `sines` the
// token's for pair 0 .. rot / 2 - 1.
template <bool kInterleaved>
PK_DEV void rotate_unit(float (&a)[8], float (&b)[8], const float *cosines, const float *sines, int j, int rot, int D) {
    const bool2 t = unit_turned<kInterleaved>(j, rot, D);
    if constexpr (kInterleaved) {
        if (t.x) rotate_vector(a, cosines + 4 * j, sines + 4 * j);
        if (t.y) rotate_vector(b, cosines + (D >> 2) + 4 * j, sines + (D >> 2) + 4 * j);
    } else if (t.x) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) turn_pairs(a[i], a[i + 1], b[i], b[i + 1], cosines + 8 * j + i, sines + 8 * j + i);
    }
}

// The same on bf16 vectors; those that are not rotated keep their bits.
template <bool kInterleaved>
PK_DEV void rotate_unit(uint4 &a, uint4 &b, const float *cosines, const float *sines, int j, int rot, int D) {
    const bool2 t = unit_turned<kInterleaved>(j, rot, D);
    float fa[8], fb[8];
    if constexpr (kInterleaved) {
        if (t.x) {
            unpack8(a, fa);
            rotate_vector(fa, cosines + 4 * j, sines + 4 * j);
            a = pack8(fa);
        }
        if (t.y) {
            unpack8(b, fb);
            rotate_vector(fb, cosines + (D >> 2) + 4 * j, sines + (D >> 2) + 4 * j);
            b = pack8(fb);
        }
    } else if (t.x) {
        unpack8(a, fa);
        unpack8(b, fb);
        rotate_unit<kInterleaved>(fa, fb, cosines, sines, j, rot, D);
        a = pack8(fa);
        b = pack8(fb);
    }
}

// Host-side checks that both rotary appends share: sizes, token strides (in
// elements, whole 16-byte vectors) and the rotation's own arguments.
inline int check_rope_args(int64_t q_out_stride, int64_t q_stride, int64_t k_stride, int64_t v_stride, int rot_dim,
                           float factor, int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                           int num_blocks, int block_size) {
    if (num_tokens < 0 || num_heads < 0 || num_kv_heads <= 0 || num_blocks < 0 || block_size <= 0) return PK_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128) return PK_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PK_ERR_UNSUPPORTED;
    if (num_heads > 65535 || num_kv_heads > 32767) return PK_ERR_SHAPE;
    if (rot_dim < 0 || rot_dim > head_dim) return PK_ERR_SHAPE;
    if (rot_dim % 16) return PK_ERR_UNSUPPORTED;
    if (!(factor >= 0x1p-20f && factor <= 0x1p20f)) return PK_ERR_SHAPE;
    const int64_t q_row = static_cast<int64_t>(num_heads) * head_dim;
    const int64_t kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (num_heads > 0 && (q_stride < q_row || q_out_stride < q_row)) return PK_ERR_SHAPE;
    if (k_stride < kv_row || v_stride < kv_row) return PK_ERR_SHAPE;
    if ((num_heads > 0 && (q_stride % 8 || q_out_stride % 8)) || k_stride % 8 || v_stride % 8)
        return PK_ERR_ALIGNMENT;
    return PK_OK;
}

}  // namespace pk
