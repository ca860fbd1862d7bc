// Rotary positions of Q and K rows on their way into MXFP4, shared by the
// rotating quantizer and the rotating cache append.
//
// A row of 128 channels has rotary / 2 pairs; pair i turns by the angle of its
// axis's position, whose cosine and sine the caller's table holds:
//   y_a = bf16(x_a c - x_b s),   y_b = bf16(x_b c + x_a s),
// (c, s) = table[position of axis(i)][i]. Pair i is channels (i, i + rotary/2),
// or (2i, 2i + 1) with adjacent pairs. Channels from `rotary` on pass through.
//
// The rotated value decides a 4-bit code, and an amax on a power of two the
// scale of 32 of them, so it is rounded as from exact arithmetic, whatever the
// order of the additions: bf16(fp32(x_a c - x_b s)) with the products and the
// difference in fp64 (the products of a bf16 and an fp32 value are exact
// there). The kernels get these bits from fp32: with p = fl(x_b s) and its exact
// remainder e from a fused multiply-add, y = fma(x_a, c, -p) - e is within two
// units in the last place of fp32, and rounds to the same bf16 value unless it
// lies within 4 such units of a border between two (9 of 65536 values); those
// pairs are done again in fp64. So are all of a lane with a result that is not finite, or
// with a pair whose results are both below 2^-20: where both products are below 2^-101 the
// remainders underflow, and a result that rounds to zero may come out with the wrong sign.
// (With a result from 2^-20 up beside it, a cosine or sine would have to be below 2^-80 and
// not 0, or 0 beside one below 2^-17: no rotation, whatever its scaling.) Rows of zeros take
// that way as well: 137 us where others take 92.
// The bf16 rounding itself is part of the operator: a model that rotates in
// its bf16 activations and then quantizes gets the same bytes.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "../../include/qk4v8.h"
#include "mx_encode.cuh"
#include "ptx.cuh"
#include "qk4v8_internal.h"

namespace qk4v8 {

// Eight lanes share a row (lane j = 0..7 of the row). After the rotation lane j
// holds channel chunks j and j + 8 (8 channels each). Before it, with half-split
// pairs, lane j < nrot (= rotary / 16) holds chunks j and j + nrot, the two
// halves of pairs 8j .. 8j + 7, and the other lanes the chunks that pass
// through; so a pair never crosses lanes. Adjacent pairs stay inside a chunk.
__device__ __forceinline__ void rope_chunks(bool adjacent, int nrot, int j, int &c0, int &c1) {
    if (adjacent || j < nrot) {
        c0 = j;
        c1 = j + (adjacent ? 8 : nrot);
    } else {
        c0 = nrot + j;  // 2 nrot + (j - nrot)
        c1 = 8 + j;     // c0 + (8 - nrot)
    }
}

// (cos, sin) of the lane's 8 pairs, and their owner's flag: does this lane rotate
// its first four pairs (x) / last four (y)?
struct RopeTrig {
    float2 c[4], s[4];  // pairs 2i, 2i + 1
    bool lo, hi;
};

// Position of token t of batch entry b on an axis. A position outside the table reads
// row 0 and is reported.
__device__ __forceinline__ int rope_position(const RopeParams &r, int b, int t, int axis, int base, int32_t *status) {
    const int pos = r.positions ? r.positions[axis * r.pos_sa + b * r.pos_sb + t * r.pos_st] : base + t;
    if (pos >= 0 && pos < r.max_pos) return pos;
    if (status) atomicCAS(status, 0, QK4V8_ERR_INVALID_ARG);
    return 0;
}

template <bool kAdjacent>
__device__ __forceinline__ void rope_load(const RopeParams &r, int b, int t, int base, int j, bool valid,
                                          int32_t *status, RopeTrig &g) {
    const int nrot = r.rotary >> 4;
    g.lo = valid && (kAdjacent ? j < 2 * nrot : j < nrot);
    g.hi = valid && (kAdjacent ? j + 8 < 2 * nrot : j < nrot);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        g.c[i] = make_float2(1.f, 1.f);
        g.s[i] = make_float2(0.f, 0.f);
    }
    if (!valid) return;
    const int half = r.rotary >> 1;
    if (r.n_axes == 1) {
        const float *row = r.table + static_cast<int64_t>(rope_position(r, b, t, 0, base, status)) * r.rotary;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // Pairs 2i, 2i + 1 of the lane: one 16-byte load.
            const int pair = kAdjacent ? 4 * (j + 8 * (i >> 1)) + 2 * (i & 1) : 8 * j + 2 * i;
            if (pair < half) {
                const float4 v = *reinterpret_cast<const float4 *>(row + 2 * pair);
                g.c[i] = make_float2(v.x, v.z);
                g.s[i] = make_float2(v.y, v.w);
            }
        }
        return;
    }
    int pos[4] = {0, 0, 0, 0};
#pragma unroll
    for (int a = 0; a < 4; ++a)
        if (a < r.n_axes) pos[a] = rope_position(r, b, t, a, base, status);
    // The axes of the lane's pairs, two bits each: one run of 8, or two of 4.
    const uint32_t axes =
        kAdjacent ? static_cast<uint32_t>(r.pair_axis[0] >> (8 * j)) << 24 >> 24 |
                        static_cast<uint32_t>(r.pair_axis[1] >> (8 * j)) << 24 >> 16
                  : static_cast<uint32_t>((j < 4 ? r.pair_axis[0] : r.pair_axis[1]) >> (16 * (j & 3)));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int pair = kAdjacent ? 4 * (j + 8 * (i >> 2)) + (i & 3) : 8 * j + i;
        if (pair < half) {
            const int axis = static_cast<int>((axes >> (2 * i)) & 3);
            const int at = axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
            const float2 v = *reinterpret_cast<const float2 *>(r.table + static_cast<int64_t>(at) * r.rotary + 2 * pair);
            if (i & 1) {
                g.c[i >> 1].y = v.x;
                g.s[i >> 1].y = v.y;
            } else {
                g.c[i >> 1].x = v.x;
                g.s[i >> 1].x = v.y;
            }
        }
    }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// One pair in fp64.
__device__ __forceinline__ void rotate_pair_f64(float a, float b, float c, float s, float &ya, float &yb) {
    const double da = a, db = b, dc = c, ds = s;
    ya = __double2float_rn(__dsub_rn(__dmul_rn(da, dc), __dmul_rn(db, ds)));
    yb = __double2float_rn(__dadd_rn(__dmul_rn(db, dc), __dmul_rn(da, ds)));
}

// Two bf16 magnitudes' maximum, twice (signs are not defined); a NaN stays one.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The same, but of a number and a NaN the number.
__device__ __forceinline__ uint32_t max_abs_number_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The least magnitude of two.
__device__ __forceinline__ uint32_t min_abs_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Whether a magnitude of `low` is below 2^-20, or one of `big` an infinity or a NaN.
__device__ __forceinline__ bool not_within_bf16x2(uint32_t low, uint32_t big) {
    uint32_t d;
    asm("{\n\t.reg .pred p, q, r, s;\n\t.reg .b32 l, b;\n\tabs.bf16x2 l, %1;\n\tabs.bf16x2 b, %2;\n\t"
        "setp.lt.bf16x2 p|q, l, %3;\n\tsetp.geu.bf16x2 r|s, b, %4;\n\t"
        "or.pred p, p, q;\n\tor.pred r, r, s;\n\tor.pred p, p, r;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(d)
        : "r"(low), "r"(big), "r"(0x35803580u), "r"(0x7F807F80u));
    return d != 0;
}

// Pairs 2i, 2i + 1 of the lane, from its two chunks' words: a, b the pairs' first and second values.
template <bool kAdjacent>
__device__ __forceinline__ void unpack_pairs(uint32_t u, uint32_t v, float2 &a, float2 &b) {
    if (kAdjacent) {  // two words of a chunk
        a = make_float2(bf16_lo(u), bf16_lo(v));
        b = make_float2(bf16_hi(u), bf16_hi(v));
    } else {          // a word of each chunk
        a = make_float2(bf16_lo(u), bf16_hi(u));
        b = make_float2(bf16_lo(v), bf16_hi(v));
    }
}

// Rotates the lane's eight pairs: wa, wb the rotated first and second values, in bf16.
template <bool kAdjacent>
__device__ __forceinline__ void rotate_pairs(const RopeTrig &g, const uint32_t (&w0)[4], const uint32_t (&w1)[4],
                                             uint32_t (&wa)[4], uint32_t (&wb)[4]) {
    auto word = [&](int i, bool second) {
        if (!kAdjacent) return second ? w1[i] : w0[i];
        return i < 2 ? w0[2 * i + second] : w1[2 * (i - 2) + second];
    };
    uint32_t near[4];  // least distance from a bf16 border, per half, offset to 0..8
    uint32_t big = 0, low = 0;  // largest magnitude; least of the pairs' larger ones
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 c = g.c[i], s = g.s[i], ns = make_float2(-s.x, -s.y);
        float2 a, b;
        unpack_pairs<kAdjacent>(word(i, false), word(i, true), a, b);
        // x_a c - x_b s: np = -fl(x_b s); fma(x_b, s, np) is what fl() lost.
        const float2 np = fmul2(b, ns);
        const float2 ya = fsub2(ffma2(a, c, np), ffma2(b, s, np));
        // x_b c + x_a s: p = fl(x_a s); fma(x_a, -s, p) is -(what fl() lost).
        const float2 p = fmul2(a, s);
        const float2 yb = fsub2(ffma2(b, c, p), ffma2(a, ns, p));
        const uint32_t na = __vadd2(__byte_perm(__float_as_uint(ya.x), __float_as_uint(ya.y), 0x5410), 0x80048004u);
        near[i] = __viaddmin_u16x2(__byte_perm(__float_as_uint(yb.x), __float_as_uint(yb.y), 0x5410), 0x80048004u, na);
        wa[i] = pack_bf16(ya.x, ya.y);
        wb[i] = pack_bf16(yb.x, yb.y);
        const uint32_t top = max_abs_bf16x2(wa[i], wb[i]);
        big = i == 0 ? top : max_abs_bf16x2(top, big);
        low = i == 0 ? top : min_abs_bf16x2(top, low);
    }
    // (A result that is not finite in fp32 is not in bf16 either.)
    const bool odd = not_within_bf16x2(low, big);
    const uint32_t least = __vminu2(__vminu2(near[0], near[1]), __vminu2(near[2], near[3]));
    if (odd || (least & 0xFFFFu) <= 8u || (least >> 16) <= 8u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!odd && (near[i] & 0xFFFFu) > 8u && (near[i] >> 16) > 8u) continue;
            // Unpacked anew: held for this seldom path, the values would take 16 registers.
            uint32_t u = word(i, false), v = word(i, true);
            asm volatile("" : "+r"(u), "+r"(v));
            float2 a, b, ya, yb;
            unpack_pairs<kAdjacent>(u, v, a, b);
            rotate_pair_f64(a.x, b.x, g.c[i].x, g.s[i].x, ya.x, yb.x);
            rotate_pair_f64(a.y, b.y, g.c[i].y, g.s[i].y, ya.y, yb.y);
            wa[i] = pack_bf16(ya.x, ya.y);
            wb[i] = pack_bf16(yb.x, yb.y);
        }
    }
}

// Rotates a row held as rope_chunks() gives it (w0, w1: bf16 words of the lane's
// two chunks) and leaves chunks j and j + 8 in w0, w1. Every lane of the warp
// calls it together.
template <bool kAdjacent>
__device__ __forceinline__ void rope_row(const RopeTrig &g, int nrot, int j, uint32_t (&w0)[4], uint32_t (&w1)[4]) {
    if (g.lo) {
        uint32_t wa[4], wb[4];
        rotate_pairs<kAdjacent>(g, w0, w1, wa, wb);
        if (kAdjacent) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                w0[2 * i] = __byte_perm(wa[i], wb[i], 0x5410);
                w0[2 * i + 1] = __byte_perm(wa[i], wb[i], 0x7632);
                if (g.hi) {  // the second chunk may pass through
                    w1[2 * i] = __byte_perm(wa[i + 2], wb[i + 2], 0x5410);
                    w1[2 * i + 1] = __byte_perm(wa[i + 2], wb[i + 2], 0x7632);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w0[i] = wa[i];
                w1[i] = wb[i];
            }
        }
    }
    __syncwarp();
    if (kAdjacent || nrot == 8) return;
    // Half-split pairs of a part of the head: chunk q sits in slot 0 of lane q
    // (q < nrot), slot 1 of lane q - nrot (q < 2 nrot), or further up among the
    // chunks that pass through. Lane j takes chunks j and j + 8.
    auto find = [&](int q, int &lane, bool &second) {
        if (q < 2 * nrot) {
            second = q >= nrot;
            lane = second ? q - nrot : q;
        } else {
            second = q - 2 * nrot >= 8 - nrot;
            lane = second ? q - 8 : q - nrot;
        }
    };
    const int row = static_cast<int>(threadIdx.x & 24);
    int l0, l1;
    bool s0, s1;
    find(j, l0, s0);
    find(j + 8, l1, s1);
    uint32_t n0[4], n1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a0 = __shfl_sync(0xffffffffu, w0[i], row + l0), a1 = __shfl_sync(0xffffffffu, w1[i], row + l0);
        const uint32_t b0 = __shfl_sync(0xffffffffu, w0[i], row + l1), b1 = __shfl_sync(0xffffffffu, w1[i], row + l1);
        n0[i] = s0 ? a1 : a0;
        n1[i] = s1 ? b1 : b0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w0[i] = n0[i];
        w1[i] = n1[i];
    }
}

// MXFP4 of a row whose lane j holds chunks j and j + 8 (bf16 words), after the
// Hadamard rotation of hadamard128_rows (the same additions in the same order)
// when kHadamard. c0, c1: the two chunks' codes; in lane j = 0, sf: the row's
// four scale bytes. Every lane of the warp calls it together.
template <bool kHadamard>
__device__ __forceinline__ void mxfp4_row8(const uint32_t (&w0)[4], const uint32_t (&w1)[4], int j, uint32_t &c0,
                                           uint32_t &c1, uint32_t &sf) {
    float v0[8], v1[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v0[2 * i] = bf16_lo(w0[i]);
        v0[2 * i + 1] = bf16_hi(w0[i]);
        v1[2 * i] = bf16_lo(w1[i]);
        v1[2 * i + 1] = bf16_hi(w1[i]);
    }
    uint32_t e;  // exponent fields of the two chunks' largest magnitudes
    if (kHadamard) {
        // Two values to an instruction from the second stage on: pairs (2i, 2i + 1).
        float2 u0[4], u1[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u0[i] = make_float2(v0[2 * i] + v0[2 * i + 1], v0[2 * i] - v0[2 * i + 1]);
            u1[i] = make_float2(v1[2 * i] + v1[2 * i + 1], v1[2 * i] - v1[2 * i + 1]);
        }
#pragma unroll
        for (int s = 1; s < 4; s *= 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i & s) continue;
                const float2 a = u0[i], b = u0[i + s], c = u1[i], d = u1[i + s];
                u0[i] = fadd2(a, b);
                u0[i + s] = fsub2(a, b);
                u1[i] = fadd2(c, d);
                u1[i + s] = fsub2(c, d);
            }
        }
#pragma unroll
        for (int m = 1; m < 8; m *= 2) {  // strides 8, 16, 32: the row's other lanes
            const float sgn = (j & m) != 0 ? -1.f : 1.f;  // fma(+-1, v, o) rounds as o - v, v + o
            const float2 sgn2 = make_float2(sgn, sgn);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 o0 = make_float2(__shfl_xor_sync(0xffffffffu, u0[i].x, m), __shfl_xor_sync(0xffffffffu, u0[i].y, m));
                const float2 o1 = make_float2(__shfl_xor_sync(0xffffffffu, u1[i].x, m), __shfl_xor_sync(0xffffffffu, u1[i].y, m));
                u0[i] = ffma2(sgn2, u0[i], o0);
                u1[i] = ffma2(sgn2, u1[i], o1);
            }
        }
        constexpr float kRsqrt128 = 0x1.6a09e6p-4f;
        const float2 r2 = make_float2(kRsqrt128, kRsqrt128);
        uint32_t m0 = 0, m1 = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // stride 64: the lane's two chunks
            const float2 a = fmul2(fadd2(u0[i], u1[i]), r2), b = fmul2(fsub2(u0[i], u1[i]), r2);
            v0[2 * i] = a.x, v0[2 * i + 1] = a.y;
            v1[2 * i] = b.x, v1[2 * i + 1] = b.y;
            m0 = max(m0, max(__float_as_uint(a.x) & 0x7FFFFFFFu, __float_as_uint(a.y) & 0x7FFFFFFFu));
            m1 = max(m1, max(__float_as_uint(b.x) & 0x7FFFFFFFu, __float_as_uint(b.y) & 0x7FFFFFFFu));
        }
        e = (m0 >> 23) | ((m1 >> 23) << 16);
    } else {
        const uint32_t m0 =
            max_abs_bf16x2(max_abs_bf16x2(w0[0], w0[1]), max_abs_bf16x2(w0[2], w0[3])) & 0x7FFF7FFFu;
        const uint32_t m1 =
            max_abs_bf16x2(max_abs_bf16x2(w1[0], w1[1]), max_abs_bf16x2(w1[2], w1[3])) & 0x7FFF7FFFu;
        const uint32_t lo = __byte_perm(m0, m1, 0x5410), hi = __byte_perm(m0, m1, 0x7632);
        e = (__vmaxu2(lo, hi) >> 7) & 0x00FF00FFu;
    }
    e = __vmaxu2(e, __shfl_xor_sync(0xffffffffu, e, 1));
    e = __vmaxu2(e, __shfl_xor_sync(0xffffffffu, e, 2));
    // X = e - 127 - 2, at least -127; f = 2^-X.
    const int X0 = max(static_cast<int>(e & 0xFFFFu) - 129, -127), X1 = max(static_cast<int>(e >> 16) - 129, -127);
    const float f0 = pow2_neg(X0), f1 = pow2_neg(X1);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 a = fmul2(make_float2(v0[i], v0[i + 1]), make_float2(f0, f0));
        const float2 b = fmul2(make_float2(v1[i], v1[i + 1]), make_float2(f1, f1));
        v0[i] = a.x, v0[i + 1] = a.y;
        v1[i] = b.x, v1[i + 1] = b.y;
    }
    c0 = cvt_e2m1x8(v0);
    c1 = cvt_e2m1x8(v1);
    // Lane 0 has groups 0 and 2, lane 4 groups 1 and 3.
    const uint32_t mine = static_cast<uint32_t>(X0 + 127) | (static_cast<uint32_t>(X1 + 127) << 16);
    sf = mine | (__shfl_down_sync(0xffffffffu, mine, 4) << 8);
}

// How a warp takes rows: TS tokens by HS heads at a time (TS * HS = 4), `heads` heads
// (a multiple of HS) of its tokens in all, so that a token's cosines and sines
// are read once for them. (Times here are kernel durations in a profiler's trace.) With 32
// heads or more, one token by four heads: 8 steps use its cosines up, and the table is
// read once for 32 rows (96 us for 32768 tokens of 32 heads; four tokens by one head: 99). With fewer, four tokens by one head, so that a lane's
// cosines still serve a head a step (8192 appended tokens of 8 heads, 4 sequences: 55 us;
// one token by four heads: 64).
struct RopeTiling {
    int hs_log2;        // HS = 1, 2 or 4
    int heads;          // heads of one item
    int head_chunks;    // items over the heads
    int token_groups;   // items over the tokens
};

inline RopeTiling rope_tiling(int B, int tokens, int H) {
    RopeTiling t;
    t.hs_log2 = H >= 32 || tokens == 1 ? 2 : tokens == 2 ? 1 : 0;
    if (H < 3) t.hs_log2 = H - 1 < t.hs_log2 ? H - 1 : t.hs_log2;
    const int hs = 1 << t.hs_log2, ts = 4 >> t.hs_log2;
    t.token_groups = (tokens + ts - 1) / ts;
    // Up to 8 steps over the heads an item, fewer while the items would not give every SM
    // 16 warps, two thirds of what it holds: with 32 asked for, an item's start (position, then
    // cosines) is paid in two waves of short items (3 x 1601 tokens of 8 heads 13.8 us,
    // here 11.6), with 8 too few warps hide each other's (13.6). (2047 tokens of 64 heads, half of
    // the channels rotated, pay for it: 18.7 us with 32, here 19.2.)
    int steps = 8;
    auto chunks = [&](int s) { return (H + s * hs - 1) / (s * hs); };
    while (steps > 1 && static_cast<int64_t>(B) * t.token_groups * chunks(steps) < 148 * 16) steps >>= 1;
    t.heads = steps * hs;
    t.head_chunks = chunks(steps);
    return t;
}

}  // namespace qk4v8
