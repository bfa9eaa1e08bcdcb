// kv_turn.h -- the position rotation of keys and queries.
//
// Pair i of a token at position p turns by the angle a = p * f_i:
//   x' = x cos a - y sin a        y' = x sin a + y cos a
// The angle, its sine and its cosine are made in 64 bits: in 32 an angle of
// position 100,000 would be off by 2^-8.  Keys stay in 64 bits and are rounded
// once, to their code: beside the border between two codes, or a page's largest
// beside that between two scales, 32 bits would fall on either side.  Queries
// are products in 32 bits, off by up to 2^-22 of the pair's larger number (sine
// and cosine rounded, a product, a sum): little beside the 2^-11 at least that
// their type rounds by, but where the two products cancel it is an absolute
// error that may exceed the small result's own rounding.
//
// The angle is taken in turns, p * (f / 2 pi), of which only the fraction
// counts; a quarter turn more or less swaps sine and cosine, so that their
// series (z - z^3/3! + ..., 1 - z^2/2! + ...) are needed up to pi/4, where what
// follows z^15 and z^16 is below 2^-53.  Some 30 operations a (token, pair): a
// lane does those of 4 pairs, and a workgroup of queries uses them for 8 heads.
#ifndef ARENA_COMPACTION_KV_TURN_H
#define ARENA_COMPACTION_KV_TURN_H
#include "kv_device.h"

namespace ac {
namespace {

// (2-byte alignment will do: gfx950 reads and writes up to 16 bytes anywhere)
__device__ inline u32x4 load8(const uint16_t *p) {
    u32x4 r;
    __builtin_memcpy(&r, p, 16);
    return r;
}

// sin and cos of p * turns whole turns, each divided by 4.
__device__ inline void quarter_sin_cos(double turns, int p, double &s, double &c) {
    double u = turns * (double)p;
    u -= __builtin_rint(u);
    const double q = __builtin_rint(4.0 * u);
    const double z = __builtin_fma(-0.25, q, u) * 6.283185307179586;
    const double y = z * z;
    double ps = -0.25 / 1307674368000.0, pc = 0.25 / 20922789888000.0;
    ps = __builtin_fma(ps, y, 0.25 / 6227020800.0);
    pc = __builtin_fma(pc, y, -0.25 / 87178291200.0);
    ps = __builtin_fma(ps, y, -0.25 / 39916800.0);
    pc = __builtin_fma(pc, y, 0.25 / 479001600.0);
    ps = __builtin_fma(ps, y, 0.25 / 362880.0);
    pc = __builtin_fma(pc, y, -0.25 / 3628800.0);
    ps = __builtin_fma(ps, y, -0.25 / 5040.0);
    pc = __builtin_fma(pc, y, 0.25 / 40320.0);
    ps = __builtin_fma(ps, y, 0.25 / 120.0);
    pc = __builtin_fma(pc, y, -0.25 / 720.0);
    ps = __builtin_fma(ps, y, -0.25 / 6.0);
    pc = __builtin_fma(pc, y, 0.25 / 24.0);
    ps = __builtin_fma(ps, y, 0.25) * z;
    pc = __builtin_fma(pc, y, -0.25 / 2.0);
    pc = __builtin_fma(pc, y, 0.25);
    const int k = (int)q;
    const double ss = k & 1 ? pc : ps, cc = k & 1 ? ps : pc;
    s = k & 2 ? -ss : ss;
    c = (k + 1) & 2 ? -cc : cc;
}

// x as a float32 whose last bit says whether something was cut off: rounding
// that to fewer bits (to nearest, ties to even) gives what rounding x would.
// What lies outside the range becomes its largest number.
__device__ inline float to_odd(double x) {
    const float f = (float)x;
    const double d = (double)f;
    uint32_t b = __builtin_bit_cast(uint32_t, f);
    const uint32_t other = __builtin_fabs(d) < __builtin_fabs(x) ? b + 1 : b - 1;
    b = d != x && !(b & 1) ? other : b;
    return __builtin_bit_cast(float, b);
}

// The 8 dimensions of a lane, the piece-th of a row's: 4 from d0 on and 4 from
// d1 on, which hold 4 pairs, or none.
struct Lane8 {
    int d0, d1;
    bool turns;
    double f[4];  // turns a position
};
__device__ inline Lane8 lane8(const KvRotary &a, int piece) {
    Lane8 r;
    r.turns = piece < (int)a.rotary / 8;
    const bool halves = r.turns && !a.next;
    r.d0 = halves ? 4 * piece : 8 * piece;
    r.d1 = halves ? 4 * piece + (int)a.rotary / 2 : 8 * piece + 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.f[i] = r.turns ? a.freq[4 * piece + i] * 0.15915494309189535 : 0.0;  // 1 / (2 pi)
    return r;
}

__device__ inline u32x4 load_pairs(const uint16_t *row, const Lane8 &at) {
    u32x2 x, y;
    __builtin_memcpy(&x, row + at.d0, 8);
    __builtin_memcpy(&y, row + at.d1, 8);
    return u32x4{x[0], x[1], y[0], y[1]};
}

// The lane's 8 numbers x as 4 pairs, first in the low half.
__device__ inline void pairs_of(const u32x4 &x, bool next, uint32_t (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = x[i / 2], hi = x[2 + i / 2];
        const uint32_t halves = i % 2 ? lo >> 16 | (hi & 0xFFFF0000u) : (lo & 0xFFFFu) | hi << 16;
        w[i] = next ? x[i] : halves;
    }
}
// Two results a pair in the order of x.
__device__ inline void unpair(const float (&first)[4], const float (&second)[4], bool next, float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[i] = next ? (i % 2 ? second[i / 2] : first[i / 2]) : first[i];
        y[4 + i] = next ? (i % 2 ? second[2 + i / 2] : first[2 + i / 2]) : second[i];
    }
}

// The lane's 8 numbers turned by the 4 angles, each divided by 4 (so that what
// two numbers of the type's range add up to is still a float32).
template <int DTYPE>
__device__ inline void turn8(const u32x4 &x, bool next, const double (&s)[4], const double (&c)[4], float (&y)[8]) {
    uint32_t w[4];
    float first[4], second[4];
    pairs_of(x, next, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double a = (double)to_float<DTYPE>((uint16_t)w[i]), b = (double)to_float<DTYPE>((uint16_t)(w[i] >> 16));
        first[i] = to_odd(__builtin_fma(a, c[i], -(b * s[i])));
        second[i] = to_odd(__builtin_fma(a, s[i], b * c[i]));
    }
    unpair(first, second, next, y);
}

template <int DTYPE>
__device__ inline void turn_lane(const u32x4 &x, const KvRotary &a, const Lane8 &at, int p, float (&y)[8]) {
    if (at.turns) {
        double s[4], c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) quarter_sin_cos(at.f[i], p, s[i], c[i]);
        turn8<DTYPE>(x, a.next, s, c, y);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = 0.25f * to_float<DTYPE>((uint16_t)(x[i / 2] >> (16 * (i % 2))));
    }
}

// Position of a sequence's number-th new token, whose first one's is `first`
// where they are not given one by one.
__device__ inline int token_position(const KvRotary &a, int first, int64_t token, int64_t number) {
    return a.token_pos ? a.token_pos[token] : (int)((uint32_t)first + (uint32_t)number);
}

// Turns the queries of count tokens, from `token` on (the number-th new one of
// its sequence), for up to kRotaryHeads heads.  A lane takes 8 dimensions of a
// token in every head; where there are fewer tokens than the lanes could take,
// the heads are dealt out too.
template <int D, int DTYPE>
__device__ inline void turn_queries(const KvRotary &a, int lanes, uint32_t head, int first, int64_t token, int count, int64_t number) {
    constexpr int kPer = D / 8, kAhead = 4;
    const int slots = lanes / kPer, slot = threadIdx.x / kPer, tokens = count < slots ? count : slots, deal = slots / tokens;
    const int left = (int)(a.q_heads - head), heads = left < (int)kRotaryHeads ? left : (int)kRotaryHeads;
    const int mine = slot / tokens;
    if (mine >= deal) return;
    const Lane8 at = lane8(a, threadIdx.x % kPer);
    for (int t = slot % tokens; t < count; t += tokens) {
        const int p = token_position(a, first, token + t, number + t);
        const uint16_t *from = a.q + (token + t) * a.q_row + (int64_t)head * a.q_head;
        uint16_t *to = a.q_out + (token + t) * a.o_row + (int64_t)head * a.o_head;
        float s[4], c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            double ss, cc;
            quarter_sin_cos(at.f[i], p, ss, cc);
            s[i] = 4.0f * (float)ss;
            c[i] = 4.0f * (float)cc;
        }
        for (int h0 = mine; h0 < heads; h0 += kAhead * deal) {
            u32x4 x[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {  // behind the last head the last one again
                const int h = h0 + u * deal;
                x[u] = load_pairs(from + (h < heads ? h : heads - 1) * a.q_head, at);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int h = h0 + u * deal;
                if (h >= heads) continue;
                u32x2 w0 = {x[u][0], x[u][1]}, w1 = {x[u][2], x[u][3]};
                if (at.turns) {
                    uint32_t w[4];
                    float one[4], two[4], y[8];
                    pairs_of(x[u], a.next, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float v0 = to_float<DTYPE>((uint16_t)w[i]), v1 = to_float<DTYPE>((uint16_t)(w[i] >> 16));
                        one[i] = __builtin_fmaf(v0, c[i], -(v1 * s[i]));
                        two[i] = __builtin_fmaf(v0, s[i], v1 * c[i]);
                    }
                    unpair(one, two, a.next, y);
                    w0 = u32x2{pack2<DTYPE>(y[0], y[1]), pack2<DTYPE>(y[2], y[3])};
                    w1 = u32x2{pack2<DTYPE>(y[4], y[5]), pack2<DTYPE>(y[6], y[7])};
                }
                __builtin_memcpy(to + h * a.o_head + at.d0, &w0, 8);
                __builtin_memcpy(to + h * a.o_head + at.d1, &w1, 8);
            }
        }
    }
}

}  // namespace
}  // namespace ac

#endif
