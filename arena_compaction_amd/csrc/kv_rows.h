// kv_rows.h -- what the attention kernels share: a sequence's place in the
// call, the running maximum and sums of a softmax over pages, and values that
// are no numbers.
#ifndef ARENA_COMPACTION_KV_ROWS_H
#define ARENA_COMPACTION_KV_ROWS_H
#include "kv_mfma.h"

namespace ac {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
// Weights are kept below 2^kRoom; a new running maximum leaves them below
// 2^kLift, so that it need not follow every small growth.
constexpr float kLift = 13.0f, kRoom = 15.0f;
#define KV_NEG_INF (-__builtin_inff())

// Place of a call's sequence b: its new tokens, and how many tokens it holds.
struct Seq {
    uint64_t first;
    int count, len, had;
};

__device__ inline Seq sequence(const KvAttend &a, uint32_t b, bool *bad) {
    Seq s;
    new_tokens(a.starts, a.tokens, a.max_new, b, &s.first, &s.count, bad);
    s.len = a.c.lens[b];
    if (s.len < 0 || (uint32_t)s.len > a.max_len) {  // as a sequence that holds nothing
        *bad = true;
        s.len = 0;
    }
    s.had = s.len - s.count;
    return s;
}

// Pages that the rows of block rb may see (its last row sees most; under a
// mask any of them may see all).
__device__ inline int block_pages(const KvAttend &a, const Seq &s, int rb, bool masked) {
    if (masked) return (s.len + kKvPage - 1) / kKvPage;
    const int rows = s.count * (int)a.group;
    int last = (rb + 1) * (int)a.rows;
    last = (last < rows ? last : rows) - 1;
    const int see = s.had + last / (int)a.group + 1;
    return see > 0 ? (see + kKvPage - 1) / kKvPage : 0;
}

// Running state of the 16 rows of a tile; a lane holds row lane % 16.
// m is a whole number, so that ev - m is exact, and -infinity before the
// first token; l is this lane's share of the sum.
struct Soft {
    float m, l;
};

// The first n of a lane's 16 tokens as bits.
__device__ inline uint32_t first_bits(int n) { return n >= 16 ? 0xFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }

// What a row sees of the sequence's new tokens: words of its mask.
struct Words {
    uint64_t lo, hi;
};
// Words that hold the bits of the 16 places from `at` on; token: the row's, of
// the call.  (Words behind the row's last one hold no new token's bit.)
__device__ inline Words mask_words(const KvAttend &a, const Seq &s, uint64_t token, int at) {
    const int w = at > s.had ? (at - s.had) / 64 : 0, last = (int)a.mask_words - 1;
    const uint64_t *row = a.mask + token * a.mask_words;
    return Words{row[w < last ? w : last], row[w + 1 < last ? w + 1 : last]};
}
// Bits of these places that the row sees (all before the new tokens).
__device__ inline uint32_t mask_bits(const Words &x, const Seq &s, int at) {
    const int off = at - s.had;
    uint64_t bits = 0xFFFFu;
    if (off >= 0) {
        bits = x.lo >> (off & 63);
        if (off & 63) bits |= x.hi << (64 - (off & 63));
    } else if (off > -16) {
        bits = x.lo << -off | ((1u << -off) - 1u);
    }
    return (uint32_t)bits & first_bits(s.len - at);
}

// Scores (in powers of two) that the row does not see.
__device__ inline void hide(f32x4 (&w)[4], uint32_t bits) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (!((bits >> i) & 1)) w[i / 4][i % 4] = KV_NEG_INF;
}

// Sums over codes w to w * f, capped, + add, in powers of two.  A score goes by
// a form that the cap and its own size choose, so that nothing beside it, seen or
// not, changes a bit of it.
//   c tanh(x) = c - 2 c / (2^(2 x log2(e)) + 1)
// is off by up to 2^-21 of c (the quotient q by 2^-23 of itself, the sum by 2^-24,
// the power by 2^-23 and its exponent by 2^-23, which q (1 - q) <= 1/4 and 0.23
// weigh, all doubled: 2 c (1.5 q + 0.48) 2^-23).  Up to kLowCap that is no more
// than 2^-14 of a weight, beside the 2^-11 that rounding it to float16 costs, and
// every score goes by it.  Above, those from c / 8 on do (there 1.3 * 2^-22 of c,
// less than 2^-18 of the score), and smaller ones are c x + c x^3 (a1 + a2 x^2), with the a that leave least, 2^-27 of the
// score, so that a large cap is none; pages without any from c / 8 on leave the
// exponents out.  (Choosing so under every cap costs a prompt a third: chunks of
// 2000 tokens x 32 heads of 128 under a cap of 30 376 us for 285.)
// (kLowCap is in kv.h: kernels of kCapped know the first form alone.)
template <int MODE>
__device__ inline void cap_scores(const KvAttend &a, f32x4 (&w)[4], float f, float add) {
    if (MODE == kCapped || a.score_cap != 0.0f) {
        // z = 2 x log2(e), so that x = z ln(2) / 2; its factor stays finite, as
        // a sum of 0 is 0 under a small cap over large keys too
        const float c = a.score_cap * kLog2e, top = c + add;
        const float by = __builtin_amdgcn_fmed3f(f * a.cap_by, -__FLT_MAX__, __FLT_MAX__);
        auto large = [&](float z) __attribute__((always_inline)) {
            return __builtin_fmaf(-2.0f * c, __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(z) + 1.0f), top);
        };
        if (MODE == kCapped || a.score_cap <= kLowCap) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i / 4][i % 4] = large(w[i / 4][i % 4] * by);
        } else {
            const float limit = 0.25f * kLog2e, a1 = c * (-0.333327708f * 0.0416280815f), a2 = c * (0.132167363f * 0.00500008430f);
            auto small = [&](float v, float z) __attribute__((always_inline)) {
                const float y = z * z;
                return __builtin_fmaf(__builtin_fmaf(a2, y, a1), y * z, __builtin_fmaf(v, f, add));
            };
            float most = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(w[i / 4][i % 4]));
            if (__builtin_amdgcn_ballot_w64(!(most * fabsf(by) < limit))) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float v = w[i / 4][i % 4], z = v * by;
                    w[i / 4][i % 4] = fabsf(z) < limit ? small(v, z) : large(z);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i / 4][i % 4] = small(w[i / 4][i % 4], w[i / 4][i % 4] * by);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i / 4][i % 4] = __builtin_fmaf(w[i / 4][i % 4], f, add);
    }
}

// The same plus slope * (position of the lane's i-th token - the row's): slope
// is that of the row's head times log2(e); positions are key_pos(i), or where
// there are none the places, from `place` on.
template <typename Pos>
__device__ inline void term_scores(const KvAttend &a, f32x4 (&w)[4], float f, float slope, int row_pos, int place, Pos key_pos,
                                   float add) {
    cap_scores<kTerms>(a, w, f, a.pos ? add : __builtin_fmaf(slope, (float)(place - row_pos), add));
    if (!a.slopes) return;
    if (a.pos) {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i / 4][i % 4] = __builtin_fmaf(slope, (float)(key_pos(i) - row_pos), w[i / 4][i % 4]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i / 4][i % 4] = __builtin_fmaf(slope, (float)i, w[i / 4][i % 4]);
    }
}

// A row's slope, in powers of two, and its position, where there are slopes.
__device__ inline void row_terms(const KvAttend &a, const Seq &s, uint32_t b, uint32_t h, int t, int hg, float &slope, int &pos) {
    slope = 0.0f;
    pos = s.had + t;
    if (!a.slopes) return;
    slope = a.slopes[h * a.group + hg] * kLog2e;
    if (a.pos && pos >= 0) pos = a.pos[((uint64_t)b * a.c.heads + h) * a.pos_cap + pos];
}

// Scores of a page (in w) to exponents, at most kRoom, which replace them:
// make(c) turns them to score + c, c = ev - m, and hides what is not seen.
// Returns what the row's earlier sums are to be multiplied by (1 almost
// always: the maximum moves only when an exponent would pass kRoom).
template <typename Make>
__device__ inline float soft_step(Soft &s, f32x4 (&w)[4], int ei, Make make) {
    const bool first = s.m == KV_NEG_INF;
    float top = KV_NEG_INF;
    make((float)ei - (first ? 0.0f : s.m));
#pragma unroll
    for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, w[tt][i]);
    float fade = 1.0f;
    if (__builtin_amdgcn_ballot_w64(top > (first ? KV_NEG_INF : kRoom))) {
        top = across_groups(top, [](float x, float y) { return fmaxf(x, y); });
        if (top > (first ? KV_NEG_INF : kRoom)) {
            const float by = ceilf(top) - kLift;
            fade = first ? 0.0f : __builtin_amdgcn_exp2f(-by);
            s.m = first ? by : s.m + by;
            s.l *= fade;
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                for (int i = 0; i < 4; ++i) w[tt][i] -= by;
        }
    }
    return fade;
}

// The same for sums over codes, which f scales.  `see`: how many of the lane's
// 16 tokens the row sees, or with BITS which, looked at where `edge` says that
// some row misses some.
template <bool BITS = false>
__device__ inline float soft_scores(Soft &s, f32x4 (&w)[4], float f, int ei, bool edge, int see) {
    return soft_step(s, w, ei, [&](float c) __attribute__((always_inline)) {
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[tt][i] = __builtin_fmaf(w[tt][i], f, c);
        if (__builtin_expect(edge, 0)) {
            if constexpr (BITS) {
                hide(w, (uint32_t)see);
            } else {
#pragma unroll
                for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (tt * 4 + i >= see) w[tt][i] = KV_NEG_INF;
            }
        }
    });
}

// Weights of 8 of the lane's tokens as the operand of a product over 32
// tokens, from the exponents of two tiles; adds the weights' sum to `sum`.
__device__ inline u32x4 soft_weights(const f32x4 &w0, const f32x4 &w1, float &sum) {
    float e[8];
    u32x4 p;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        e[i] = __builtin_amdgcn_exp2f(i < 4 ? w0[i] : w1[i - 4]);
        sum += e[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = pack2<kFp16>(e[2 * i], e[2 * i + 1]);
    return p;
}

// float16 rounds a weight by up to 2^-11, an eighth of what an output in
// bfloat16 is rounded by; beside one in float16 it would show (errors half as
// large again).  There the weights are summed twice, as they were and as they
// were rounded, and the result is multiplied by the sums' quotient: of each
// weight's rounding only what differs from their mean is left: nothing where
// one weight makes the result, most of it where a few alike do, little where
// many do (errors against 64 bits 2.5e-4 over 8200 tokens x 32 heads of 64,
// 2.1e-4 from 32-bit weights; carrying the rest of each weight as a second
// operand left none, for a sixth more time).  Both sums are
// of 2^(t - m) with the value scale in it, so that pages count by what they add.
template <int DTYPE>
struct Rounding {
    __device__ void add(const u32x4 &) {}
    __device__ void add_exact(float) {}
    __device__ void fade(float) {}
    __device__ float factor() const { return 1.0f; }
};
template <>
struct Rounding<kFp16> {
    float exact = 0.0f, rounded = 0.0f;  // this lane's shares
    __device__ void add(const u32x4 &p) {
        const half2v ones = {(_Float16)1.0f, (_Float16)1.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t two = p[i];
            rounded = __builtin_amdgcn_fdot2(__builtin_bit_cast(half2v, two), ones, rounded, false);
        }
    }
    __device__ void add_exact(float sum) { exact += sum; }
    __device__ void fade(float f) {
        exact *= f;
        rounded *= f;
    }
    __device__ float factor() const {
        const auto plus = [](float x, float y) { return x + y; };
        const float all = across_groups(exact, plus), all_rounded = across_groups(rounded, plus);
        return all_rounded == 0.0f ? 1.0f : all / all_rounded;
    }
};

// Exponent of a page's value scale (a page never written may hold a scale of
// 0: its 2^-ei must stay finite).
__device__ inline int value_exp(float scale) {
    const int e = exp_of_pow2(scale);
    return e < -100 ? -100 : e;
}

// A running maximum holds for pages whose value scales are at most 2^kBand
// apart; pages are taken by such bands, from the smallest scales up.  A larger
// scale that comes later makes the earlier sums fade in 32 bits, where nothing
// is lost; the other way round it would leave the later weights below what
// float16 holds.  A page's weight is then rounded as if it were at least
// 2^(kBand - 38) of the row's sum.  Most caches are one band, seen by a ballot.
constexpr int kBand = 8;
constexpr int kNoExp = 1 << 20;  // of a page that is none: above every exponent
__device__ inline int least_of(int e) {
    return wave_reduce(e, [](int x, int y) { return x < y ? x : y; });
}
__device__ inline int most_of(int e) {
    return wave_reduce(e, [](int x, int y) { return x > y ? x : y; });
}

// Codes of four tokens from place k on, of which the first `there` are the
// cache's own; the others may hold no numbers and become 0.
__device__ inline uint32_t only_there(uint32_t codes, int there) {
    return there >= 4 ? codes : there <= 0 ? 0u : codes & ((1u << (8 * there)) - 1u);
}

// Puts a NaN into the sums of the rows that see a token whose value is NaN:
// sums over a page's tokens of (the row sees it) x (its value is NaN).
// values: the lane's first value code of the page; see: for each row tile,
// which of the lane's 16 tokens its row sees.
template <int D, int R>
__device__ inline void put_nan(const uint8_t *values, const uint32_t (&see)[R], f32x4 (&o)[R][D / 16]) {
    u32x4 sees[R][2];
#pragma unroll
    for (int rt = 0; rt < R; ++rt)
#pragma unroll
        for (int x = 0; x < 8; ++x)
            sees[rt][x / 4][x % 4] = (see[rt] >> (2 * x) & 1u) * 0x3C00u | (see[rt] >> (2 * x + 1) & 1u) * 0x3C000000u;
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(values + dt * 16 * kKvPage);
        uint32_t one[4];  // 0x38 is the code of 1
#pragma unroll
        for (int x = 0; x < 4; ++x) one[x] = (nan_codes(v[x]) >> 7) * 0x38u;
#pragma unroll
        for (int rt = 0; rt < R; ++rt) {
            f32x4 hit = {0, 0, 0, 0};
            hit = mfma16<kFp16>(widen8<kE4m3, kFp16>(one[0], one[1]), sees[rt][0], hit);
            hit = mfma16<kFp16>(widen8<kE4m3, kFp16>(one[2], one[3]), sees[rt][1], hit);
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (hit[x] > 0.0f) o[rt][dt][x] = __builtin_nanf("");
        }
    }
}

// Queries of a wave's row tiles and how many tokens each row sees (none for a
// row that is not there).
template <int D, int R>
__device__ inline void load_rows(const KvAttend &a, const Seq &s, uint32_t h, int first, int lane,
                                 u32x4 (&q)[R][D / 32], int (&lim)[R]) {
    const int n = lane % 16, g = lane / 16, G = (int)a.group;
#pragma unroll
    for (int rt = 0; rt < R; ++rt) {
        const int r = first + rt * 16 + n;
        const bool real = r < s.count * G;
        const int t = real ? r / G : 0, hg = real ? r % G : 0;
        lim[rt] = real ? s.had + t + 1 : 0;
        const uint16_t *p = a.q + (int64_t)(s.first + t) * a.q_row + (int64_t)(h * G + hg) * a.q_head;
#pragma unroll
        for (int st = 0; st < D / 32; ++st) {
            q[rt][st] = u32x4{0, 0, 0, 0};
            if (real) q[rt][st] = load_q8(p + dim_of<D>(st, g));
        }
    }
}

// Logarithm and inverse of a row's sum, where they are asked for.
__device__ inline void put_sum(const KvAttend &a, uint64_t row, float m, float l) {
    if (a.lse) a.lse[row] = l == 0.0f ? KV_NEG_INF : (m + log2f(l)) * kLn2;
    if (a.sums) a.sums[row] = make_float2(m, l == 0.0f ? 0.0f : 1.0f / l);
}

}  // namespace
}  // namespace ac

#endif
