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

// Pages that the rows of block rb may see (its last row sees most).
__device__ inline int block_pages(const KvAttend &a, const Seq &s, int rb) {
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

// Scores of a page (sums over codes, in w) to exponents f * score + ev - m,
// at most kRoom, which replace them.  `see`: how many of the lane's 16 tokens
// the row sees, looked at where `edge` says that some row misses some.
// Returns what the row's earlier sums are to be multiplied by (1 almost
// always: the maximum moves only when an exponent would pass kRoom).
__device__ inline float soft_scores(Soft &s, f32x4 (&w)[4], float f, int ei, bool edge, int see) {
    const bool first = s.m == KV_NEG_INF;
    const float c = (float)ei - (first ? 0.0f : s.m);
    float top = KV_NEG_INF;
#pragma unroll
    for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[tt][i] = __builtin_fmaf(w[tt][i], f, c);
    if (__builtin_expect(edge, 0)) {
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (tt * 4 + i >= see) w[tt][i] = KV_NEG_INF;
    }
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
// how many of the lane's 16 tokens its row sees.
template <int D, int R>
__device__ inline void put_nan(const uint8_t *values, const int (&see)[R], f32x4 (&o)[R][D / 16]) {
    u32x4 sees[R][2];
#pragma unroll
    for (int rt = 0; rt < R; ++rt)
#pragma unroll
        for (int x = 0; x < 8; ++x)
            sees[rt][x / 4][x % 4] = (2 * x < see[rt] ? 0x3C00u : 0u) | (2 * x + 1 < see[rt] ? 0x3C000000u : 0u);
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
