// kv_few.h -- attention of few new tokens' queries over the 8-bit cache.
//
// For query row r of head h (rows of all the query heads that share h) and
// tokens j it may see, with q.k over key codes, ek and ev the page's scales:
//   s_rj = scale * ek * q_r.k_j        p_rj = exp(s_rj) / sum_j exp(s_rj)
//   out_r = sum_j p_rj * ev * v_j      lse_r = log sum_j exp(s_rj)
//   weight_j += sum_r p_rj             (where asked for)
//
// Everything runs in powers of two, t_rj = log2(e) * s_rj + log2(ev): with
// the value scale inside the exponent, w_rj = 2^(t_rj - m) multiplies value
// codes of any page, and sum_j w_rj / ev is the softmax's sum, one factor a
// page.  m lies 13 to 15 below the running maximum of t: float16 weights then
// reach down to 2^-37 of the largest before they lose their last bit.  With
// the value scale in them that is a reach of w * ev, and a token of small
// values behind one of large values would lose what it gives to dimensions
// where the large ones are 0; pages therefore go by bands of value scales,
// small ones first (kBand in kv_rows.h).
//
// A wave takes whole pages, one at a time, with its own running maximum and
// sums; a page's codes are loaded while the page before it is summed, keys
// into the registers its scores have freed, values into those its sums have.
// Scores come out of the matrix instruction transposed (tokens x rows), so
// that a lane holds 16 tokens of one row: the maximum needs two steps across
// lanes, the rescaling none, and the weights are the next product's operand
// where they are.  Four waves share a workgroup's rows and join through LDS;
// workgroups split a long cache and k_kv_finish joins their parts.
//
// It is bound by the cache's bytes: two documents of 131,000 tokens x 8 heads
// of 128 (510 MB) take 96 us, 5.3 TB/s, where a reduction over 4 GiB reads 5.9;
// a ragged batch of 64 x 4096 x 8 heads (296 MB) 61 us, 4.9 TB/s.
//
// Terms (kv_rows.h) add a few instructions a score, which the loads hide, and
// registers: a cap over 64 x 4096 x 4 heads of 256 takes 72 us where none takes
// 70; a bias with positions of 48 x 8000 x 8 heads of 128, with weights (536
// MB), 127 us and a join of 19 (two waves a SIMD, where three without terms;
// three with 19 registers in memory took 155 for 140).
#ifndef ARENA_COMPACTION_KV_FEW_H
#define ARENA_COMPACTION_KV_FEW_H
#include "kv_rows.h"

namespace ac {
namespace {

// Waves of a SIMD that share its registers: 3 where a page's codes and the
// sums of 16 rows fit a third of them.
template <int D, int DTYPE, int R, bool KEEP, int MODE>
constexpr int kWavesASimd = D > 128 ? 1 : R == 1 && !(D == 128 && ((DTYPE == kFp16 && KEEP) || MODE == kTerms)) ? 3 : 2;

// KEEP: scores are kept for the weights.  MODE: kPlain, kMasked or kTerms.
template <int D, int CODES, int DTYPE, int R, bool KEEP, int MODE>
__global__ __launch_bounds__(kThreads, (kWavesASimd<D, DTYPE, R, KEEP, MODE>)) void k_kv_attend(KvAttend a) {
    constexpr int kSteps = D / 32, kTiles = D / 16, kRows = 16 * R, kJoin = 4;
    __shared__ f32x4 sm_o[kWaves][R * kJoin * 64];
    __shared__ float sm_m[kWaves][kRows], sm_l[kWaves][kRows];
    __shared__ int sm_pos[MODE == kTerms ? kWaves : 1][MODE == kTerms ? kKvPage : 1];
    const int split = blockIdx.x % a.splits, rb = blockIdx.x / a.splits;
    const uint32_t h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, wave = wave_uniform(tid / 64), lane = tid % 64;
    const int n = lane % 16, g = lane / 16, G = (int)a.group;
    bool bad;
    const Seq s = sequence(a, b, &bad);
    if (bad && a.c.n_invalid && blockIdx.x == 0 && h == 0 && tid == 0) atomicAdd(a.c.n_invalid, 1ull);
    const int rows = s.count * G;
    if (rb * kRows >= rows) return;
    const bool masked = MODE != kPlain && a.mask != nullptr;
    const int pages = block_pages(a, s, rb, masked);
    const int per = (int)a.per_split;
    const int active = pages > per ? (pages + per - 1) / per : 1;
    if (split >= active) return;
    const int p_lo = split * per, p_hi = p_lo + per < pages ? p_lo + per : pages;
    const bool counts = a.c.n_invalid && h == 0 && (rb + 1) * kRows >= rows && lane == 0;  // once a page

    u32x4 q[R][kSteps];
    int lim[R];
    load_rows<D, R>(a, s, h, rb * kRows, lane, q, lim);
    // of the block's first row, or under a mask of any
    const int see_least = masked ? s.had : s.had + rb * kRows / G + 1;
    [[maybe_unused]] float slope[R];
    [[maybe_unused]] int row_pos[R];
    if constexpr (MODE == kTerms) {
#pragma unroll
        for (int rt = 0; rt < R; ++rt) {
            const int r = rb * kRows + rt * 16 + n < rows ? rb * kRows + rt * 16 + n : 0;
            row_terms(a, s, b, h, r / G, r % G, slope[rt], row_pos[rt]);
        }
    }
    // which of the lane's 16 tokens of the page from `base` on a row sees
    auto seen = [&](int rt, int base) __attribute__((always_inline)) {
        const int at = base + g * 16;
        if (!masked) return first_bits(lim[rt] - at);
        const int r = rb * kRows + rt * 16 + n;
        const uint32_t bits = mask_bits(mask_words(a, s, s.first + (r < rows ? r / G : 0), at), s, at);
        return r < rows ? bits : 0u;
    };
    f32x4 o[R][kTiles];
    Soft soft[R];
    Rounding<DTYPE> rounding[R];
#pragma unroll
    for (int rt = 0; rt < R; ++rt) {
        soft[rt] = Soft{KV_NEG_INF, 0.0f};
#pragma unroll
        for (int dt = 0; dt < kTiles; ++dt) o[rt][dt] = f32x4{0, 0, 0, 0};
    }

    // this wave's pages, every fourth: lane i keeps the i-th one's offset and
    // scales, so that the loop waits for neither
    const int np = p_hi - p_lo > wave ? (p_hi - p_lo - wave + kWaves - 1) / kWaves : 0;
    const uint64_t off = lane < np ? page_offset(a.c, b, p_lo + wave + kWaves * lane) : kNoPage;
    const uint64_t good = __builtin_amdgcn_ballot_w64(off != kNoPage);
    f32x2 scales = {0, 0};
    if (off != kNoPage) scales = *reinterpret_cast<const f32x2 *>(page_scales(a.c, a.c.arena + off, h));
    if (counts && np) {
        const int none = np - __builtin_popcountll(good);
        if (none) atomicAdd(a.c.n_invalid, (unsigned long long)none);
    }
    const uint8_t *strips = a.c.arena + (uint64_t)h * 2 * kKvPage * D;
    uint32_t kraw[4][D / 16];
    u32x4 vraw[kTiles];
    // position of the page's token `lane`, dealt out through LDS, each wave's
    // own (where there are none, what is at hand instead: loads are never under
    // a condition)
    [[maybe_unused]] int key_pos = 0;
    auto get_keys = [&](int i) __attribute__((always_inline)) {
        const uint8_t *strip = strips + lane_u64(off, i);
        load_keys<D>(strip, lane, kraw);
        if constexpr (MODE == kTerms) {
            const uint64_t at = ((uint64_t)b * a.c.heads + h) * a.pos_cap + (uint64_t)(p_lo + wave + kWaves * i) * kKvPage;
            key_pos = (a.pos && a.slopes ? a.pos + at : reinterpret_cast<const int32_t *>(strip))[lane];
        }
    };
    auto get_values = [&](int i) {
        const uint8_t *from = strips + lane_u64(off, i) + kKvPage * D + n * kKvPage + g * 16;
#pragma unroll
        for (int dt = 0; dt < kTiles; ++dt) vraw[dt] = *reinterpret_cast<const u32x4 *>(from + dt * 16 * kKvPage);
    };
    // positions of the set bits of `good` are the pages that are there; of
    // `todo` those of the band under way, of `later` the bands above it
    uint64_t todo = 0, later = good;
    uint32_t no_numbers = 0;
    if (good) {
        get_keys(__builtin_ctzll(good));
        get_values(__builtin_ctzll(good));
    }
    arrived(scales[0]);
    arrived(scales[1]);
    auto next_band = [&]() __attribute__((always_inline)) {
        const int left = (later >> lane) & 1 ? value_exp(scales[1]) : kNoExp;
        todo = later & __builtin_amdgcn_ballot_w64(left <= least_of(left) + kBand);
        later &= ~todo;
    };
    const int near = value_exp(scales[1]) - value_exp(lane_f32(scales[1], good ? __builtin_ctzll(good) : 0)) + kBand / 2;
    if (good & __builtin_amdgcn_ballot_w64(near < 0 || near > kBand)) {
        next_band();
        get_keys(__builtin_ctzll(todo));
        get_values(__builtin_ctzll(todo));
    } else {  // one band
        todo = good;
        later = 0;
    }
    while (todo) {
        const int i = __builtin_ctzll(todo);
        todo &= todo - 1;
        if (!todo && later) next_band();
        // the last page is loaded once more: loads under a condition would be
        // waited for as if they had not been issued, all of them at once
        const int next = todo ? __builtin_ctzll(todo) : i;
        const int base = (p_lo + wave + kWaves * i) * kKvPage;
        const float f = a.scale * kLog2e * lane_f32(scales[0], i);
        const int ei = value_exp(lane_f32(scales[1], i));
        f32x4 w[R][4];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
            for (int rt = 0; rt < R; ++rt) w[rt][tt] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                const u32x4 kk = widen8<CODES, DTYPE>(kraw[tt][2 * st], kraw[tt][2 * st + 1]);
#pragma unroll
                for (int rt = 0; rt < R; ++rt) w[rt][tt] = mfma16<DTYPE>(kk, q[rt][st], w[rt][tt]);
            }
        }
        const bool edge = base + kKvPage > see_least;
        [[maybe_unused]] uint32_t bits[R];
        if constexpr (MODE != kPlain) {
#pragma unroll
            for (int rt = 0; rt < R; ++rt) bits[rt] = 0xFFFFu;
            if (edge) {
#pragma unroll
                for (int rt = 0; rt < R; ++rt) bits[rt] = seen(rt, base);
            }
        }
        // sums to scores + c
        [[maybe_unused]] auto terms = [&](int rt, float c) __attribute__((always_inline)) {
            term_scores(a, w[rt], f, slope[rt], row_pos[rt], base + g * 16, [&](int x) { return sm_pos[wave][g * 16 + x]; }, c);
            if (edge) hide(w[rt], bits[rt]);
        };
        if constexpr (MODE == kTerms) {
            sm_pos[wave][lane] = key_pos;
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
        constexpr bool kDone = MODE != kPlain && KEEP;  // w holds scores of what is seen
        if constexpr (kDone && MODE == kTerms) {
            terms(0, 0.0f);
        } else if constexpr (kDone) {
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) w[0][tt] = w[0][tt] * f;
            if (edge) hide(w[0], bits[0]);
        }
        // (the terms that are not kept are made below; the next page's
        // positions would overwrite this one's)
        [[maybe_unused]] float fades[R];
        if constexpr (MODE == kTerms && !KEEP) {
#pragma unroll
            for (int rt = 0; rt < R; ++rt)
                fades[rt] = soft_step(soft[rt], w[rt], ei, [&](float c) __attribute__((always_inline)) { terms(rt, c); });
        }
        get_keys(next);
        if constexpr (KEEP) {
            float *to = a.scores + ((uint64_t)b * a.c.heads + h) * a.score_pages * a.score_rows * kKvPage;
            to += (uint64_t)(p_lo + wave + kWaves * i) * a.score_rows * kKvPage;
            if (n < rows) {  // one row block of one tile
#pragma unroll
                for (int tt = 0; tt < 4; ++tt)
                    *reinterpret_cast<f32x4 *>(to + ((tt * 4 + g) * (int)a.score_rows + n) * 4) = kDone ? w[0][tt] : w[0][tt] * f;
            }
        }
        u32x4 pw[R][2];
#pragma unroll
        for (int rt = 0; rt < R; ++rt) {
            float fade;
            if constexpr (MODE == kTerms && !KEEP)
                fade = fades[rt];
            else if constexpr (kDone)
                fade = soft_scores(soft[rt], w[rt], 1.0f, ei, false, 0);
            else if constexpr (MODE == kMasked)
                fade = soft_scores<true>(soft[rt], w[rt], f, ei, edge, (int)bits[rt]);
            else
                fade = soft_scores(soft[rt], w[rt], f, ei, edge, lim[rt] - base - g * 16);
            float sum = 0.0f;
            pw[rt][0] = soft_weights(w[rt][0], w[rt][1], sum);
            pw[rt][1] = soft_weights(w[rt][2], w[rt][3], sum);
            soft[rt].l = __builtin_fmaf(sum, pow2(-ei), soft[rt].l);
            if (__builtin_amdgcn_ballot_w64(fade != 1.0f)) {
#pragma unroll
                for (int dt = 0; dt < kTiles; ++dt)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[rt][dt][x] *= fade;
                rounding[rt].fade(fade);
            }
            rounding[rt].add(pw[rt][0]);
            rounding[rt].add(pw[rt][1]);
            rounding[rt].add_exact(sum);
        }
        if (base + kKvPage > s.len) {
#pragma unroll
            for (int dt = 0; dt < kTiles; ++dt)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    vraw[dt][x] = only_there(vraw[dt][x], s.len - base - g * 16 - 4 * x);
        }
        if constexpr (CODES == kE4m3) {
            // a value that is no number must not reach rows that do not see
            // its token (their weight is 0, and 0 x NaN is NaN): left out
            // here, it is put in below for the rows that see it
            if (edge) {
#pragma unroll
                for (int dt = 0; dt < kTiles; ++dt)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t no = nan_codes(vraw[dt][x]);
                        vraw[dt][x] &= ~((no >> 7) * 255u);
                        no_numbers |= no;
                    }
            }
        }
#pragma unroll
        for (int dt = 0; dt < kTiles; ++dt) {
            const u32x4 v0 = widen8<CODES, kFp16>(vraw[dt][0], vraw[dt][1]);
            const u32x4 v1 = widen8<CODES, kFp16>(vraw[dt][2], vraw[dt][3]);
#pragma unroll
            for (int rt = 0; rt < R; ++rt) {
                o[rt][dt] = mfma16<kFp16>(v0, pw[rt][0], o[rt][dt]);
                o[rt][dt] = mfma16<kFp16>(v1, pw[rt][1], o[rt][dt]);
            }
        }
        get_values(next);
    }
    if constexpr (CODES == kE4m3) {
        if (__builtin_amdgcn_ballot_w64(no_numbers != 0)) {
            for (todo = good; todo; todo &= todo - 1) {
                const int i = __builtin_ctzll(todo), base = (p_lo + wave + kWaves * i) * kKvPage;
                if (base + kKvPage <= see_least) continue;
                uint32_t see[R];
#pragma unroll
                for (int rt = 0; rt < R; ++rt) see[rt] = seen(rt, base);
                put_nan<D, R>(strips + lane_u64(off, i) + kKvPage * D + n * kKvPage + g * 16, see, o);
            }
        }
    }

    // join the four waves
#pragma unroll
    for (int rt = 0; rt < R; ++rt) {
        const float sum = across_groups(soft[rt].l, [](float x, float y) { return x + y; });
        if (g == 0) {
            sm_m[wave][rt * 16 + n] = soft[rt].m;
            sm_l[wave][rt * 16 + n] = sum;
        }
    }
    __syncthreads();
    const uint64_t heads = (uint64_t)a.c.heads * G, all = a.tokens * heads;
#pragma unroll
    for (int rt = 0; rt < R; ++rt) {
        const int x = rt * 16 + n;
        float top = fmaxf(fmaxf(sm_m[0][x], sm_m[1][x]), fmaxf(sm_m[2][x], sm_m[3][x]));
        if (top == KV_NEG_INF) top = 0.0f;
        const float fade = __builtin_amdgcn_exp2f(soft[rt].m - top) * rounding[rt].factor();
#pragma unroll
        for (int dt = 0; dt < kTiles; ++dt)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[rt][dt][i] *= fade;
    }
    for (int d0 = 0; d0 < kTiles; d0 += kJoin) {
        if (d0) __syncthreads();
#pragma unroll
        for (int dt = 0; dt < kTiles; ++dt) {
            if (dt >= d0 && dt < d0 + kJoin) {
#pragma unroll
                for (int rt = 0; rt < R; ++rt) sm_o[wave][(rt * kJoin + dt - d0) * 64 + lane] = o[rt][dt];
            }
        }
        __syncthreads();
        for (int e = tid; e < R * kJoin * 64; e += kThreads) {
            const int rt = e / (kJoin * 64), dt = d0 + e / 64 % kJoin;
            const int x = rt * 16 + n, r = rb * kRows + x;
            if (r >= rows || dt >= kTiles) continue;
            float mm[kWaves], top = KV_NEG_INF, sum = 0.0f;
#pragma unroll
            for (int k = 0; k < kWaves; ++k) top = fmaxf(top, mm[k] = sm_m[k][x]);
            const float ts = top == KV_NEG_INF ? 0.0f : top;
#pragma unroll
            for (int k = 0; k < kWaves; ++k) sum += sm_l[k][x] * __builtin_amdgcn_exp2f(mm[k] - ts);
            const f32x4 v = sm_o[0][e] + sm_o[1][e] + sm_o[2][e] + sm_o[3][e];
            const uint64_t row = (s.first + r / G) * heads + (uint64_t)h * G + r % G;
            const int d = dt * 16 + g * 4;
            if (active == 1) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                u32x2 w;
                w[0] = pack2<DTYPE>(v[0] * inv, v[1] * inv);
                w[1] = pack2<DTYPE>(v[2] * inv, v[3] * inv);
                *reinterpret_cast<u32x2 *>(a.out + row * D + d) = w;
                if (d == 0) put_sum(a, row, ts, sum);
            } else {
                *reinterpret_cast<f32x4 *>(a.part + ((uint64_t)split * all + row) * D + d) = v;
                if (d == 0) {
                    float *ml = a.part + (uint64_t)a.splits * all * D + ((uint64_t)split * all + row) * 2;
                    ml[0] = top;
                    ml[1] = sum;
                }
            }
        }
    }
}

template <int MODE, int D, int CODES, int DTYPE>
void attend_go(const KvAttend &a, hipStream_t s) {
    const dim3 grid(a.splits * a.row_blocks, a.c.heads, a.c.batch);
    if constexpr (D <= 128) {
        if (a.rows == 32)
            hipLaunchKernelGGL((k_kv_attend<D, CODES, DTYPE, 2, false, MODE>), grid, dim3(kThreads), 0, s, a);
    }
    if (a.rows == 16 && a.scores)
        hipLaunchKernelGGL((k_kv_attend<D, CODES, DTYPE, 1, true, MODE>), grid, dim3(kThreads), 0, s, a);
    else if (a.rows == 16)
        hipLaunchKernelGGL((k_kv_attend<D, CODES, DTYPE, 1, false, MODE>), grid, dim3(kThreads), 0, s, a);
}

template <int MODE, int D, int CODES>
void attend_dtype(const KvAttend &a, int dtype, hipStream_t s) {
    if (dtype == kBf16)
        attend_go<MODE, D, CODES, kBf16>(a, s);
    else
        attend_go<MODE, D, CODES, kFp16>(a, s);
}

template <int MODE, int D>
void attend_codes(const KvAttend &a, int codes, int dtype, hipStream_t s) {
    if (codes == kE4m3)
        attend_dtype<MODE, D, kE4m3>(a, dtype, s);
    else
        attend_dtype<MODE, D, kInt8>(a, dtype, s);
}

}  // namespace

template <int MODE>
hipError_t launch_kv_few(const KvAttend &a, int codes, int dtype, hipStream_t s) {
    switch (a.c.dim) {
        case 64: attend_codes<MODE, 64>(a, codes, dtype, s); break;
        case 96: attend_codes<MODE, 96>(a, codes, dtype, s); break;
        case 128: attend_codes<MODE, 128>(a, codes, dtype, s); break;
        case 192: attend_codes<MODE, 192>(a, codes, dtype, s); break;
        case 256: attend_codes<MODE, 256>(a, codes, dtype, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace ac

#endif
