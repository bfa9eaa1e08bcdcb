// kv_prompt.h -- attention of many query rows over the 8-bit cache (a
// prompt's tokens, times the heads that share a key/value head).
//
// The mathematics is that of kv_few.h; what differs is who holds what.
// With many rows the cost is the matrix products and, per score, an exponent,
// so a workgroup takes 128 rows, and all its waves go over the same pages:
// each page is loaded once, its codes brought to 16 bits once (a share of the
// page a wave) and put into LDS in the very order in which the matrix
// instructions' operands are read, 16 bytes a lane, in a line.  Two pages are
// in LDS, one being summed and one being filled, while the codes of a third
// are on their way.
//
// What bounds it: the vector pipe (an exponent, a fused product, an addition
// and half a conversion a score) and the matrix pipe, which two waves a SIMD
// overlap only in part.  Chunks of 2000 tokens x 32 heads of 128 behind 2048
// (169 GFLOP) take 211 us, 0.80 PFLOP/s, where a product of 8192 cubed reaches
// 1.26: the matrix pipe is busy for 31% of the cycles, the vector pipe for 37%,
// and 22% are lost to the last rows, which see most.  With 64 dimensions the
// vector pipe is busy for 83% (8200 tokens x 32 heads, float16: 366 us).  (All calls named here in
// turn in one loop; the first after a pause are slower by up to a tenth.)
//
// Terms (kv_rows.h): a page's mask words are loaded a page ahead, one a lane,
// and dealt out where some row misses some token; a wave whose rows see nothing
// of a page only brings the next one to LDS.  A causal mask costs the prompt of
// 8200 tokens 395 us for 366, five documents in it take 144, behind 1 to 63
// tokens 231, as no page is then left out before the first one that is seen; a
// cap costs the chunks above 273 for 211, with the vector pipe busy for 54% of the
// cycles, and above kLowCap 289.  With a distance bias registers leave two waves
// a SIMD for 64 dimensions, where the plain kernel has three: 566 us for 366,
// documents 205 (three, with 60 registers in memory, took an eighth and a quarter more).
//
// Registers go to memory where the type of int8 is bfloat16 (20 of 128 dimensions
// under a cap, 27 under a mask, 98 with all terms; 41 to 107 of 256, the plain
// kernel's 91 among them), in float16 over e4m3 of 256 under a cap (80), and some
// 10 of 256 with any term.
//
// Workgroups of one key/value head run on one XCD where the heads are a
// multiple of 8, so that its pages stay in that XCD's L2; the last rows,
// which see most, start first.
#ifndef ARENA_COMPACTION_KV_PROMPT_H
#define ARENA_COMPACTION_KV_PROMPT_H
#include "kv_rows.h"

namespace ac {
namespace {

// 32 rows a wave; above 128 dimensions 16, whose sums and queries leave two
// waves a SIMD their registers.
template <int D, int ROWS>
constexpr int kPromptWaves = D <= 128 ? ROWS / 32 > 4 ? ROWS / 32 : 4 : 8;

template <int D, int CODES, int DTYPE, int MODE, int ROWS>
__global__ __launch_bounds__((kPromptWaves<D, ROWS>)*64, D == 64 && ((CODES == kE4m3 && DTYPE == kBf16 && MODE == kPlain) || MODE == kMasked) ? 3 : 2) void k_kv_prompt(
    KvAttend a) {
    constexpr int kN = kPromptWaves<D, ROWS>, kRows = ROWS, R = kRows / 16 / kN;
    constexpr int kSteps = D / 32, kTiles = D / 16;
    constexpr int kBatch = kTiles % 4 ? 3 : 4, kBatches = kTiles / kBatch;  // value tiles read at a time
    // a wave's share of a page: of the keys' 4 tiles x chunks of 64 dimensions
    // and of the values' tiles, every kN-th
    constexpr int kChunks = (D + 63) / 64, kKeyJobs = (4 * kChunks + kN - 1) / kN, kValueJobs = (kTiles + kN - 1) / kN;
    __shared__ u32x4 sm_k[2][4 * kSteps * 64], sm_v[2][kTiles * 2 * 64];
    __shared__ int sm_nan;
    __shared__ uint64_t sm_vis[MODE != kPlain ? kN : 1];
    __shared__ int sm_seen[2][MODE != kPlain ? kN : 1];
    __shared__ int sm_pos[MODE == kTerms ? 2 : 1][MODE == kTerms ? kKvPage : 1];  // positions of the pages' tokens
    const uint32_t units = a.c.batch * a.c.heads, block = block_number();
    if (block >= units * a.row_blocks * a.splits) return;
    const uint32_t unit = block % units, piece = block / units;
    const uint32_t b = unit / a.c.heads, h = unit % a.c.heads;
    const int split = piece % a.splits, rb = (int)(a.row_blocks - 1 - piece / a.splits);
    const int tid = threadIdx.x, wave = wave_uniform(tid / 64), lane = tid % 64;
    const int n = lane % 16, g = lane / 16, G = (int)a.group;
    bool bad;
    const Seq s = sequence(a, b, &bad);
    if (bad && a.c.n_invalid && rb == 0 && split == 0 && h == 0 && tid == 0) atomicAdd(a.c.n_invalid, 1ull);
    const int rows = s.count * G;
    if (rb * kRows >= rows) return;
    const bool masked = MODE != kPlain && a.mask != nullptr;
    const int pages = block_pages(a, s, rb, masked);
    const int per = (int)a.per_split;
    const int active = pages > per ? (pages + per - 1) / per : 1;
    if (split >= active) return;
    int p_lo = split * per, p_hi = p_lo + per < pages ? p_lo + per : pages;
    const bool speaks = a.c.n_invalid && h == 0 && (rb + 1) * kRows >= rows;  // once a page
    const bool counts = speaks && !masked && tid == 0;
    if constexpr (MODE != kPlain) {
        if (masked && speaks) {
            for (int p = p_lo + tid; p < p_hi; p += kN * 64)
                if (page_offset(a.c, b, p) == kNoPage) atomicAdd(a.c.n_invalid, 1ull);
        }
        // With few places before the new tokens, the pages from the first to
        // the last that a row of the workgroup sees: of documents packed into
        // a prompt that is one's (8200 tokens, five documents: 230 us without,
        // 221 with).
        if (masked && s.had < kKvPage) {
            const int words = (s.count + 63) / 64, t_first = rb * kRows / G;
            const int t_last = ((rb + 1) * kRows < rows ? (rb + 1) * kRows - 1 : rows - 1) / G;
            int low = 0x7FFFFFFF, high = -1;
            for (int w0 = lane; w0 < words + lane; w0 += 256) {
                uint64_t x[4] = {};  // 4 words and 4 rows at a time, the last ones again
                for (int t0 = t_first + wave; t0 <= t_last; t0 += 4 * kN) {
                    uint64_t y[4][4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int t = t0 + u * kN;
                        const uint64_t *row = a.mask + (s.first + (t <= t_last ? t : t_last)) * a.mask_words;
#pragma unroll
                        for (int v = 0; v < 4; ++v) y[u][v] = row[w0 + v * 64 < words ? w0 + v * 64 : words - 1];
                    }
#pragma unroll
                    for (int v = 0; v < 4; ++v) x[v] |= (y[0][v] | y[1][v]) | (y[2][v] | y[3][v]);
                }
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int w = w0 + v * 64;
                    if (w == words - 1 && s.count % 64) x[v] &= (1ull << s.count % 64) - 1;
                    low = w < words && x[v] && w < low ? w : low;
                    high = w < words && x[v] && w > high ? w : high;
                }
            }
            low = least_of(low);
            high = most_of(high);
            if (lane == 0) {
                sm_seen[0][wave] = low;
                sm_seen[1][wave] = high;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                low = sm_seen[0][k] < low ? sm_seen[0][k] : low;
                high = sm_seen[1][k] > high ? sm_seen[1][k] : high;
            }
            const int64_t from = high < 0 || s.had > 0 ? 0 : s.had + low * 64ll, to = high < 0 ? s.had : s.had + high * 64ll + 64;
            const int first_page = from > 0 ? (int)(from / kKvPage) : 0, end_page = to > 0 ? (int)((to + kKvPage - 1) / kKvPage) : 0;
            p_lo = first_page > p_lo ? first_page : p_lo;
            p_hi = end_page < p_hi ? end_page : p_hi;
        }
    }

    const int first = rb * kRows + wave * 16 * R;  // the wave's rows
    u32x4 q[R][kSteps];
    int lim[R];
    load_rows<D, R>(a, s, h, first, lane, q, lim);
    // what the workgroup's first row sees, and the wave's first and last
    const int block_least = masked ? s.had : s.had + rb * kRows / G + 1, least = masked ? s.had : s.had + first / G + 1;
    const int last = (first + 16 * R < rows ? first + 16 * R : rows) - 1;
    const int most = first >= rows ? 0 : masked ? s.len : s.had + last / G + 1;
    [[maybe_unused]] float slope[R];
    [[maybe_unused]] int row_pos[R];
    if constexpr (MODE == kTerms) {
#pragma unroll
        for (int rt = 0; rt < R; ++rt) {
            const int r = first + rt * 16 + n < rows ? first + rt * 16 + n : 0;
            row_terms(a, s, b, h, r / G, r % G, slope[rt], row_pos[rt]);
        }
    }
    // which of the lane's 16 tokens of the page from `base` on a row sees
    auto seen = [&](int rt, int base) __attribute__((always_inline)) {
        const int at = base + g * 16;
        if (!masked) return first_bits(lim[rt] - at);
        const int r = first + rt * 16 + n;
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
    if (tid == 0) sm_nan = 0;
    __syncthreads();

    const uint8_t *strips = a.c.arena + (uint64_t)h * 2 * kKvPage * D;
    // Bands of value scales (kv_rows.h).  Up to 64 pages their scales are at
    // hand in the one turn of the loop below; where there are more, all are
    // read first, 256 pages at a time.
    const bool many = p_hi - p_lo > 64;
    int from = kNoExp, highest = -kNoExp;
    if (many) {
        for (int p0 = p_lo + lane; p0 < p_hi + lane; p0 += 256) {
            uint64_t off[4];
            float scale[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) off[x] = p0 + x * 64 < p_hi ? page_offset(a.c, b, p0 + x * 64) : kNoPage;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (off[x] != kNoPage) scale[x] = page_scales(a.c, a.c.arena + off[x], h)[1];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if (off[x] == kNoPage) continue;
                const int e = value_exp(scale[x]);
                from = e < from ? e : from;
                highest = e > highest ? e : highest;
            }
        }
        from = least_of(from);
        highest = most_of(highest);
    }
    bool first_band = true;
    for (int p0 = p_lo; p0 < p_hi;) {
        const int np = p_hi - p0 < 64 ? p_hi - p0 : 64;
        const uint64_t off = lane < np ? page_offset(a.c, b, p0 + lane) : kNoPage;
        const uint64_t there = __builtin_amdgcn_ballot_w64(off != kNoPage);
        f32x2 scales = {0, 0};
        if (off != kNoPage) scales = *reinterpret_cast<const f32x2 *>(page_scales(a.c, a.c.arena + off, h));
        if (counts && first_band && __builtin_popcountll(there) != np)
            atomicAdd(a.c.n_invalid, (unsigned long long)(np - __builtin_popcountll(there)));
        struct Raw {
            u32x4 k[kKeyJobs], v[kValueJobs];
            int pos;  // of the lane's token
        };
        Raw ra, rz;
        // (where the waves outnumber what is left, the last piece again: loads
        // are never under a condition, see k_kv_attend)
        auto load = [&](int i, Raw &r) __attribute__((always_inline)) {
            const uint8_t *strip = strips + lane_u64(off, i);
            const uint8_t *row = strip + token_of(wave % 4, n) * D;
#pragma unroll
            for (int x = 0; x < kKeyJobs; ++x) {
                if (D % 64 != 0 && x == kChunks - 1) {
                    const u32x2 w = *reinterpret_cast<const u32x2 *>(row + x * 64 + g * 8);
                    r.k[x] = u32x4{w[0], w[1], 0, 0};
                } else {
                    const int c = wave / 4 + x * (kN / 4);
                    r.k[x] = *reinterpret_cast<const u32x4 *>(row + (c < kChunks ? c : kChunks - 1) * 64 + g * 16);
                }
            }
#pragma unroll
            for (int x = 0; x < kValueJobs; ++x) {
                const int dt = wave + x * kN, at = kTiles % kN == 0 || dt < kTiles ? dt : kTiles - 1;
                r.v[x] = *reinterpret_cast<const u32x4 *>(strip + kKvPage * D + (at * 16 + n) * kKvPage + g * 16);
            }
            if constexpr (MODE == kTerms) {  // (where there are no positions, what is at hand instead)
                const uint64_t at = ((uint64_t)b * a.c.heads + h) * a.pos_cap + (uint64_t)(p0 + i) * kKvPage;
                r.pos = (a.pos && a.slopes ? a.pos + at : reinterpret_cast<const int32_t *>(strip))[lane];
            }
        };
        // values that are not the cache's own, or are no numbers (as in
        // k_kv_attend); few pages have any
        auto clean = [&](int i, Raw &r) __attribute__((always_inline)) {
            const int base = (p0 + i) * kKvPage;
            if (base + kKvPage > s.len) {
#pragma unroll
                for (int c = 0; c < kValueJobs; ++c)
#pragma unroll
                    for (int x = 0; x < 4; ++x) r.v[c][x] = only_there(r.v[c][x], s.len - base - g * 16 - 4 * x);
            }
            if constexpr (CODES == kE4m3) {
                if (base + kKvPage > block_least) {
                    uint32_t nan = 0;
#pragma unroll
                    for (int c = 0; c < kValueJobs; ++c) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint32_t no = nan_codes(r.v[c][x]);
                            r.v[c][x] &= ~((no >> 7) * 255u);
                            nan |= no;
                        }
                    }
                    if (nan) sm_nan = 1;
                }
            }
        };
        auto store_keys = [&](int to, int x, Raw &r) __attribute__((always_inline)) {
            const int c = wave / 4 + x * (kN / 4);
            if (4 * kChunks % kN == 0 || c < kChunks) {
                u32x4 *p = &sm_k[to][(wave % 4 * kSteps + 2 * c) * 64 + lane];
                p[0] = widen8<CODES, DTYPE>(r.k[x][0], r.k[x][1]);
                if (D % 64 == 0 || x != kChunks - 1) p[64] = widen8<CODES, DTYPE>(r.k[x][2], r.k[x][3]);
            }
        };
        auto store_values = [&](int to, int x, Raw &r) __attribute__((always_inline)) {
            const int dt = wave + x * kN;
            if (kTiles % kN == 0 || dt < kTiles) {
                sm_v[to][dt * 128 + lane] = widen8<CODES, kFp16>(r.v[x][0], r.v[x][1]);
                sm_v[to][dt * 128 + 64 + lane] = widen8<CODES, kFp16>(r.v[x][2], r.v[x][3]);
            }
        };
        auto store_pos = [&](int to, Raw &r) __attribute__((always_inline)) {
            if constexpr (MODE == kTerms) {
                if (wave == 0) sm_pos[to][lane] = r.pos;
            }
        };
        auto store = [&](int to, Raw &r) __attribute__((always_inline)) {
            store_pos(to, r);
#pragma unroll
            for (int c = 0; c < kKeyJobs; ++c) store_keys(to, c, r);
#pragma unroll
            for (int c = 0; c < kValueJobs; ++c) store_values(to, c, r);
        };
        arrived(scales[0]);
        arrived(scales[1]);
        const int exp_here = off == kNoPage ? kNoExp : value_exp(scales[1]);
        if (!many && first_band && there) {
            const int e0 = __builtin_amdgcn_readlane(exp_here, __builtin_ctzll(there)), near = exp_here - e0 + kBand / 2;
            from = e0 - kBand / 2;
            if (there & __builtin_amdgcn_ballot_w64(near < 0 || near > kBand)) {  // not one band
                from = least_of(exp_here);
                highest = most_of(off == kNoPage ? -kNoExp : exp_here);
            }
        }
        uint64_t good = there & __builtin_amdgcn_ballot_w64(exp_here >= from && exp_here <= from + kBand);
        if constexpr (MODE != kPlain) {
            // Behind a cached prefix pages that no row of the workgroup sees
            // are left out here: a page a lane, the tokens of the workgroup's
            // rows over the waves.  (Without one the range from the first to
            // the last is known, which seldom has holes.)
            if (masked && s.had >= kKvPage && (p0 + 64) * kKvPage > s.had) {
                const int at = (p0 + lane) * kKvPage, off = at - s.had, words = (int)a.mask_words;
                const int t_last = ((rb + 1) * kRows < rows ? (rb + 1) * kRows - 1 : rows - 1) / G;
                uint64_t any = off < 0 ? 1u : 0u;
                if (off >= 0 && off / 64 < words && lane < np) {
                    const uint64_t *word = a.mask + off / 64;
                    const int more = off / 64 + 1 < words ? 1 : 0, sh = off % 64;
                    for (int t0 = rb * kRows / G + wave; t0 <= t_last; t0 += 4 * kN) {
                        uint64_t x[4], y[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int t = t0 + u * kN;
                            const uint64_t *row = word + (s.first + (t <= t_last ? t : t_last)) * (uint64_t)words;
                            x[u] = row[0];
                            y[u] = row[more];
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) any |= x[u] >> sh | (sh ? y[u] << (64 - sh) : 0);
                    }
                }
                const uint64_t vis = __builtin_amdgcn_ballot_w64(any != 0);
                if (lane == 0) sm_vis[wave] = vis;
                __syncthreads();
                uint64_t all = 0;
#pragma unroll
                for (int k = 0; k < kN; ++k) all |= sm_vis[k];
                good &= all;
                __syncthreads();
            }
        }
        // page i is summed from LDS while the next one's codes, loaded two
        // pages before, are brought to 16 bits, and a third page's are loaded
        uint64_t todo = good;
        auto take = [&]() __attribute__((always_inline)) {
            const int i = todo ? __builtin_ctzll(todo) : -1;
            todo &= todo - 1;
            return i;
        };
        int i = take(), next = take(), after = -1;
        // what the wave's rows see of a page under a mask, 64 tokens a row:
        // words that hold the first and the last of them, one a lane, loaded
        // a page ahead
        [[maybe_unused]] uint64_t word_ahead = 0;
        auto load_word = [&](int page) __attribute__((always_inline)) -> uint64_t {
            const int off = (p0 + page) * kKvPage - s.had;
            if (off <= -kKvPage) return 0;
            const int r = first + lane % (16 * R), last_word = (int)a.mask_words - 1;
            const int w = (off < 0 ? 0 : off / 64) + (lane / (16 * R) == 1 ? 1 : 0);
            return a.mask[(s.first + (r < rows ? r / G : 0)) * a.mask_words + (w < last_word ? w : last_word)];
        };
        if constexpr (MODE != kPlain) {
            if (masked && i >= 0) word_ahead = load_word(i);
        }
        if (i >= 0) {
            load(i, ra);
            load(next >= 0 ? next : i, rz);
            clean(i, ra);
            store(0, ra);
            __syncthreads();
        }
        // the page in buffer `cur`; the next one's codes are in `now`, those
        // of the one after it go to `then`
        auto sum_page = [&](const int cur, Raw &now, Raw &then) __attribute__((always_inline)) {
            const int base = (p0 + i) * kKvPage;
            after = take();
            load(after >= 0 ? after : i, then);
            if (next >= 0) clean(next, now);
            [[maybe_unused]] uint64_t mine = ~0ull;  // of row lane % (16 R)
            bool any = base < most, edge = base + kKvPage > least;
            if constexpr (MODE != kPlain) {
                if (masked && edge) {
                    const int off = base - s.had, left = s.len - base;
                    const uint64_t lo = word_ahead;
                    const uint64_t hi = (uint64_t)__builtin_amdgcn_ds_bpermute((lane % (16 * R) + 16 * R) * 4, (int)(uint32_t)lo) & 0xFFFFFFFFu;
                    const uint64_t hi2 = (uint64_t)(uint32_t)__builtin_amdgcn_ds_bpermute((lane % (16 * R) + 16 * R) * 4, (int)(lo >> 32));
                    const uint64_t second = hi | hi2 << 32;
                    if (off >= 0) {
                        mine = lo >> (off & 63);
                        if (off & 63) mine |= second << (64 - (off & 63));
                    } else if (off > -64) {
                        mine = lo << -off | ((1ull << -off) - 1);
                    }
                    if (left < 64) mine &= (1ull << left) - 1;
                    if (first + lane % (16 * R) >= rows) mine = 0;
                    const uint64_t of_rows = 16 * R == 64 ? ~0ull : (1ull << (16 * R % 64)) - 1;
                    any = any && (__builtin_amdgcn_ballot_w64(mine != 0) & of_rows);
                    edge = (__builtin_amdgcn_ballot_w64(mine != ~0ull) & of_rows) != 0;
                }
                if (masked && next >= 0) word_ahead = load_word(next);
            }
            if (any) {
                const float f = a.scale * kLog2e * lane_f32(scales[0], i);
                const int ei = value_exp(lane_f32(scales[1], i));
                // Operands are read a stage ahead of their products; nothing
                // moves across the stages' borders, or the reads would sink to
                // where they are used and be waited for one by one.
                f32x4 w[R][4];
                u32x4 kk[2][kSteps], vv[2][kBatch];
                auto read_keys = [&](int tt) {
#pragma unroll
                    for (int st = 0; st < kSteps; ++st) kk[tt % 2][st] = sm_k[cur][(tt * kSteps + st) * 64 + lane];
                };
                auto read_values = [&](int at) {  // batch `at` of the first half's, then the second's
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
                        vv[at % 2][k] =
                            sm_v[cur][(at % kBatches * kBatch + k) * 128 + at / kBatches * 64 + lane];
                };
                read_keys(0);
#pragma unroll
                for (int tt = 0; tt < 4; ++tt) {
                    if (tt < 3)
                        read_keys(tt + 1);
                    else
                        read_values(0);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int rt = 0; rt < R; ++rt) w[rt][tt] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int st = 0; st < kSteps; ++st)
#pragma unroll
                        for (int rt = 0; rt < R; ++rt) w[rt][tt] = mfma16<DTYPE>(kk[tt % 2][st], q[rt][st], w[rt][tt]);
                    // a share of the next page (of the last: what is there once more)
#pragma unroll
                    for (int c = 0; c < kKeyJobs; ++c)
                        if (c % 4 == tt) store_keys(cur ^ 1, c, now);
#pragma unroll
                    for (int c = 0; c < kValueJobs; ++c)
                        if ((kKeyJobs + c) % 4 == tt) store_values(cur ^ 1, c, now);
                    if (tt == 3) store_pos(cur ^ 1, now);
                    __builtin_amdgcn_sched_barrier(0);
                }
                float fade[R];
#pragma unroll
                for (int rt = 0; rt < R; ++rt) {
                    if constexpr (MODE == kPlain) {
                        fade[rt] = soft_scores(soft[rt], w[rt], f, ei, edge, lim[rt] - base - g * 16);
                    } else {
                        uint32_t bits = 0xFFFFu;
                        if (edge) {
                            if (masked) {
                                const int from = (rt * 16 + n) * 4;
                                const uint32_t lo = __builtin_amdgcn_ds_bpermute(from, (int)(uint32_t)mine);
                                const uint32_t hi = __builtin_amdgcn_ds_bpermute(from, (int)(mine >> 32));
                                bits = ((g & 2 ? hi : lo) >> (g & 1 ? 16 : 0)) & 0xFFFFu;
                            } else {
                                bits = first_bits(lim[rt] - base - g * 16);
                            }
                        }
                        if constexpr (MODE == kMasked) {
                            fade[rt] = soft_scores<true>(soft[rt], w[rt], f, ei, edge, (int)bits);
                        } else {
                            fade[rt] = soft_step(soft[rt], w[rt], ei, [&](float c) __attribute__((always_inline)) {
                                if constexpr (MODE == kTerms)
                                    term_scores(a, w[rt], f, slope[rt], row_pos[rt], base + g * 16,
                                                [&](int x) { return sm_pos[cur][g * 16 + x]; }, c);
                                else
                                    cap_scores<MODE>(a, w[rt], f, c);
                                if (edge) hide(w[rt], bits);
                            });
                        }
                    }
                }
#pragma unroll
                for (int rt = 0; rt < R; ++rt) {
                    if (__builtin_amdgcn_ballot_w64(fade[rt] != 1.0f)) {
#pragma unroll
                        for (int dt = 0; dt < kTiles; ++dt)
#pragma unroll
                            for (int x = 0; x < 4; ++x) o[rt][dt][x] *= fade[rt];
                        rounding[rt].fade(fade[rt]);
                    }
                }
                // the first half's products run beside the second half's exponents
                float sum[R] = {};
                u32x4 pw[R][2];
#pragma unroll
                for (int rt = 0; rt < R; ++rt)
                    pw[rt][0] = soft_weights(w[rt][0], w[rt][1], sum[rt]);
#pragma unroll
                for (int at = 0; at < 2 * kBatches; ++at) {
                    if (at + 1 < 2 * kBatches) read_values(at + 1);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
#pragma unroll
                        for (int rt = 0; rt < R; ++rt) {
                            f32x4 &to = o[rt][at % kBatches * kBatch + k];
                            to = mfma16<kFp16>(vv[at % 2][k], pw[rt][at / kBatches], to);
                        }
                    if (at % kBatches == 0) {
#pragma unroll
                        for (int rt = 0; rt < R; ++rt) rounding[rt].add(pw[rt][at / kBatches]);
                    }
#pragma unroll
                    for (int rt = 0; rt < R; ++rt)
                        if (at == (rt < kBatches ? rt : kBatches - 1))
                            pw[rt][1] = soft_weights(w[rt][2], w[rt][3], sum[rt]);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int rt = 0; rt < R; ++rt)
                {
                    soft[rt].l = __builtin_fmaf(sum[rt], pow2(-ei), soft[rt].l);
                    rounding[rt].add_exact(sum[rt]);
                }
            } else {
                store(cur ^ 1, now);
            }
            __syncthreads();
            i = next;
            next = after;
        };
        while (i >= 0) {
            sum_page(0, rz, ra);
            if (i < 0) break;
            sum_page(1, ra, rz);
        }
        p0 += 64;
        if (p0 >= p_hi && (from += kBand + 1) <= highest) {  // once more, over the next band
            first_band = false;
            p0 = p_lo;
        }
    }
    if constexpr (CODES == kE4m3) {
        __syncthreads();
        if (sm_nan) {
            for (int p = block_least / kKvPage > p_lo ? block_least / kKvPage : p_lo; p < p_hi; ++p) {
                const uint64_t off = wave_uniform(page_offset(a.c, b, p));
                if (off == kNoPage) continue;
                uint32_t see[R];
#pragma unroll
                for (int rt = 0; rt < R; ++rt) see[rt] = seen(rt, p * kKvPage);
                put_nan<D, R>(strips + off + kKvPage * D + n * kKvPage + g * 16, see, o);
            }
        }
    }

    const uint64_t heads = (uint64_t)a.c.heads * G, all = a.tokens * heads;
#pragma unroll
    for (int rt = 0; rt < R; ++rt) {
        const float sum = across_groups(soft[rt].l, [](float x, float y) { return x + y; });
        const float factor = rounding[rt].factor();
        const int r = first + rt * 16 + n;
        if (r >= rows) continue;
        const uint64_t row = (s.first + r / G) * heads + (uint64_t)h * G + r % G;
        if (active == 1) {
            const float inv = sum == 0.0f ? 0.0f : factor / sum;
#pragma unroll
            for (int dt = 0; dt < kTiles; ++dt) {
                u32x2 x;
                x[0] = pack2<DTYPE>(o[rt][dt][0] * inv, o[rt][dt][1] * inv);
                x[1] = pack2<DTYPE>(o[rt][dt][2] * inv, o[rt][dt][3] * inv);
                *reinterpret_cast<u32x2 *>(a.out + row * D + dt * 16 + g * 4) = x;
            }
            if (g == 0) put_sum(a, row, soft[rt].m == KV_NEG_INF ? 0.0f : soft[rt].m, sum);
        } else {
            float *part = a.part + ((uint64_t)split * all + row) * D;
#pragma unroll
            for (int dt = 0; dt < kTiles; ++dt) *reinterpret_cast<f32x4 *>(part + dt * 16 + g * 4) = o[rt][dt] * factor;
            if (g == 0)
                *reinterpret_cast<f32x2 *>(a.part + (uint64_t)a.splits * all * D + ((uint64_t)split * all + row) * 2) =
                    f32x2{soft[rt].m, sum};
        }
    }
}

template <int MODE, int D, int CODES, int ROWS>
void prompt_rows(const KvAttend &a, int dtype, hipStream_t s) {
    const dim3 grid = grid_of(kv_prompt_blocks(a.splits, a.row_blocks, a.c.heads, a.c.batch)), block(kPromptWaves<D, ROWS> * 64);
    if (dtype == kBf16)
        hipLaunchKernelGGL((k_kv_prompt<D, CODES, kBf16, MODE, ROWS>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((k_kv_prompt<D, CODES, kFp16, MODE, ROWS>), grid, block, 0, s, a);
}

template <int MODE, int D, int CODES>
void prompt_go(const KvAttend &a, int dtype, hipStream_t s) {
    if constexpr (MODE == kMasked && D <= 128) {
        if (a.rows == kKvTreeRows) return prompt_rows<MODE, D, CODES, (int)kKvTreeRows>(a, dtype, s);
    }
    prompt_rows<MODE, D, CODES, (int)kKvPromptRows>(a, dtype, s);
}

template <int MODE, int D>
void prompt_codes(const KvAttend &a, int codes, int dtype, hipStream_t s) {
    if (codes == kE4m3)
        prompt_go<MODE, D, kE4m3>(a, dtype, s);
    else
        prompt_go<MODE, D, kInt8>(a, dtype, s);
}

}  // namespace

template <int MODE>
hipError_t launch_kv_prompt(const KvAttend &a, int codes, int dtype, hipStream_t s) {
    switch (a.c.dim) {
        case 64: prompt_codes<MODE, 64>(a, codes, dtype, s); break;
        case 96: prompt_codes<MODE, 96>(a, codes, dtype, s); break;
        case 128: prompt_codes<MODE, 128>(a, codes, dtype, s); break;
        case 192: prompt_codes<MODE, 192>(a, codes, dtype, s); break;
        case 256: prompt_codes<MODE, 256>(a, codes, dtype, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace ac

#endif
