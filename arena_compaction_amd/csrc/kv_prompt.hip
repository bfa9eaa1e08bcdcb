// kv_prompt.hip -- attention of many query rows over the 8-bit cache (a
// prompt's tokens, times the heads that share a key/value head).
//
// The mathematics is that of kv_attend.hip; what differs is who holds what.
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
// (169 GFLOP) take 223 us, 0.76 PFLOP/s, where a product of 8192 cubed reaches
// 1.18: the matrix pipe is busy for 31% of the cycles, the vector pipe for 37%,
// and 22% are lost to the last rows, which see most.  With 64 dimensions the
// vector pipe is busy for 83% (8200 tokens x 32 heads, float16: 380 us).
//
// Workgroups of one key/value head run on one XCD where the heads are a
// multiple of 8, so that its pages stay in that XCD's L2; the last rows,
// which see most, start first.
#include "kv_rows.h"

namespace ac {
namespace {

// 32 rows a wave; above 128 dimensions 16, whose sums and queries leave two
// waves a SIMD their registers.
template <int D>
constexpr int kPromptWaves = D <= 128 ? 4 : 8;

template <int D, int CODES, int DTYPE>
__global__ __launch_bounds__(kPromptWaves<D> * 64, D == 64 && CODES == kE4m3 && DTYPE == kBf16 ? 3 : 2) void k_kv_prompt(KvAttend a) {
    constexpr int kN = kPromptWaves<D>, kRows = (int)kKvPromptRows, R = kRows / 16 / kN;
    constexpr int kSteps = D / 32, kTiles = D / 16;
    constexpr int kBatch = kTiles % 4 ? 3 : 4, kBatches = kTiles / kBatch;  // value tiles read at a time
    // a wave's share of a page: of the keys' 4 tiles x chunks of 64 dimensions
    // and of the values' tiles, every kN-th
    constexpr int kChunks = (D + 63) / 64, kKeyJobs = (4 * kChunks + kN - 1) / kN, kValueJobs = (kTiles + kN - 1) / kN;
    __shared__ u32x4 sm_k[2][4 * kSteps * 64], sm_v[2][kTiles * 2 * 64];
    __shared__ int sm_nan;
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
    const int pages = block_pages(a, s, rb);
    const int per = (int)a.per_split;
    const int active = pages > per ? (pages + per - 1) / per : 1;
    if (split >= active) return;
    const int p_lo = split * per, p_hi = p_lo + per < pages ? p_lo + per : pages;
    const bool counts = a.c.n_invalid && h == 0 && (rb + 1) * kRows >= rows && tid == 0;  // once a page

    const int first = rb * kRows + wave * 16 * R;  // the wave's rows
    u32x4 q[R][kSteps];
    int lim[R];
    load_rows<D, R>(a, s, h, first, lane, q, lim);
    // what the workgroup's first row sees, and the wave's first and last
    const int block_least = s.had + rb * kRows / G + 1, least = s.had + first / G + 1;
    const int last = (first + 16 * R < rows ? first + 16 * R : rows) - 1;
    const int most = first < rows ? s.had + last / G + 1 : 0;
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
        auto store = [&](int to, Raw &r) __attribute__((always_inline)) {
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
        const uint64_t good = there & __builtin_amdgcn_ballot_w64(exp_here >= from && exp_here <= from + kBand);
        // page i is summed from LDS while the next one's codes, loaded two
        // pages before, are brought to 16 bits, and a third page's are loaded
        uint64_t todo = good;
        auto take = [&]() __attribute__((always_inline)) {
            const int i = todo ? __builtin_ctzll(todo) : -1;
            todo &= todo - 1;
            return i;
        };
        int i = take(), next = take(), after = -1;
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
            if (base < most) {
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
                    __builtin_amdgcn_sched_barrier(0);
                }
                float fade[R];
#pragma unroll
                for (int rt = 0; rt < R; ++rt)
                    fade[rt] = soft_scores(soft[rt], w[rt], f, ei, base + kKvPage > least, lim[rt] - base - g * 16);
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
                int see[R];
#pragma unroll
                for (int rt = 0; rt < R; ++rt) see[rt] = lim[rt] - p * kKvPage - g * 16;
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

template <int D, int CODES>
void prompt_go(const KvAttend &a, int dtype, hipStream_t s) {
    const dim3 grid = grid_of(kv_prompt_blocks(a.splits, a.row_blocks, a.c.heads, a.c.batch));
    if (dtype == kBf16)
        hipLaunchKernelGGL((k_kv_prompt<D, CODES, kBf16>), grid, dim3(kPromptWaves<D> * 64), 0, s, a);
    else
        hipLaunchKernelGGL((k_kv_prompt<D, CODES, kFp16>), grid, dim3(kPromptWaves<D> * 64), 0, s, a);
}

template <int D>
void prompt_codes(const KvAttend &a, int codes, int dtype, hipStream_t s) {
    if (codes == kE4m3)
        prompt_go<D, kE4m3>(a, dtype, s);
    else
        prompt_go<D, kInt8>(a, dtype, s);
}

}  // namespace

hipError_t launch_kv_prompt(const KvAttend &a, int codes, int dtype, hipStream_t s) {
    switch (a.c.dim) {
        case 64: prompt_codes<64>(a, codes, dtype, s); break;
        case 96: prompt_codes<96>(a, codes, dtype, s); break;
        case 128: prompt_codes<128>(a, codes, dtype, s); break;
        case 192: prompt_codes<192>(a, codes, dtype, s); break;
        case 256: prompt_codes<256>(a, codes, dtype, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace ac
