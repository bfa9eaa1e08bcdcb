// kv_prompt.hip -- attention of many query rows over the 8-bit cache (a
// prompt's tokens, times the heads that share a key/value head).
//
// The mathematics is that of kv_attend.hip; what differs is who holds what.
// With many rows the cost is the matrix products and, per score, an exponent,
// so a workgroup takes 128 rows, 32 a wave, and all its waves go over the
// same pages: each page is loaded once, its codes brought to 16 bits once (a
// quarter of a page a wave) and put into LDS in the very order in which the
// matrix instructions' operands are read, 16 bytes a lane, in a line.  Two
// pages are in LDS, one being summed and one being filled, while the codes of
// a third are on their way.
//
// Workgroups of one key/value head run on one XCD where the heads are a
// multiple of 8, so that its pages stay in that XCD's L2; the last rows,
// which see most, start first.
#include "kv_rows.h"

namespace ac {
namespace {

template <int D, int CODES, int DTYPE>
__global__ __launch_bounds__(kThreads, D <= 128 ? 2 : 1) void k_kv_prompt(KvAttend a) {
    constexpr int R = 2, kSteps = D / 32, kTiles = D / 16, kRows = (int)kKvPromptRows;
    constexpr int kKeyJobs = (D + 63) / 64, kValueJobs = (kTiles + kWaves - 1) / kWaves;
    __shared__ u32x4 sm_k[2][4 * kSteps * 64], sm_v[2][kTiles * 2 * 64];
    __shared__ int sm_nan;
    const uint32_t units = a.c.batch * a.c.heads, unit = blockIdx.x % units, piece = blockIdx.x / units;
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
#pragma unroll
    for (int rt = 0; rt < R; ++rt) {
        soft[rt] = Soft{KV_NEG_INF, 0.0f};
#pragma unroll
        for (int dt = 0; dt < kTiles; ++dt) o[rt][dt] = f32x4{0, 0, 0, 0};
    }
    if (tid == 0) sm_nan = 0;
    __syncthreads();

    const uint8_t *strips = a.c.arena + (uint64_t)h * 2 * kKvPage * D;
    for (int p0 = p_lo; p0 < p_hi; p0 += 64) {
        const int np = p_hi - p0 < 64 ? p_hi - p0 : 64;
        const uint64_t off = lane < np ? page_offset(a.c, b, p0 + lane) : kNoPage;
        const uint64_t good = __builtin_amdgcn_ballot_w64(off != kNoPage);
        f32x2 scales = {0, 0};
        if (off != kNoPage) scales = *reinterpret_cast<const f32x2 *>(page_scales(a.c, a.c.arena + off, h));
        if (counts && __builtin_popcountll(good) != np)
            atomicAdd(a.c.n_invalid, (unsigned long long)(np - __builtin_popcountll(good)));
        // a wave's share of a page: key tile `wave`, and every fourth of the value tiles
        u32x4 kr[kKeyJobs], vr[kValueJobs];
        auto load = [&](int i) {
            const uint8_t *strip = strips + lane_u64(off, i);
            const uint8_t *row = strip + token_of(wave, n) * D;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) kr[c] = *reinterpret_cast<const u32x4 *>(row + c * 64 + g * 16);
            if constexpr (D % 64 != 0) {
                const u32x2 x = *reinterpret_cast<const u32x2 *>(row + D / 64 * 64 + g * 8);
                kr[kKeyJobs - 1] = u32x4{x[0], x[1], 0, 0};
            }
#pragma unroll
            for (int c = 0; c < kValueJobs; ++c) {
                const int dt = wave + c * kWaves;
                if (dt < kTiles)
                    vr[c] = *reinterpret_cast<const u32x4 *>(strip + kKvPage * D + (dt * 16 + n) * kKvPage + g * 16);
            }
        };
        auto store = [&](int i, int to) {
            const int base = (p0 + i) * kKvPage;
#pragma unroll
            for (int c = 0; c < kKeyJobs; ++c) {
                sm_k[to][(wave * kSteps + 2 * c) * 64 + lane] = widen8<CODES, DTYPE>(kr[c][0], kr[c][1]);
                if (2 * c + 1 < kSteps)
                    sm_k[to][(wave * kSteps + 2 * c + 1) * 64 + lane] = widen8<CODES, DTYPE>(kr[c][2], kr[c][3]);
            }
            uint32_t nan = 0;
#pragma unroll
            for (int c = 0; c < kValueJobs; ++c) {
                const int dt = wave + c * kWaves;
                if (base + kKvPage > s.len) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) vr[c][x] = only_there(vr[c][x], s.len - base - g * 16 - 4 * x);
                }
                if constexpr (CODES == kE4m3) {  // as in k_kv_attend
                    if (base + kKvPage > block_least && dt < kTiles) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint32_t no = nan_codes(vr[c][x]);
                            vr[c][x] &= ~((no >> 7) * 255u);
                            nan |= no;
                        }
                    }
                }
                if (dt < kTiles) {
                    sm_v[to][dt * 128 + lane] = widen8<CODES, kFp16>(vr[c][0], vr[c][1]);
                    sm_v[to][dt * 128 + 64 + lane] = widen8<CODES, kFp16>(vr[c][2], vr[c][3]);
                }
            }
            if (nan) sm_nan = 1;
        };
        arrived(scales[0]);
        arrived(scales[1]);
        uint64_t todo = good;
        int cur = 0;
        if (todo) {
            load(__builtin_ctzll(todo));
            store(__builtin_ctzll(todo), 0);
            __syncthreads();
        }
        while (todo) {
            const int i = __builtin_ctzll(todo), base = (p0 + i) * kKvPage;
            todo &= todo - 1;
            const int next = todo ? __builtin_ctzll(todo) : -1;
            if (next >= 0) load(next);
            if (base < most) {
                const float f = a.scale * kLog2e * lane_f32(scales[0], i);
                const int ei = value_exp(lane_f32(scales[1], i));
                f32x4 w[R][4];
#pragma unroll
                for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
                    for (int rt = 0; rt < R; ++rt) w[rt][tt] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int st = 0; st < kSteps; ++st) {
                        const u32x4 kk = sm_k[cur][(tt * kSteps + st) * 64 + lane];
#pragma unroll
                        for (int rt = 0; rt < R; ++rt) w[rt][tt] = mfma16<DTYPE>(kk, q[rt][st], w[rt][tt]);
                    }
                }
                u32x4 pw[R][2];
#pragma unroll
                for (int rt = 0; rt < R; ++rt) {
                    const float fade =
                        soft_page(soft[rt], w[rt], f, ei, base + kKvPage > least, lim[rt] - base - g * 16);
                    pack_weights(w[rt], pw[rt]);
                    if (__builtin_amdgcn_ballot_w64(fade != 1.0f)) {
#pragma unroll
                        for (int dt = 0; dt < kTiles; ++dt)
#pragma unroll
                            for (int x = 0; x < 4; ++x) o[rt][dt][x] *= fade;
                    }
                }
#pragma unroll
                for (int dt = 0; dt < kTiles; ++dt) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const u32x4 vv = sm_v[cur][dt * 128 + x * 64 + lane];
#pragma unroll
                        for (int rt = 0; rt < R; ++rt) o[rt][dt] = mfma16<kFp16>(vv, pw[rt][x], o[rt][dt]);
                    }
                }
            }
            if (next >= 0) store(next, cur ^ 1);
            __syncthreads();
            cur ^= 1;
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
        const int r = first + rt * 16 + n;
        if (r >= rows) continue;
        const uint64_t row = (s.first + r / G) * heads + (uint64_t)h * G + r % G;
        if (active == 1) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int dt = 0; dt < kTiles; ++dt) {
                u32x2 x;
                x[0] = pack2<DTYPE>(o[rt][dt][0] * inv, o[rt][dt][1] * inv);
                x[1] = pack2<DTYPE>(o[rt][dt][2] * inv, o[rt][dt][3] * inv);
                *reinterpret_cast<u32x2 *>(a.out + row * D + dt * 16 + g * 4) = x;
            }
            if (g == 0) put_sum(a, row, soft[rt].m, sum);
        } else {
            float *part = a.part + ((uint64_t)split * all + row) * D;
#pragma unroll
            for (int dt = 0; dt < kTiles; ++dt) *reinterpret_cast<f32x4 *>(part + dt * 16 + g * 4) = o[rt][dt];
            if (g == 0)
                *reinterpret_cast<f32x2 *>(a.part + (uint64_t)a.splits * all * D + ((uint64_t)split * all + row) * 2) =
                    f32x2{soft[rt].m, sum};
        }
    }
}

template <int D, int CODES>
void prompt_go(const KvAttend &a, int dtype, hipStream_t s) {
    const dim3 grid(a.splits * a.row_blocks * a.c.heads * a.c.batch);
    if (dtype == kBf16)
        hipLaunchKernelGGL((k_kv_prompt<D, CODES, kBf16>), grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((k_kv_prompt<D, CODES, kFp16>), grid, dim3(kThreads), 0, s, a);
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
