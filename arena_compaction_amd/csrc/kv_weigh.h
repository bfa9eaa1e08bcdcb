// kv_weigh.h -- the weight that every cached token receives, from scores that
// are made again (kv_finish.hip says when, and what it costs without terms).
//
// With terms an exponent a score is not all: 4 sequences of 500 tokens behind
// 1000, 8 heads x 4 query heads each, documents, e4m3; the pass over the pages
// alone and with the weights, without terms, under a mask, with a bias:
//    64 dimensions   40  72    44  75    52 102 us
//   128              57 104    60 117    71 140
//   256             107 178   110 235   124 254
// Of 256 dimensions 34 registers go to memory under a mask and 51 to 56 with all
// terms, none without.
#ifndef ARENA_COMPACTION_KV_WEIGH_H
#define ARENA_COMPACTION_KV_WEIGH_H
#include "kv_rows.h"

namespace ac {
namespace {

// Tiles of 16 rows [first, end) of a piece of the rows that see something of
// the page from token `base` on; none: false.
__device__ inline bool piece_tiles(const KvAttend &a, const Seq &s, int base, int piece, int *first, int *end) {
    const int tiles = (s.count * (int)a.group + 15) / 16, each = (int)a.weigh_tiles;
    // earlier rows see nothing here
    const int least = !a.mask && base > s.had ? (base - s.had) * (int)a.group / 16 : 0;
    *first = least > piece * each ? least : piece * each;
    *end = tiles < (piece + 1) * each ? tiles : (piece + 1) * each;
    return *first < *end;
}

// Waves of a workgroup: with terms never 16, whose 128 registers would spill.
// (Pieces of the rows are sized by the plain kernel's, so that a call's workspace
// does not depend on its terms.  Sized by 8 waves, twice as many for 64
// dimensions: 2 x 206 tokens x 3 heads x 16 query heads under a mask 27.7 us for
// 29.6, under a cap 30.3 for 34.7; 700 behind 300, 2 heads x 8, 37.1 for 35.3.)
template <int D, int MODE>
constexpr int kWeighWaves = MODE == kPlain ? (int)kv_weigh_waves(D) : 8;

template <int D, int CODES, int DTYPE, int MODE>
__global__ __launch_bounds__((kWeighWaves<D, MODE>)*64) void k_kv_weigh(KvAttend a) {
    constexpr int kSteps = D / 32, kN = kWeighWaves<D, MODE>;
    constexpr int kPieces = D / 8, kPitch = kPieces + 1;  // of 16 bytes; odd, so that rows start in other banks
    __shared__ float sm[kN][kKvPage];
    __shared__ u32x4 sm_q[kN][16 * kPitch];
    __shared__ int sm_pos[MODE == kTerms ? kKvPage : 1];  // positions of the page's tokens
    // the last rows first: every page's rows end there, so that workgroups
    // that start together read the same queries
    const uint32_t units = a.c.heads * a.c.batch, block = block_number();
    if (block >= units * a.score_pages * a.weigh_pieces) return;
    const uint32_t unit = block % units, h = unit % a.c.heads, b = unit / a.c.heads;
    const uint32_t piece = a.weigh_pieces - 1 - block / (units * a.score_pages);
    const int tid = threadIdx.x, wave = wave_uniform(tid / 64), lane = tid % 64;
    const int n = lane % 16, g = lane / 16, G = (int)a.group;
    bool bad;
    const Seq s = sequence(a, b, &bad);
    const int p = (int)(block / units % a.score_pages), base = p * kKvPage;
    if (base >= s.len || s.count == 0) return;
    const int rows = s.count * (int)a.group;
    int first, tiles;
    if (!piece_tiles(a, s, base, (int)piece, &first, &tiles)) return;
    const uint64_t off = wave_uniform(page_offset(a.c, b, p));
    if (off == kNoPage) return;
    const float f = a.scale * kLog2e * page_scales(a.c, a.c.arena + off, h)[0];
    u32x4 kk[4][kSteps];
    {
        const uint8_t *strip = a.c.arena + off + (uint64_t)h * 2 * kKvPage * D + g * 8;
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                const u32x2 x = *reinterpret_cast<const u32x2 *>(strip + token_of(tt, n) * D + st * 32);
                kk[tt][st] = widen8<CODES, DTYPE>(x[0], x[1]);
            }
    }
    const bool masked = MODE != kPlain && a.mask != nullptr, page_edge = base + kKvPage > s.had;
    if constexpr (MODE == kTerms) {
        if (a.slopes && a.pos) {
            if (tid < kKvPage) sm_pos[tid] = a.pos[((uint64_t)b * a.c.heads + h) * a.pos_cap + base + tid];
            __syncthreads();
        }
    }
    float acc[16] = {};
    const uint64_t heads = (uint64_t)a.c.heads * G;
    // Tiles of 16 rows, every kN-th, from the last one down, since all pages'
    // rows end there: workgroups that start together go through the same
    // queries together, out of L2.  A tile's first token is the wave's (t0) and its
    // address scalar; a lane adds where its row lies from there, which is the
    // same in every turn where the group's heads divide the rows of a turn.
    // Queries are loaded with neighbouring lanes on neighbouring bytes and
    // dealt out through LDS, each wave's own: as the operand wants them,
    // neighbouring lanes on neighbouring rows, L1 would serve 16 bytes at a
    // time, and be what the kernel waits for.
    const int least = first + wave;
    const int turns = tiles > least ? (tiles - least + kN - 1) / kN : 0;
    const uint32_t by_group = ((1u << 20) + G - 1) / G;  // v / G = v * by_group >> 20 for v < G + 16
    const bool same = kN * 16 % G == 0;
    const int see0 = s.had + 1 - base - g * 16;
    int64_t q_at[kSteps];  // in elements, from the tile's first token
    int sum_at = 0, lane_t = 0;
    auto place = [&](int v0, int most) __attribute__((always_inline)) {  // v0: the tile's first row less t0 * G
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int item = i * 64 + lane, row = item / kPieces;
            const int v = v0 + (row < most ? row : 0), t = (int)((uint32_t)v * by_group >> 20);
            q_at[i] = t * a.q_row + (v - t * G) * a.q_head + item % kPieces * 8;
        }
        const int v = v0 + (n < most ? n : 0);
        lane_t = (int)((uint32_t)v * by_group >> 20);
        sum_at = lane_t * (int)heads + (v - lane_t * G);
    };
    u32x4 q[kSteps];
    float2 ml = make_float2(0.0f, 0.0f);
    int see = 0;
    [[maybe_unused]] Words words{~0ull, ~0ull};
    [[maybe_unused]] float slope = 0.0f;
    [[maybe_unused]] int row_pos = 0;
    auto load = [&](int x, bool last) __attribute__((always_inline)) {  // last: some rows may not be there
        const int t0 = wave_uniform(x * 16 / G), v0 = x * 16 - t0 * G, most = last ? rows - x * 16 : 16;
        if (last || !same) place(v0, most);
        const uint16_t *tile = a.q + (int64_t)(s.first + t0) * a.q_row + (int64_t)h * G * a.q_head;
        ml = a.sums[(s.first + t0) * heads + (uint64_t)h * G + sum_at];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) q[i] = load_q8(tile + q_at[i]);
        see = n < most ? see0 + t0 + lane_t : 0;
        if constexpr (MODE != kPlain) {
            if (masked && page_edge) words = mask_words(a, s, s.first + t0 + lane_t, base + g * 16);
        }
        if constexpr (MODE == kTerms) {
            const int v = v0 + (n < most ? n : 0);
            row_terms(a, s, b, h, t0 + lane_t, v - lane_t * G, slope, row_pos);
        }
        if (last && same) place(v0, 16);
    };
    u32x4 *const mine = sm_q[wave];
    int x = least + (turns - 1) * kN;
    if (turns) load(x, true);
    for (int k = 0; k < turns; ++k) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int item = i * 64 + lane;
            mine[item / kPieces * kPitch + item % kPieces] = q[i];
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        u32x4 qq[kSteps];
#pragma unroll
        for (int st = 0; st < kSteps; ++st) qq[st] = mine[n * kPitch + st * 4 + g];
        const float2 now = ml;
        const int see_now = see;
        // some row misses some token
        const bool edge = k == 0 || (masked ? page_edge : x * 16 / G + s.had + 1 - base < 64);
        [[maybe_unused]] uint32_t bits = 0xFFFFu;
        [[maybe_unused]] const float slope_now = slope;
        [[maybe_unused]] const int pos_now = row_pos;
        if constexpr (MODE != kPlain) {
            if (edge) {
                if (!masked)
                    bits = first_bits(see_now);
                else if (page_edge)
                    bits = mask_bits(words, s, base + g * 16);
                if (masked && k == 0 && x * 16 + n >= rows) bits = 0;
            }
        }
        if (k + 1 < turns) {
            x -= kN;
            load(x, false);  // all 16 rows are there: only the last tile may have fewer
        }
        f32x4 w[4];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
            w[tt] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int st = 0; st < kSteps; ++st) w[tt] = mfma16<DTYPE>(kk[tt][st], qq[st], w[tt]);
        }
        if constexpr (MODE == kTerms) {
            term_scores(a, w, f, slope_now, pos_now, base + g * 16, [&](int i) { return sm_pos[g * 16 + i]; }, -now.x);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i / 4][i % 4] = __builtin_fmaf(w[i / 4][i % 4], f, -now.x);
        }
        if (edge) {
            if constexpr (MODE == kPlain) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (i >= see_now) w[i / 4][i % 4] = KV_NEG_INF;
            } else {
                hide(w, bits);
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
            acc[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(w[i / 4][i % 4]), now.y, acc[i]);
        __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float v = acc[i];
        v += dpp_move<kDppQuadSwap1>(v);
        v += dpp_move<kDppQuadSwap2>(v);
        v += dpp_move<kDppRowHalfMirror>(v);
        v += dpp_move<kDppRowMirror>(v);
        if (n == 0) sm[wave][g * 16 + i] = v;
    }
    __syncthreads();
    if (tid < kKvPage && base + tid < s.len) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kN; ++k) sum += sm[k][tid];
        if (a.weigh_part)
            a.weigh_part[(((uint64_t)piece * a.c.batch + b) * a.c.heads + h) * a.score_pages * kKvPage + base + tid] = sum;
        else
            a.weight[((uint64_t)b * a.c.heads + h) * a.cap + base + tid] += sum;
    }
}

// Adds up what the pieces of the rows made, a token a lane, in their order.
__global__ __launch_bounds__(kThreads) void k_kv_add(KvAttend a) {
    const uint32_t h = blockIdx.y, b = blockIdx.z;
    const int j = (int)(blockIdx.x * kThreads + threadIdx.x), base = j / kKvPage * kKvPage;
    bool bad;
    const Seq s = sequence(a, b, &bad);
    if (j >= s.len || s.count == 0) return;
    if (page_offset(a.c, b, j / kKvPage) == kNoPage) return;
    const uint64_t unit = (uint64_t)b * a.c.heads + h, step = (uint64_t)a.c.batch * a.c.heads * a.score_pages * kKvPage;
    const float *part = a.weigh_part + unit * a.score_pages * kKvPage + j;
    float sum = 0.0f;
    for (uint32_t k = 0; k < a.weigh_pieces; ++k) {
        int first, tiles;
        if (piece_tiles(a, s, base, (int)k, &first, &tiles)) sum += part[k * step];
    }
    a.weight[unit * a.cap + j] += sum;
}

template <int MODE, int D, int CODES>
void weigh_go(const KvAttend &a, int dtype, hipStream_t s) {
    const dim3 grid = grid_of(kv_weigh_blocks(a.score_pages, a.weigh_pieces, a.c.heads, a.c.batch)), block(kWeighWaves<D, MODE> * 64);
    if (dtype == kBf16)
        hipLaunchKernelGGL((k_kv_weigh<D, CODES, kBf16, MODE>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((k_kv_weigh<D, CODES, kFp16, MODE>), grid, block, 0, s, a);
}

template <int MODE, int D>
void weigh_codes(const KvAttend &a, int codes, int dtype, hipStream_t s) {
    if (codes == kE4m3)
        weigh_go<MODE, D, kE4m3>(a, dtype, s);
    else
        weigh_go<MODE, D, kInt8>(a, dtype, s);
}

}  // namespace

template <int MODE>
hipError_t launch_kv_weigh(const KvAttend &a, int codes, int dtype, hipStream_t s) {
    if (a.max_len == 0) return hipSuccess;
    switch (a.c.dim) {
        case 64: weigh_codes<MODE, 64>(a, codes, dtype, s); break;
        case 96: weigh_codes<MODE, 96>(a, codes, dtype, s); break;
        case 128: weigh_codes<MODE, 128>(a, codes, dtype, s); break;
        case 192: weigh_codes<MODE, 192>(a, codes, dtype, s); break;
        case 256: weigh_codes<MODE, 256>(a, codes, dtype, s); break;
        default: return hipErrorInvalidValue;
    }
    if (a.weigh_part) {
        const dim3 grid((a.max_len + kThreads - 1) / kThreads, a.c.heads, a.c.batch);
        hipLaunchKernelGGL(k_kv_add, grid, dim3(kThreads), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace ac

#endif
