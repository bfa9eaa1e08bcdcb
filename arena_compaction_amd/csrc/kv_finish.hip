// kv_finish.hip -- what follows attention's pass over the pages: joining the
// parts of rows whose cache was split, and the weight that every cached token
// receives,
//   weight_j += sum_r 2^(t_rj - m_r) / l_r
// over the query rows r that see token j, once each row's m and l are known.
//
//   k_kv_finish  joins parts and, where attention kept its scores (few rows),
//                adds up the weights, in one launch: the weights' workgroups
//                work out m and l from the parts themselves;
//   k_kv_weigh   many rows: makes the scores again.  One workgroup a (page,
//                head) holds the page's keys and goes over all the rows that
//                see it, or a piece of them, whose sums k_kv_add adds up.
// The second is bound by the vector pipe (74% of the cycles) with an exponent
// and two fused products a score: 241 us for 8200 tokens x 32 heads of 64.  The
// first moves 36 MB for 48 x 8000 tokens x 4 heads, 28 of them scores, in 14 us.
//
// A token belongs to one workgroup, and its rows are added in one order,
// whatever else runs: no atomics, the same bits every time.
#include "kv_rows.h"

namespace ac {
namespace {

// Parts of the rows of block rb (1: the first pass has written the result).
__device__ inline int parts_of(const KvAttend &a, const Seq &s, int rb) {
    const int pages = block_pages(a, s, rb);
    return (pages + (int)a.per_split - 1) / (int)a.per_split;
}

__device__ inline const float *part_sums(const KvAttend &a, uint64_t all, uint64_t row) {
    return a.part + (uint64_t)a.splits * all * a.c.dim + row * 2;
}

static_assert(kKeptTokens == 2 * kThreads, "two tokens a lane");
constexpr uint32_t kFewParts = 16;  // a wave a row, above them a workgroup a row

// Row and head `unit` of sequence b from its parts k = first, first + STEP...
// 64 maxima and sums are read at once, a lane each, then 8 parts at a time.
template <int STEP>
__device__ inline void join_parts(const KvAttend &a, uint64_t all, uint64_t row, int first, int parts, int lane,
                                  float *top, float *sum, f32x4 *v) {
    const uint32_t D = a.c.dim;
    const float *ml = part_sums(a, all, row);
    const bool holds = lane < (int)D / 4;  // 4 dimensions a lane
    *top = KV_NEG_INF;
    *sum = 0.0f;
    *v = f32x4{0, 0, 0, 0};
    for (int k0 = first; k0 < parts; k0 += STEP * 64) {
        const int mine = k0 + lane * STEP;
        f32x2 x = {KV_NEG_INF, 0.0f};
        if (mine < parts) x = *reinterpret_cast<const f32x2 *>(ml + mine * all * 2);
        const float m = x[0], l = x[1];
        const float now = fmaxf(*top, wave_reduce(m, [](float p, float q) { return fmaxf(p, q); }));
        const float ts = now == KV_NEG_INF ? 0.0f : now;
        const float fade = __builtin_amdgcn_exp2f(m - ts), old = __builtin_amdgcn_exp2f(*top - ts);
        *top = now;
        *sum = *sum * old + wave_reduce(l * fade, [](float p, float q) { return p + q; });
        *v *= old;
        const int n = (parts - k0 + STEP - 1) / STEP < 64 ? (parts - k0 + STEP - 1) / STEP : 64;
        const float *src = a.part + (k0 * all + row) * D + (holds ? lane * 4 : 0);
        for (int k = 0; k < n; k += 8) {
            f32x4 o[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (k + u < n) o[u] = *reinterpret_cast<const f32x4 *>(src + (uint64_t)(k + u) * STEP * all * D);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (k + u < n) *v += o[u] * lane_f32(fade, k + u);
        }
    }
}

template <int DTYPE>
__device__ inline void put_row(const KvAttend &a, uint64_t row, int lane, float top, float sum, const f32x4 &v) {
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (lane < (int)a.c.dim / 4) {
        u32x2 w;
        w[0] = pack2<DTYPE>(v[0] * inv, v[1] * inv);
        w[1] = pack2<DTYPE>(v[2] * inv, v[3] * inv);
        *reinterpret_cast<u32x2 *>(a.out + row * a.c.dim + lane * 4) = w;
    }
    if (lane == 0) put_sum(a, row, top == KV_NEG_INF ? 0.0f : top, sum);
}

template <int DTYPE>
__global__ __launch_bounds__(kThreads) void k_kv_finish(KvAttend a, uint32_t join_blocks) {
    __shared__ f32x4 sm_v[kWaves][64];
    __shared__ float sm_m[16], sm_l[16];
    const uint32_t b = blockIdx.y;
    const int tid = threadIdx.x, wave = wave_uniform(tid / 64), lane = tid % 64, G = (int)a.group;
    const uint64_t heads = (uint64_t)a.c.heads * G, all = a.tokens * heads;
    bool bad;
    const Seq s = sequence(a, b, &bad);
    if (blockIdx.x < join_blocks) {
        const bool few = a.splits <= kFewParts;
        const uint64_t unit = few ? (uint64_t)blockIdx.x * kWaves + wave : blockIdx.x;
        const uint64_t t = unit / heads, hq = unit % heads;
        if (t >= (uint64_t)s.count) return;
        const int parts = parts_of(a, s, (int)((t * G + hq % G) / a.rows));
        if (parts <= 1) return;
        const uint64_t row = (s.first + t) * heads + hq;
        float top, sum;
        f32x4 v;
        if (few) {
            join_parts<1>(a, all, row, 0, parts, lane, &top, &sum, &v);
            put_row<DTYPE>(a, row, lane, top, sum, v);
            return;
        }
        join_parts<kWaves>(a, all, row, wave, parts, lane, &top, &sum, &v);
        if (lane == 0) {
            sm_m[wave] = top;
            sm_l[wave] = sum;
        }
        sm_v[wave][lane] = v;
        __syncthreads();
        if (wave) return;
        top = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
        const float ts = top == KV_NEG_INF ? 0.0f : top;
        sum = 0.0f;
        v = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < kWaves; ++k) {
            const float fade = __builtin_amdgcn_exp2f(sm_m[k] - ts);
            sum += sm_l[k] * fade;
            v += sm_v[k][lane] * fade;
        }
        put_row<DTYPE>(a, row, lane, top, sum, v);
        return;
    }
    // weights of 512 tokens of a head from the kept scores (at most 16 rows)
    const uint32_t y = blockIdx.x - join_blocks, h = y % a.c.heads;
    const int j0 = (int)(y / a.c.heads * kKeptTokens), rows = s.count * G;
    if (j0 >= s.len || rows == 0) return;
    const uint64_t unit = (uint64_t)b * a.c.heads + h;
    // (scores of a page that is none were never written; they are not used)
    float score[2][16], was[2] = {};
    bool there[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int j = j0 + x * kThreads + tid;
        there[x] = j < s.len && (uint64_t)j < a.cap;
        if (there[x]) {
            const float *p = a.scores + (unit * a.score_pages + j / kKvPage) * a.score_rows * kKvPage;
            p += (j % 16 / 4 * 4 + j % 64 / 16) * (int)a.score_rows * 4 + j % 4;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (r < rows) score[x][r] = p[r * 4];
            was[x] = a.weight[unit * a.cap + j];
            there[x] = page_offset(a.c, b, j / kKvPage) != kNoPage;
        }
    }
    if (wave == 0) {  // a row a lane, its parts over the four groups of lanes
        const int r = lane % 16, parts = parts_of(a, s, 0);
        const uint64_t row = (s.first + (r < rows ? r / G : 0)) * heads + (uint64_t)h * G + (r < rows ? r % G : 0);
        float m, inv;
        if (parts > 1) {
            const float *ml = part_sums(a, all, row);
            float top = KV_NEG_INF, sum = 0.0f;
            for (int k = lane / 16; k < parts; k += 4) {
                const f32x2 x = *reinterpret_cast<const f32x2 *>(ml + k * all * 2);
                const float now = fmaxf(top, x[0]), ts = now == KV_NEG_INF ? 0.0f : now;
                sum = sum * __builtin_amdgcn_exp2f(top - ts) + x[1] * __builtin_amdgcn_exp2f(x[0] - ts);
                top = now;
            }
            m = across_groups(top, [](float x, float y) { return fmaxf(x, y); });
            if (m == KV_NEG_INF) m = 0.0f;
            sum = across_groups(sum * __builtin_amdgcn_exp2f(top - m), [](float x, float y) { return x + y; });
            inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        } else {
            const float2 x = a.sums[row];
            m = x.x;
            inv = x.y;
        }
        if (lane < 16) {
            sm_m[r] = m;
            sm_l[r] = inv;
        }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int j = j0 + x * kThreads + tid;
        if (!there[x]) continue;
        const int from = j > s.had ? (j - s.had) * G : 0;  // earlier rows do not see the token
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (r < rows && r >= from)
                sum = __builtin_fmaf(__builtin_amdgcn_exp2f(score[x][r] - sm_m[r]), sm_l[r], sum);
        a.weight[unit * a.cap + j] = was[x] + sum;
    }
}

// Tiles of 16 rows [first, end) of a piece of the rows that see something of
// the page from token `base` on; none: false.
__device__ inline bool piece_tiles(const KvAttend &a, const Seq &s, int base, int piece, int *first, int *end) {
    const int tiles = (s.count * (int)a.group + 15) / 16, each = (int)a.weigh_tiles;
    const int least = base > s.had ? (base - s.had) * (int)a.group / 16 : 0;  // earlier rows see nothing here
    *first = least > piece * each ? least : piece * each;
    *end = tiles < (piece + 1) * each ? tiles : (piece + 1) * each;
    return *first < *end;
}

template <int D, int CODES, int DTYPE>
__global__ __launch_bounds__(kv_weigh_waves(D) * 64) void k_kv_weigh(KvAttend a) {
    constexpr int kSteps = D / 32, kN = (int)kv_weigh_waves(D);
    constexpr int kPieces = D / 8, kPitch = kPieces + 1;  // of 16 bytes; odd, so that rows start in other banks
    __shared__ float sm[kN][kKvPage];
    __shared__ u32x4 sm_q[kN][16 * kPitch];
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
    auto load = [&](int x, bool last) __attribute__((always_inline)) {  // last: some rows may not be there
        const int t0 = wave_uniform(x * 16 / G), v0 = x * 16 - t0 * G, most = last ? rows - x * 16 : 16;
        if (last || !same) place(v0, most);
        const uint16_t *tile = a.q + (int64_t)(s.first + t0) * a.q_row + (int64_t)h * G * a.q_head;
        ml = a.sums[(s.first + t0) * heads + (uint64_t)h * G + sum_at];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) q[i] = load_q8(tile + q_at[i]);
        see = n < most ? see0 + t0 + lane_t : 0;
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
        const bool edge = k == 0 || x * 16 / G + s.had + 1 - base < 64;  // some row misses some token
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
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i / 4][i % 4] = __builtin_fmaf(w[i / 4][i % 4], f, -now.x);
        if (edge) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i >= see_now) w[i / 4][i % 4] = KV_NEG_INF;
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

template <int D, int CODES>
void weigh_go(const KvAttend &a, int dtype, hipStream_t s) {
    const dim3 grid = grid_of(kv_weigh_blocks(a.score_pages, a.weigh_pieces, a.c.heads, a.c.batch)), block(kv_weigh_waves(D) * 64);
    if (dtype == kBf16)
        hipLaunchKernelGGL((k_kv_weigh<D, CODES, kBf16>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((k_kv_weigh<D, CODES, kFp16>), grid, block, 0, s, a);
}

template <int D>
void weigh_codes(const KvAttend &a, int codes, int dtype, hipStream_t s) {
    if (codes == kE4m3)
        weigh_go<D, kE4m3>(a, dtype, s);
    else
        weigh_go<D, kInt8>(a, dtype, s);
}

}  // namespace

hipError_t launch_kv_finish(const KvAttend &a, int dtype, hipStream_t s) {
    const uint32_t units = a.max_new * a.c.heads * a.group;
    const uint32_t join = a.splits == 1 ? 0 : a.splits <= kFewParts ? (units + kWaves - 1) / kWaves : units;
    const uint32_t weigh = a.scores ? (uint32_t)kv_kept_blocks(a.max_len, a.c.heads) : 0;
    if (join + weigh == 0) return hipSuccess;
    const dim3 grid(join + weigh, a.c.batch);
    if (dtype == kBf16)
        hipLaunchKernelGGL((k_kv_finish<kBf16>), grid, dim3(kThreads), 0, s, a, join);
    else
        hipLaunchKernelGGL((k_kv_finish<kFp16>), grid, dim3(kThreads), 0, s, a, join);
    return hipGetLastError();
}

hipError_t launch_kv_weigh(const KvAttend &a, int codes, int dtype, hipStream_t s) {
    if (a.max_len == 0) return hipSuccess;
    switch (a.c.dim) {
        case 64: weigh_codes<64>(a, codes, dtype, s); break;
        case 96: weigh_codes<96>(a, codes, dtype, s); break;
        case 128: weigh_codes<128>(a, codes, dtype, s); break;
        case 192: weigh_codes<192>(a, codes, dtype, s); break;
        case 256: weigh_codes<256>(a, codes, dtype, s); break;
        default: return hipErrorInvalidValue;
    }
    if (a.weigh_part) {
        const dim3 grid((a.max_len + kThreads - 1) / kThreads, a.c.heads, a.c.batch);
        hipLaunchKernelGGL(k_kv_add, grid, dim3(kThreads), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace ac
