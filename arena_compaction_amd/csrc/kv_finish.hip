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
#include "kv_weigh.h"

namespace ac {
namespace {

// Parts of the rows of block rb (1: the first pass has written the result).
__device__ inline int parts_of(const KvAttend &a, const Seq &s, int rb) {
    const int pages = block_pages(a, s, rb, a.mask != nullptr);
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
        // earlier rows do not see the token (what a mask hides has a score of -infinity)
        const int from = !a.mask && j > s.had ? (j - s.had) * G : 0;
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (r < rows && r >= from)
                sum = __builtin_fmaf(__builtin_amdgcn_exp2f(score[x][r] - sm_m[r]), sm_l[r], sum);
        a.weight[unit * a.cap + j] = was[x] + sum;
    }
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

template hipError_t launch_kv_weigh<kPlain>(const KvAttend &a, int codes, int dtype, hipStream_t s);

}  // namespace ac
