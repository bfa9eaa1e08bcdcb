// kv_weigh.hip -- the weight that every cached token receives:
//   weight_j += sum_r 2^(t_rj - m_r) / l_r
// over the query rows r that see token j, once each row's m and l are known.
//
//   k_kv_weigh_kept  few rows: from the scores that attention kept;
//   k_kv_weigh       makes the scores again: one workgroup a (page, head)
//                    holds the page's keys and goes over all the rows that
//                    see it.
// A token belongs to one workgroup, and its rows are added in one order,
// whatever else runs: no atomics, the same bits every time.
#include "kv_rows.h"

namespace ac {
namespace {

__global__ __launch_bounds__(kThreads) void k_kv_weigh_kept(KvAttend a) {
    const uint32_t h = blockIdx.y, b = blockIdx.z;
    const int G = (int)a.group, j = (int)(blockIdx.x * kThreads + threadIdx.x);
    bool bad;
    const Seq s = sequence(a, b, &bad);
    if (j >= s.len || (uint64_t)j >= a.cap) return;
    const int rows = s.count * G, from = j > s.had ? (j - s.had) * G : 0;
    if (from >= rows || page_offset(a.c, b, j / kKvPage) == kNoPage) return;
    const uint64_t unit = (uint64_t)b * a.c.heads + h, heads = (uint64_t)a.c.heads * G;
    const float *p = a.scores + (unit * a.score_pages + j / kKvPage) * a.score_rows * kKvPage + j % kKvPage;
    const float2 *sums = a.sums + s.first * heads + (uint64_t)h * G;
    float sum = 0.0f;
#pragma unroll 4
    for (int r = from; r < rows; ++r) {
        const float2 ml = sums[r / G * heads + r % G];
        sum = __builtin_fmaf(__builtin_amdgcn_exp2f(p[r * kKvPage] - ml.x), ml.y, sum);
    }
    a.weight[unit * a.cap + j] += sum;
}

template <int D, int CODES, int DTYPE>
__global__ __launch_bounds__(D <= 96 ? 1024 : 512) void k_kv_weigh(KvAttend a) {
    constexpr int kSteps = D / 32, kN = D <= 96 ? 16 : 8, kStride = kN * 16;  // waves, rows a turn
    __shared__ float sm[kN][kKvPage];
    const uint32_t h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, wave = wave_uniform(tid / 64), lane = tid % 64;
    const int n = lane % 16, g = lane / 16, G = (int)a.group;
    bool bad;
    const Seq s = sequence(a, b, &bad);
    const int p = blockIdx.x, base = p * kKvPage;
    if (base >= s.len || s.count == 0) return;
    const uint64_t off = wave_uniform(page_offset(a.c, b, p));
    if (off == kNoPage) return;
    const float f = a.scale * kLog2e * page_scales(a.c, a.c.arena + off, h)[0];
    u32x4 kk[4][kSteps];
    {
        uint32_t kraw[4][D / 16];
        load_keys<D>(a.c.arena + off + (uint64_t)h * 2 * kKvPage * D, lane, kraw);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int st = 0; st < kSteps; ++st)
                kk[tt][st] = widen8<CODES, DTYPE>(kraw[tt][2 * st], kraw[tt][2 * st + 1]);
    }
    float acc[16] = {};
    const int rows = s.count * G;
    const uint64_t heads = (uint64_t)a.c.heads * G;
    // this lane's row, its token and head among the group's, and where its
    // query and sums are; kStride rows on in each turn
    int r = (base > s.had ? (base - s.had) * G / 16 * 16 : 0) + wave * 16 + n;  // earlier rows see nothing here
    int t = r / G, hg = r - t * G;
    const int dt = kStride / G, dg = kStride - dt * G;
    const uint16_t *q = a.q + (int64_t)(s.first + t) * a.q_row + (int64_t)(h * G + hg) * a.q_head;
    const float2 *sums = a.sums + (s.first + t) * heads + (uint64_t)h * G + hg;
    const int64_t q_on = dt * a.q_row + dg * a.q_head, q_wrap = a.q_row - G * a.q_head;
    const int64_t s_on = (int64_t)dt * heads + dg, s_wrap = (int64_t)heads - G;
    u32x4 qn[kSteps];
    float2 mln = make_float2(0.0f, 0.0f);
    auto load = [&]() {
#pragma unroll
        for (int st = 0; st < kSteps; ++st) qn[st] = u32x4{0, 0, 0, 0};
        if (r < rows) {
            mln = *sums;
#pragma unroll
            for (int st = 0; st < kSteps; ++st) qn[st] = load_q8(q + dim_of<D>(st, g), a.vec_q);
        }
    };
    load();
    const int turns = (rows - (r - n) + kStride - 1) / kStride;  // the same in all lanes
    for (int x = 0; x < turns; ++x) {
        const int see = r < rows ? s.had + t + 1 - base - g * 16 : 0;
        const float2 ml = mln;
        f32x4 w[4];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
            w[tt] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int st = 0; st < kSteps; ++st) w[tt] = mfma16<DTYPE>(kk[tt][st], qn[st], w[tt]);
        }
        r += kStride;
        t += dt;
        hg += dg;
        q += q_on;
        sums += s_on;
        if (hg >= G) {
            hg -= G;
            ++t;
            q += q_wrap;
            sums += s_wrap;
        }
        load();
        if (__builtin_amdgcn_ballot_w64(see < 16)) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(w[i / 4][i % 4], f, -ml.x));
                if (i < see) acc[i] = __builtin_fmaf(e, ml.y, acc[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(w[i / 4][i % 4], f, -ml.x));
                acc[i] = __builtin_fmaf(e, ml.y, acc[i]);
            }
        }
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
    if (tid < kKvPage && base + tid < s.len && (uint64_t)(base + tid) < a.cap) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kN; ++k) sum += sm[k][tid];
        a.weight[((uint64_t)b * a.c.heads + h) * a.cap + base + tid] += sum;
    }
}

template <int D, int CODES>
void weigh_go(const KvAttend &a, int dtype, hipStream_t s) {
    const dim3 grid((a.max_len + kKvPage - 1) / kKvPage, a.c.heads, a.c.batch), block(D <= 96 ? 1024 : 512);
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

hipError_t launch_kv_weigh(const KvAttend &a, int codes, int dtype, hipStream_t s) {
    if (a.max_len == 0) return hipSuccess;
    if (a.scores) {
        hipLaunchKernelGGL(k_kv_weigh_kept, dim3((a.max_len + kThreads - 1) / kThreads, a.c.heads, a.c.batch),
                           dim3(kThreads), 0, s, a);
        return hipGetLastError();
    }
    switch (a.c.dim) {
        case 64: weigh_codes<64>(a, codes, dtype, s); break;
        case 96: weigh_codes<96>(a, codes, dtype, s); break;
        case 128: weigh_codes<128>(a, codes, dtype, s); break;
        case 192: weigh_codes<192>(a, codes, dtype, s); break;
        case 256: weigh_codes<256>(a, codes, dtype, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace ac
