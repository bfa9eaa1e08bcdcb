// kv_evict.hip -- keeps `budget` tokens of every (sequence, head).
//
// Kept are first the safe tokens (position below `sink`, or among the last
// `recent`), then those of largest weight; equal weights go to the lowest
// place, a NaN counts as +infinity.  Kept tokens inside the first `budget`
// places stay where they are; the places of dropped ones (holes) take the
// kept tokens behind the budget, both in ascending order.
//
//   k_kv_select  one workgroup a (sequence, head): a radix select of the
//                budget-th key, then two ordered sweeps that turn flags into
//                the list src[place] by prefix sums;
//   k_kv_fold    one workgroup a (page, head): gathers the page's 64 tokens
//                by that list, finds the new scale and writes new codes.
//                Pages without a hole are left alone.
// Read places lie behind the budget or in the workgroup's own strip, and
// written ones in its own strip: no workgroup reads what another writes.
#include "kv_device.h"

namespace ac {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kDigits = 256;  // bins of a radix pass
constexpr int kFoldThreads = 256;

// Larger weight, larger key; -0 and +0 are one key, NaN that of +infinity.
__device__ inline uint32_t weight_key(float w) {
    uint32_t u = __builtin_bit_cast(uint32_t, w + 0.0f);
    if (w != w) u = 0x7F800000u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct Row {
    const float *w;
    const int32_t *pos;
    int32_t sink;
    int64_t border;
    __device__ bool safe(int i) const { return pos[i] < sink || (int64_t)pos[i] >= border; }
};

// Exclusive prefix of x over the workgroup, and the total.
__device__ inline int block_scan(int x, int *red, int *total) {
    const int incl = wave_incl_scan(x, [](int p, int q) { return p + q; });
    __syncthreads();
    if (threadIdx.x % 64 == 63) red[threadIdx.x / 64] = incl;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int k = 0; k < kSelWaves; ++k) {
        const int v = red[k];
        if (k < (int)(threadIdx.x / 64)) before += v;
        all += v;
    }
    *total = all;
    return before + incl - x;
}

// The tokens of a sequence that take part; -1 where its length or a page is
// out of range (nothing of the sequence is touched then).
__device__ inline int evict_len(const KvEvict &a, uint32_t b, int *bad_pages) {
    const int64_t n = a.c.lens[b];
    *bad_pages = 0;
    if (n < 0 || n > (int64_t)a.max_len || n > (int64_t)a.cap) return -1;
    return (int)n;
}

__global__ __launch_bounds__(kSelThreads) void k_kv_select(KvEvict a) {
    __shared__ int red[kSelWaves];
    __shared__ uint32_t hist[kDigits];
    __shared__ uint32_t sh_prefix;
    __shared__ int sh_need;
    const uint32_t h = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x, K = (int)a.budget;
    int bad_pages = 0;
    int n = evict_len(a, b, &bad_pages);
    int32_t *src = a.src + ((uint64_t)b * a.c.heads + h) * a.budget;
    if (n > K) {
        int bad = 0;
        for (int j = tid; j * kKvPage < n; j += kSelThreads) bad += page_at(a.c, b, j) == nullptr;
        block_scan(bad, red, &bad_pages);
    }
    if (n < 0 || bad_pages) {  // src[0] = -1: the second kernel passes over the row
        if (tid == 0) {
            src[0] = -1;
            if (h == 0 && a.c.n_invalid)
                atomicAdd(a.c.n_invalid, (unsigned long long)(bad_pages ? bad_pages : 1));
        }
        return;
    }
    const uint64_t at = ((uint64_t)b * a.c.heads + h) * a.cap;
    const uint64_t to = ((uint64_t)b * a.c.heads + h) * a.cap_out;
    const Row r{a.weight + at, a.pos + at, a.sink, (int64_t)a.next_pos[b] - a.recent};
    if (h == 0 && tid == 0) a.lens_out[b] = n < K ? n : K;
    if (n <= K) {
        if (tid == 0) src[0] = -1;
        for (int i = tid; i < n; i += kSelThreads) {
            a.weight_out[to + i] = r.w[i];
            a.pos_out[to + i] = r.pos[i];
        }
        return;
    }
    // safe tokens: all kept if they fit, else the choice is among them alone
    int mine = 0, safe_total;
    for (int i = tid; i < n; i += kSelThreads) mine += r.safe(i);
    block_scan(mine, red, &safe_total);
    const bool among_safe = safe_total >= K;
    if (tid == 0) {
        sh_prefix = 0;
        sh_need = among_safe ? K : K - safe_total;
    }
    // the need-th largest key of the candidates, 8 bits a pass
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < kDigits; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        const uint32_t prefix = sh_prefix;
        for (int i = tid; i < n; i += kSelThreads) {
            if (r.safe(i) != among_safe) continue;
            const uint32_t key = weight_key(r.w[i]);
            if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(&hist[(key >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            int need = sh_need, d = kDigits - 1;
            while (d > 0 && (int)hist[d] < need) need -= (int)hist[d--];
            sh_need = need;
            sh_prefix = prefix | ((uint32_t)d << shift);
        }
        __syncthreads();
    }
    const uint32_t edge = sh_prefix;
    const int ties = sh_need;  // of the tokens at the edge, the first `ties`
    int tied = 0, holes = 0, moved = 0;
    // holes in ascending order, beside the list they are filled in
    int32_t *hole = a.src + (uint64_t)a.c.batch * a.c.heads * a.budget +
                    ((uint64_t)b * a.c.heads + h) * a.budget;
    for (int i0 = 0; i0 < n; i0 += kSelThreads) {
        const int i = i0 + tid;
        bool in = i < n, safe = false, tie = false, keep = false;
        if (in) {
            safe = r.safe(i);
            if (safe != among_safe) {
                keep = safe;  // safe ones that fit, all; else no other
            } else {
                const uint32_t key = weight_key(r.w[i]);
                keep = key > edge;
                tie = key == edge;
            }
        }
        int total;
        const int rank = block_scan(tie, red, &total);
        if (tie) keep = tied + rank < ties;
        tied += total;
        const bool hl = in && i < K && !keep;
        const int hrank = block_scan(hl, red, &total);
        if (hl) hole[holes + hrank] = i;
        holes += total;
        if (in && i < K && keep) {
            src[i] = i;
            a.weight_out[to + i] = r.w[i];
            a.pos_out[to + i] = r.pos[i];
        }
        const bool mv = in && i >= K && keep;
        const int mrank = block_scan(mv, red, &total);  // its barriers also order hole[]
        if (mv) {
            const int p = hole[moved + mrank];
            src[p] = i;
            a.weight_out[to + p] = r.w[i];
            a.pos_out[to + p] = r.pos[i];
        }
        moved += total;
    }
}

template <int CODES>
__global__ __launch_bounds__(kFoldThreads) void k_kv_fold(KvEvict a) {
    __shared__ const uint8_t *from[kKvPage];
    __shared__ float scale[2][kKvPage];
    __shared__ float red[2][kFoldThreads / 64];
    const uint32_t j = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, lane = tid % 64;
    const int D = (int)a.c.dim;
    const int32_t *src = a.src + ((uint64_t)b * a.c.heads + h) * a.budget;
    if (src[0] < 0) return;
    const int32_t s = src[j * kKvPage + lane];
    if (__builtin_amdgcn_ballot_w64(s != (int32_t)(j * kKvPage + lane)) == 0) return;
    if (tid < kKvPage) {
        uint8_t *page = page_at(a.c, b, (uint64_t)s / kKvPage);
        const float *sc = page_scales(a.c, page, h);
        from[tid] = page + (uint64_t)h * 2 * kKvPage * D;
        scale[0][tid] = sc[0];
        scale[1][tid] = sc[1];
    }
    __syncthreads();
    uint8_t *page = page_at(a.c, b, j);
    float *sc = page_scales(a.c, page, h);
    uint8_t *kc = page + (uint64_t)h * 2 * kKvPage * D, *vc = kc + kKvPage * D;
    // keys: a dword is 4 dimensions of a token; values: 4 tokens of a dimension
    constexpr int kMax = kKvPage * (int)kKvMaxDim / 4 / kFoldThreads;  // 16 of each
    uint32_t kw[kMax], vw[kMax];
    const int per = D / 4, items = kKvPage * D / 4;
    float km = 0.0f, vm = 0.0f;
#pragma unroll
    for (int i = 0; i < kMax; ++i) {
        const int item = tid + i * kFoldThreads;
        if (item < items) {
            const int t = item / per, d = item % per * 4;
            const int place = src[j * kKvPage + t] % kKvPage;
            kw[i] = *reinterpret_cast<const uint32_t *>(from[t] + place * D + d);
            const int dv = item / (kKvPage / 4), t0 = item % (kKvPage / 4) * 4;
            vw[i] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int pl = src[j * kKvPage + t0 + e] % kKvPage;
                vw[i] |= (uint32_t)from[t0 + e][kKvPage * D + dv * kKvPage + pl] << (8 * e);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kMax; ++i) {
        const int item = tid + i * kFoldThreads;
        if (item < items) {
            const float f = scale[0][item / per];
            const float *g = &scale[1][item % (kKvPage / 4) * 4];
            km = fmaxf(km, finite_abs(code_value<CODES, 0>(kw[i]) * f));
            km = fmaxf(km, finite_abs(code_value<CODES, 1>(kw[i]) * f));
            km = fmaxf(km, finite_abs(code_value<CODES, 2>(kw[i]) * f));
            km = fmaxf(km, finite_abs(code_value<CODES, 3>(kw[i]) * f));
            vm = fmaxf(vm, finite_abs(code_value<CODES, 0>(vw[i]) * g[0]));
            vm = fmaxf(vm, finite_abs(code_value<CODES, 1>(vw[i]) * g[1]));
            vm = fmaxf(vm, finite_abs(code_value<CODES, 2>(vw[i]) * g[2]));
            vm = fmaxf(vm, finite_abs(code_value<CODES, 3>(vw[i]) * g[3]));
        }
    }
    km = wave_max0(km);
    vm = wave_max0(vm);
    if (lane == 0) {
        red[0][tid / 64] = km;
        red[1][tid / 64] = vm;
    }
    __syncthreads();  // all of the page has been read, too
    km = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    vm = fmaxf(fmaxf(red[1][0], red[1][1]), fmaxf(red[1][2], red[1][3]));
    const int ke = scale_exp<CODES>(km), ve = scale_exp<CODES>(vm);
    const float ki = pow2(-ke), vi = pow2(-ve);
#pragma unroll
    for (int i = 0; i < kMax; ++i) {
        const int item = tid + i * kFoldThreads;
        if (item < items) {
            const int t = item / per, d = item % per * 4;
            *reinterpret_cast<uint32_t *>(kc + t * D + d) = requant4<CODES>(kw[i], scale[0][t] * ki);
            const int dv = item / (kKvPage / 4), t0 = item % (kKvPage / 4) * 4;
            const float *g = &scale[1][t0];
            *reinterpret_cast<uint32_t *>(vc + dv * kKvPage + t0) = to_codes4<CODES>(
                code_value<CODES, 0>(vw[i]) * (g[0] * vi), code_value<CODES, 1>(vw[i]) * (g[1] * vi),
                code_value<CODES, 2>(vw[i]) * (g[2] * vi), code_value<CODES, 3>(vw[i]) * (g[3] * vi));
        }
    }
    if (tid == 0) {
        sc[0] = pow2(ke);
        sc[1] = pow2(ve);
    }
}

}  // namespace

hipError_t launch_kv_evict(const KvEvict &a, int codes, hipStream_t s) {
    hipLaunchKernelGGL(k_kv_select, dim3(a.c.heads, a.c.batch), dim3(kSelThreads), 0, s, a);
    const dim3 grid(a.budget / kKvPage, a.c.heads, a.c.batch);
    if (codes == kE4m3)
        hipLaunchKernelGGL((k_kv_fold<kE4m3>), grid, dim3(kFoldThreads), 0, s, a);
    else
        hipLaunchKernelGGL((k_kv_fold<kInt8>), grid, dim3(kFoldThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace ac
