// kv_accept.hip -- keeps the accepted path of a tree of drafted tokens.
//
// A sequence holds had + n tokens, the last n of them drafted; of these the
// path i_0 < i_1 < ... is kept.  Place had + k takes the token of place
// had + i_k, which is the same or a later one, so that pages are filled from
// the first one on and a page's tokens are read before any is written there:
// nothing that a later page needs is overwritten.
//
// A token that stays in its page keeps its codes.  One that comes from another
// page is brought to the scale of the page it comes to: for keys and values,
//   e = least e >= -64 with amax(tokens from other pages) <= largest code * 2^e,
//       and at least the page's own where a token of its own stays in it;
// codes become code * 2^(e_from - e), to the nearest code, and where e is not
// what it was the page's own tokens likewise.
//
// One workgroup a (sequence, head).  It is bound by five dependent trips to
// memory (lengths, path, page table, codes, stores): 4.2 us for one tree of 7
// drafts, 13.6 for 256 trees of 20-40 x 8 heads of 128, whose 3 MB are 16 bytes
// here and there.
#include "kv_device.h"

namespace ac {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

__device__ inline int place_page(int place) { return place / kKvPage; }

// What brings a code of one exponent to another.  Only zeros and NaN come from
// 2^128 and more above the scale that is chosen (any other code would have
// raised it), and a zero times infinity would be no number.
__device__ inline float to_scale(int from, int to) { return ldexpf(1.0f, from - to < 127 ? from - to : 127); }

// A code times f; as it is where f is 1.
template <int CODES>
__device__ inline uint8_t again1(uint8_t code, float f) {
    return f == 1.0f ? code : (uint8_t)requant4<CODES>(code, f);
}

template <int CODES>
__device__ inline float finite_magnitude(uint32_t w, int byte) {
    float x;
    if constexpr (CODES == kE4m3)
        x = fabsf(__builtin_amdgcn_cvt_f32_fp8((int)(w >> (8 * byte)), 0));
    else
        x = fabsf((float)(int8_t)(w >> (8 * byte)));
    return x <= 448.0f ? x : 0.0f;  // (a NaN is none)
}

template <int D, int CODES>
__global__ __launch_bounds__(kThreads) void k_kv_accept(KvAccept a) {
    constexpr int kPer = D / 8;
    __shared__ u32x2 sm_k[kKvPage * kPer];
    __shared__ uint8_t sm_v[D * kKvPage];
    __shared__ int sm_src[kKvPage];          // place that a place of the page takes its token from
    __shared__ int sm_exp[2][kKvPage];       // its page's exponents
    __shared__ uint8_t *sm_from[kKvPage];    // its strip
    __shared__ float sm_top[2][kWaves];
    __shared__ int sm_same, sm_bad, sm_none;  // (a word a phase: a wave may be a phase ahead of another's reading)
    const uint32_t h = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x, wave = tid / 64;
    const bool speaks = h == 0;
    uint64_t first;
    int count;
    bool bad;
    new_tokens(a.starts, a.tokens, a.max_new, b, &first, &count, &bad);
    const int len = a.c.lens[b], kept = a.kept[b];
    bad = bad || len < count || (uint64_t)len > a.c.stride * kKvPage || kept < 0 || kept > count || (uint64_t)kept > a.path_stride;
    const int32_t *path = a.path + (uint64_t)b * a.path_stride;
    if (tid == 0) sm_same = sm_bad = sm_none = 0;
    __syncthreads();
    if (!bad) {
        int same = 0, wrong = 0;
        for (int i = tid; i < kept; i += kThreads) {
            const int p = path[i];
            wrong += p <= (i ? path[i - 1] : -1) || p >= count;
            same += p == i;
        }
        if (same) atomicAdd(&sm_same, same);
        if (wrong) atomicAdd(&sm_bad, wrong);
    }
    __syncthreads();
    const int same = sm_same, had = len - count;  // the path's first tokens that are where they belong
    bad = bad || sm_bad;
    if (bad || same == kept) {
        if (speaks && tid == 0) {
            if (bad && a.c.n_invalid) atomicAdd(a.c.n_invalid, 1ull);
            a.lens_out[b] = bad ? len : had + kept;
        }
        return;
    }
    const int j_first = place_page(had + same), j_last = place_page(had + path[kept - 1]);
    {
        int none = 0;
        for (int j = j_first + tid; j <= j_last; j += kThreads) none += page_offset(a.c, b, j) == kNoPage;
        if (none) {
            atomicAdd(&sm_none, none);
            if (speaks && a.c.n_invalid) atomicAdd(a.c.n_invalid, (unsigned long long)none);
        }
    }
    __syncthreads();
    if (speaks && tid == 0) a.lens_out[b] = sm_none ? len : had + kept;
    if (sm_none) return;
    const uint64_t strip = (uint64_t)h * 2 * kKvPage * D;
    for (int j = j_first; j <= place_page(had + kept - 1); ++j) {
        const int base = j * kKvPage;
        const int lo = had + same > base ? had + same - base : 0, hi = had + kept - base < kKvPage ? had + kept - base : kKvPage;
        const int n = hi - lo;
        uint8_t *page = page_at(a.c, b, j);
        float *sc = page_scales(a.c, page, h);
        const int ke0 = exp_of_pow2(sc[0]), ve0 = exp_of_pow2(sc[1]);
        float weight = 0.0f;
        int32_t pos = 0;
        bool planes = false;
        const uint64_t row = ((uint64_t)b * a.c.heads + h) * a.cap;
        if (tid < n) {
            const int src = had + path[base + lo + tid - had];
            uint8_t *from = page_at(a.c, b, place_page(src));
            const float *s = page_scales(a.c, from, h);
            sm_src[tid] = src;
            sm_from[tid] = from + strip;
            sm_exp[0][tid] = exp_of_pow2(s[0]);
            sm_exp[1][tid] = exp_of_pow2(s[1]);
            planes = (uint64_t)src < a.cap;
            if (planes && a.weight) weight = a.weight[row + src];
            if (planes && a.pos) pos = a.pos[row + src];
        }
        __syncthreads();
        float km = 0.0f, vm = 0.0f;
        bool any_far = false, any_own = lo > 0;
        for (int i = 0; i < n; ++i) {
            const bool far = place_page(sm_src[i]) != j;
            any_far |= far;
            any_own |= !far;
        }
        for (int i = tid; i < n * kPer; i += kThreads) {
            const int t = i / kPer, c = i % kPer, src = sm_src[t];
            const u32x2 w = *reinterpret_cast<const u32x2 *>(sm_from[t] + src % kKvPage * D + c * 8);
            sm_k[i] = w;
            if (place_page(src) != j) {
                const float f = pow2(sm_exp[0][t]);
#pragma unroll
                for (int x = 0; x < 8; ++x) km = fmaxf(km, finite_magnitude<CODES>(w[x / 4], x % 4) * f);
            }
        }
        for (int i = tid; i < n * D; i += kThreads) {
            const int d = i / n, t = i - d * n, src = sm_src[t];
            const uint8_t w = sm_from[t][kKvPage * D + d * kKvPage + src % kKvPage];
            sm_v[i] = w;
            if (place_page(src) != j) vm = fmaxf(vm, finite_magnitude<CODES>(w, 0) * pow2(sm_exp[1][t]));
        }
        int ke = ke0, ve = ve0;
        if (any_far) {
            km = wave_max0(km);
            vm = wave_max0(vm);
            if (tid % 64 == 0) {
                sm_top[0][wave] = km;
                sm_top[1][wave] = vm;
            }
        }
        __syncthreads();  // all that the page gives and gets has been read
        if (any_far) {
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                km = fmaxf(km, sm_top[0][w]);
                vm = fmaxf(vm, sm_top[1][w]);
            }
            ke = scale_exp<CODES>(km);
            ve = scale_exp<CODES>(vm);
            if (any_own) {
                ke = ke0 > ke ? ke0 : ke;
                ve = ve0 > ve ? ve0 : ve;
            }
        }
        uint8_t *kc = page + strip, *vc = kc + kKvPage * D;
        for (int i = tid; i < n * kPer; i += kThreads) {
            const int t = i / kPer, c = i % kPer;
            u32x2 w = sm_k[i];
            if (sm_exp[0][t] != ke) {
                const float f = to_scale(sm_exp[0][t], ke);
                w[0] = requant4<CODES>(w[0], f);
                w[1] = requant4<CODES>(w[1], f);
            }
            *reinterpret_cast<u32x2 *>(kc + (lo + t) * D + c * 8) = w;
        }
        for (int i = tid; i < n * D; i += kThreads) {
            const int d = i / n, t = i - d * n;
            vc[d * kKvPage + lo + t] = again1<CODES>(sm_v[i], to_scale(sm_exp[1][t], ve));
        }
        if (lo > 0 && ke != ke0) {
            const float f = to_scale(ke0, ke);
            for (int i = tid; i < lo * kPer; i += kThreads) {
                u32x2 *p = reinterpret_cast<u32x2 *>(kc) + i;
                u32x2 w = *p;
                w[0] = requant4<CODES>(w[0], f);
                w[1] = requant4<CODES>(w[1], f);
                *p = w;
            }
        }
        if (lo > 0 && ve != ve0) {
            const float f = to_scale(ve0, ve);
            for (int i = tid; i < lo * D; i += kThreads) {
                uint8_t *p = vc + i / lo * kKvPage + i % lo;
                *p = again1<CODES>(*p, f);
            }
        }
        if (tid == 0 && any_far) {
            sc[0] = pow2(ke);
            sc[1] = pow2(ve);
        }
        if (planes) {
            if (a.weight) a.weight[row + base + lo + tid] = weight;
            if (a.pos) a.pos[row + base + lo + tid] = pos;
        }
        __syncthreads();  // before LDS is filled again
    }
}

template <int D>
void accept_codes(const KvAccept &a, int codes, hipStream_t s) {
    const dim3 grid(a.c.heads, a.c.batch);
    if (codes == kE4m3)
        hipLaunchKernelGGL((k_kv_accept<D, kE4m3>), grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((k_kv_accept<D, kInt8>), grid, dim3(kThreads), 0, s, a);
}

}  // namespace

hipError_t launch_kv_accept(const KvAccept &a, int codes, hipStream_t s) {
    switch (a.c.dim) {
        case 64: accept_codes<64>(a, codes, s); break;
        case 96: accept_codes<96>(a, codes, s); break;
        case 128: accept_codes<128>(a, codes, s); break;
        case 192: accept_codes<192>(a, codes, s); break;
        case 256: accept_codes<256>(a, codes, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace ac
