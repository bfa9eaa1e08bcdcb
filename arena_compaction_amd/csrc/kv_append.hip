// kv_append.hip -- new tokens into the pages of the 8-bit cache.
//
// For each (page, head) a call adds tokens to, and for keys and values each:
//   e     = least e >= -64 with amax(new tokens) <= largest code * 2^e,
//           and at least the page's exponent where it holds older tokens;
//   code  = x * 2^-e to the nearest code (ties to even), clamped;
//   older = code * 2^(e_before - e) to the nearest code, where e grew.
// The scale is a power of two, so multiplying by it is exact and the only
// rounding is the one to a code (half a step: e4m3 2^-4 of the value, int8
// half a unit); it grows at most once a page for a growing maximum.
//
// One workgroup a (page, head): every code of the strip and both scales are
// its own, so nothing is shared and the result does not depend on order.
// The new tokens' elements are read once, kept in registers through the
// reduction of the maximum, and written as codes; values go through LDS,
// since they lie token by token in the input and dimension by dimension in
// the page.
#include "kv_device.h"

namespace ac {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kTileStride = kKvPage + 4;  // bytes; rows start in other banks

// (2-byte alignment will do: gfx950 reads 16 bytes from any address)
template <int DTYPE>
__device__ inline void load8(const uint16_t *p, float (&x)[8]) {
    uint16_t h[8];
    __builtin_memcpy(h, p, 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_float<DTYPE>(h[i]);
}

template <int D, int CODES, int DTYPE>
__global__ __launch_bounds__(kAppendThreads) void k_kv_append(KvAppend a) {
    constexpr int kPer = D / 8;                              // 8-element pieces of a token
    constexpr int kItems = kKvPage * kPer / kAppendThreads;  // pieces a lane holds
    __shared__ float red[2][kAppendThreads / 64];
    __shared__ __align__(16) uint8_t tile[D * kTileStride];
    const uint32_t h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x;
    uint64_t first;
    int count;
    bool bad;
    new_tokens(a.starts, a.tokens, a.max_new, b, &first, &count, &bad);
    const int64_t len = a.c.lens[b];
    const bool fits = len >= 0 && len + count <= (int64_t)(a.c.stride * kKvPage);
    if (bad || !fits) {  // nothing of this sequence is written
        if (a.c.n_invalid && blockIdx.x == 0 && h == 0 && tid == 0) atomicAdd(a.c.n_invalid, 1ull);
        return;
    }
    const int64_t j = len / kKvPage + blockIdx.x, base = j * kKvPage;
    const int lo = (int)(len > base ? len - base : 0);
    const int64_t end = len + count - base;
    const int hi = (int)(end < kKvPage ? end : kKvPage);
    if (hi <= lo) return;
    uint8_t *page = page_at(a.c, b, j);
    if (!page) {
        if (a.c.n_invalid && h == 0 && tid == 0) atomicAdd(a.c.n_invalid, 1ull);
        return;
    }
    const uint64_t src = first + (uint64_t)(base + lo - len);  // the input's token at place lo
    float *sc = page_scales(a.c, page, h);
    uint8_t *kc = page + (uint64_t)h * 2 * kKvPage * D, *vc = kc + kKvPage * D;
    const int n = (hi - lo) * kPer;

    float kx[kItems][8], vx[kItems][8];
    float km = 0.0f, vm = 0.0f;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int item = tid + i * kAppendThreads;
        if (item < n) {
            const uint64_t t = src + item / kPer;
            const int d = item % kPer * 8;
            load8<DTYPE>(a.k + (int64_t)t * a.k_row + h * a.k_head + d, kx[i]);
            load8<DTYPE>(a.v + (int64_t)t * a.v_row + h * a.v_head + d, vx[i]);
        }
    }
    const int ke0 = exp_of_pow2(sc[0]), ve0 = exp_of_pow2(sc[1]);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (tid + i * kAppendThreads < n) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                km = fmaxf(km, finite_abs(kx[i][e]));
                vm = fmaxf(vm, finite_abs(vx[i][e]));
            }
        }
    }
    km = wave_max0(km);
    vm = wave_max0(vm);
    if (tid % 64 == 0) {
        red[0][tid / 64] = km;
        red[1][tid / 64] = vm;
    }
    __syncthreads();
    km = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    vm = fmaxf(fmaxf(red[1][0], red[1][1]), fmaxf(red[1][2], red[1][3]));
    int ke = scale_exp<CODES>(km), ve = scale_exp<CODES>(vm);
    if (lo > 0) {
        ke = ke0 > ke ? ke0 : ke;
        ve = ve0 > ve ? ve0 : ve;
    }
    // -185 at the least: in the range of ldexp, below that of a float's bits
    const float kf = lo > 0 ? ldexpf(1.0f, ke0 - ke) : 1.0f;
    const float vf = lo > 0 ? ldexpf(1.0f, ve0 - ve) : 1.0f;
    const float ki = pow2(-ke), vi = pow2(-ve);

#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int item = tid + i * kAppendThreads;
        if (item < n) {
            const int t = lo + item / kPer, d = item % kPer * 8;
            const float *x = kx[i];
            u32x2 w;
            w[0] = to_codes4<CODES>(x[0] * ki, x[1] * ki, x[2] * ki, x[3] * ki);
            w[1] = to_codes4<CODES>(x[4] * ki, x[5] * ki, x[6] * ki, x[7] * ki);
            *reinterpret_cast<u32x2 *>(kc + t * D + d) = w;
            const float *y = vx[i];
            w[0] = to_codes4<CODES>(y[0] * vi, y[1] * vi, y[2] * vi, y[3] * vi);
            w[1] = to_codes4<CODES>(y[4] * vi, y[5] * vi, y[6] * vi, y[7] * vi);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                tile[(d + e) * kTileStride + t] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
        }
    }
    if (lo > 0 && kf != 1.0f) {
        for (int i = tid; i < lo * kPer; i += kAppendThreads) {
            u32x2 *p = reinterpret_cast<u32x2 *>(kc) + i;
            u32x2 w = *p;
            w[0] = requant4<CODES>(w[0], kf);
            w[1] = requant4<CODES>(w[1], kf);
            *p = w;
        }
    }
    __syncthreads();
    // four tokens of one dimension at a time; a dword that also holds places
    // outside [lo, hi) is read first, older tokens in it brought to the new
    // scale, places behind the last one left as they are
    const int q0 = (vf != 1.0f) ? 0 : lo / 4, q1 = (hi + 3) / 4, nq = q1 - q0;
    for (int i = tid; i < nq * D; i += kAppendThreads) {
        const int d = i / nq, q = q0 + i % nq;
        uint32_t *p = reinterpret_cast<uint32_t *>(vc + d * kKvPage) + q;
        uint32_t w = 0;
        if (4 * q + 4 > lo) w = *reinterpret_cast<const uint32_t *>(tile + d * kTileStride + 4 * q);
        if (4 * q < lo || 4 * q + 4 > hi) {
            const uint32_t was = *p, again = vf != 1.0f ? requant4<CODES>(was, vf) : was;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 4 * q + e;
                const uint32_t m = 255u << (8 * e);
                if (t < lo) w = (w & ~m) | (again & m);
                if (t >= hi) w = (w & ~m) | (was & m);
            }
        }
        *p = w;
    }
    if (tid == 0) {
        sc[0] = pow2(ke);
        sc[1] = pow2(ve);
    }
    if (tid >= lo && tid < hi) {
        const uint64_t at = (uint64_t)base + tid;
        if (at < a.cap) {
            const uint64_t i = ((uint64_t)b * a.c.heads + h) * a.cap + at;
            if (a.weight) a.weight[i] = 0.0f;
            if (a.pos)
                a.pos[i] = (a.first_pos ? a.first_pos[b] : (int32_t)len) +
                           (int32_t)(base + tid - len);
        }
    }
}

__global__ void k_kv_zero(unsigned long long *p) {
    if (threadIdx.x == 0 && blockIdx.x == 0) *p = 0;
}

template <int D, int CODES>
void append_go(const KvAppend &a, int dtype, dim3 grid, hipStream_t s) {
    if (dtype == kBf16)
        hipLaunchKernelGGL((k_kv_append<D, CODES, kBf16>), grid, dim3(kAppendThreads), 0, s, a);
    else
        hipLaunchKernelGGL((k_kv_append<D, CODES, kFp16>), grid, dim3(kAppendThreads), 0, s, a);
}

template <int D>
void append_codes(const KvAppend &a, int codes, int dtype, dim3 grid, hipStream_t s) {
    if (codes == kE4m3)
        append_go<D, kE4m3>(a, dtype, grid, s);
    else
        append_go<D, kInt8>(a, dtype, grid, s);
}

}  // namespace

hipError_t launch_kv_zero(uint64_t *p, hipStream_t s) {
    hipLaunchKernelGGL(k_kv_zero, dim3(1), dim3(64), 0, s,
                       reinterpret_cast<unsigned long long *>(p));
    return hipGetLastError();
}

hipError_t launch_kv_append(const KvAppend &a, int codes, int dtype, hipStream_t s) {
    // pages that max_new tokens can touch, wherever in a page they begin
    const dim3 grid((a.max_new + kKvPage - 2) / kKvPage + 1, a.c.heads, a.c.batch);
    switch (a.c.dim) {
        case 64: append_codes<64>(a, codes, dtype, grid, s); break;
        case 96: append_codes<96>(a, codes, dtype, grid, s); break;
        case 128: append_codes<128>(a, codes, dtype, grid, s); break;
        case 192: append_codes<192>(a, codes, dtype, grid, s); break;
        case 256: append_codes<256>(a, codes, dtype, grid, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace ac
