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
// its own, so nothing is shared and the result does not depend on order.  A
// lane takes 4 tokens x 8 dimensions of both: in the input 16 bytes a token,
// in the page 8 bytes of each key row and 4 of each value row, so that the
// values turn from token by token to dimension by dimension within the lane
// (through LDS, byte by byte, 13,000 tokens of 8 heads took 26 us where this
// takes 19: 81 MB, 4.2 TB/s).  The input is read once and kept in its 16 bits
// through the reduction of the maximum.
#include "kv_device.h"

namespace ac {
namespace {

// (2-byte alignment will do: gfx950 reads 16 bytes from any address)
__device__ inline u32x4 load8(const uint16_t *p) {
    u32x4 r;
    __builtin_memcpy(&r, p, 16);
    return r;
}

// Two 16-bit numbers' magnitudes as bits, which ascend with them: the largest
// finite ones go to `most`; the top bits of `odd` are set by what is not finite.
template <int DTYPE>
__device__ inline void max_bits(uint32_t w, uint32_t &most, uint32_t &odd) {
    const uint32_t m = w & 0x7FFF7FFFu;
    const uint32_t past = (m + (DTYPE == kBf16 ? 0x00800080u : 0x04000400u)) & 0x80008000u;  // 0x8000 less infinity's
    odd |= past;
    most = max_u16x2(most, m & ~((past >> 15) * 0xFFFFu));
}

// Four finite numbers times inv, a scale's inverse that brings them within
// the codes' range, to the nearest codes.
template <int CODES>
__device__ inline uint32_t finite_codes4(float a, float b, float c, float d, float inv) {
    if constexpr (CODES == kE4m3) {
        int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
        r = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, r, true);
        return (uint32_t)r;
    } else {
        // 1.5 * 2^23 added: a float's last place is then 1, so the sum is
        // rounded to a whole number (ties to even), its low byte the code
        const float magic = 12582912.0f;
        const uint32_t x = __builtin_bit_cast(uint32_t, __builtin_fmaf(a, inv, magic));
        const uint32_t y = __builtin_bit_cast(uint32_t, __builtin_fmaf(b, inv, magic));
        const uint32_t z = __builtin_bit_cast(uint32_t, __builtin_fmaf(c, inv, magic));
        const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_fmaf(d, inv, magic));
        return __builtin_amdgcn_perm(__builtin_amdgcn_perm(w, z, 0x0C0C0400u), __builtin_amdgcn_perm(y, x, 0x0C0C0400u),
                                     0x05040100u);
    }
}

// The same for any numbers where `odd` says that some are not finite.
template <int CODES>
__device__ inline uint32_t codes4(float a, float b, float c, float d, float inv, bool odd) {
    return odd ? to_codes4<CODES>(a * inv, b * inv, c * inv, d * inv) : finite_codes4<CODES>(a, b, c, d, inv);
}

template <int DTYPE>
__device__ inline float nth(const u32x4 &x, int i) {
    return to_float<DTYPE>((uint16_t)(x[i / 2] >> (16 * (i % 2))));
}

constexpr int kPitch = 20;  // dwords of a value row in LDS: 16 and a gap, so that rows start in other banks

template <int D, int CODES, int DTYPE>
__global__ __launch_bounds__(2 * D) void k_kv_append(KvAppend a) {
    constexpr int kN = 2 * D, kPer = D / 8;  // lanes; pieces of 8 dimensions
    __shared__ float red[2][kN / 64];
    __shared__ __align__(16) uint32_t turn[D * kPitch];
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
    const int64_t src = (int64_t)first + base - len;  // the input's token at place 0, were it there
    float *sc = page_scales(a.c, page, h);
    uint8_t *kc = page + (uint64_t)h * 2 * kKvPage * D, *vc = kc + kKvPage * D;
    const int d = tid % kPer * 8, q = lo / 4 + tid / kPer, t0 = 4 * q;
    const bool mine = t0 < hi;

    u32x4 k[4], v[4];
    float km = 0.0f, vm = 0.0f;
    if (mine) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // for places without a new token the nearest one that has
            const int t = t0 + e < lo ? lo : t0 + e < hi ? t0 + e : hi - 1;
            k[e] = load8(a.k + (src + t) * a.k_row + h * a.k_head + d);
            v[e] = load8(a.v + (src + t) * a.v_row + h * a.v_head + d);
        }
    }
    const int ke0 = exp_of_pow2(sc[0]), ve0 = exp_of_pow2(sc[1]);
    uint32_t odd_bits = 0;
    if (mine) {
        uint32_t kb = 0, vb = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                max_bits<DTYPE>(k[e][i], kb, odd_bits);
                max_bits<DTYPE>(v[e][i], vb, odd_bits);
            }
        km = fmaxf(to_float<DTYPE>((uint16_t)kb), to_float<DTYPE>((uint16_t)(kb >> 16)));
        vm = fmaxf(to_float<DTYPE>((uint16_t)vb), to_float<DTYPE>((uint16_t)(vb >> 16)));
    }
    const bool odd = __builtin_amdgcn_ballot_w64(odd_bits != 0) != 0;
    km = wave_max0(km);
    vm = wave_max0(vm);
    if (tid % 64 == 0) {
        red[0][tid / 64] = km;
        red[1][tid / 64] = vm;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kN / 64; ++w) {
        km = fmaxf(km, red[0][w]);
        vm = fmaxf(vm, red[1][w]);
    }
    int ke = scale_exp<CODES>(km), ve = scale_exp<CODES>(vm);
    if (lo > 0) {
        ke = ke0 > ke ? ke0 : ke;
        ve = ve0 > ve ? ve0 : ve;
    }
    // -185 at the least: in the range of ldexp, below that of a float's bits
    const float kf = lo > 0 ? ldexpf(1.0f, ke0 - ke) : 1.0f;
    const float vf = lo > 0 ? ldexpf(1.0f, ve0 - ve) : 1.0f;
    const float ki = pow2(-ke), vi = pow2(-ve);

    // A page that is filled whole passes its value rows through LDS and writes
    // 16 bytes a lane: 4 bytes a lane, as codes are made, would reach L2 in
    // pieces of 16 (four quads of tokens a wave), 22 us for a prompt's pages
    // where this takes 19.
    const bool whole = lo == 0 && hi == kKvPage;
    if (mine) {
        // dwords that also hold places outside [lo, hi) are read first: older
        // tokens in them are brought to the new scale, places behind the last
        // one left as they are
        uint32_t fresh = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (t0 + e >= lo && t0 + e < hi) fresh |= 255u << (8 * e);
        const int old = lo - t0;
        const uint32_t older = old <= 0 ? 0u : (1u << (8 * old)) - 1u;  // old < 4, since q >= lo / 4
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t *p = reinterpret_cast<uint32_t *>(vc + (d + i) * kKvPage + t0);
            uint32_t w = codes4<CODES>(nth<DTYPE>(v[0], i), nth<DTYPE>(v[1], i), nth<DTYPE>(v[2], i), nth<DTYPE>(v[3], i),
                                       vi, odd);
            if (whole) {
                turn[(d + i) * kPitch + (q ^ (d / 16 % 4 * 4))] = w;
                continue;
            }
            if (fresh != ~0u) {
                const uint32_t was = *p, again = vf != 1.0f ? requant4<CODES>(was, vf) : was;
                w = (w & fresh) | (again & older) | (was & ~(fresh | older));
            }
            *p = w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (t0 + e >= lo && t0 + e < hi) {
                u32x2 w;
                w[0] = codes4<CODES>(nth<DTYPE>(k[e], 0), nth<DTYPE>(k[e], 1), nth<DTYPE>(k[e], 2), nth<DTYPE>(k[e], 3),
                                     ki, odd);
                w[1] = codes4<CODES>(nth<DTYPE>(k[e], 4), nth<DTYPE>(k[e], 5), nth<DTYPE>(k[e], 6), nth<DTYPE>(k[e], 7),
                                     ki, odd);
                *reinterpret_cast<u32x2 *>(kc + (t0 + e) * D + d) = w;
            }
        }
    }
    if (whole) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = (tid + i * kN) / 4, c = tid % 4;
            *reinterpret_cast<u32x4 *>(vc + row * kKvPage + c * 16) =
                *reinterpret_cast<const u32x4 *>(turn + row * kPitch + (c ^ (row / 16 % 4)) * 4);
        }
    }
    if (lo > 0 && kf != 1.0f) {
        for (int i = tid; i < lo * kPer; i += kN) {
            u32x2 *p = reinterpret_cast<u32x2 *>(kc) + i;
            u32x2 w = *p;
            w[0] = requant4<CODES>(w[0], kf);
            w[1] = requant4<CODES>(w[1], kf);
            *p = w;
        }
    }
    if (lo >= 4 && vf != 1.0f) {  // dwords of older tokens alone
        const int nq = lo / 4;
        for (int i = tid; i < nq * D; i += kN) {
            uint32_t *p = reinterpret_cast<uint32_t *>(vc + i / nq * kKvPage) + i % nq;
            *p = requant4<CODES>(*p, vf);
        }
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
        hipLaunchKernelGGL((k_kv_append<D, CODES, kBf16>), grid, dim3(2 * D), 0, s, a);
    else
        hipLaunchKernelGGL((k_kv_append<D, CODES, kFp16>), grid, dim3(2 * D), 0, s, a);
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
    const dim3 grid(kv_append_pages(a.max_new, a.c.stride), a.c.heads, a.c.batch);
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
