// kv_device.h -- number formats and page access of the 8-bit cache's kernels.
#ifndef ARENA_COMPACTION_KV_DEVICE_H
#define ARENA_COMPACTION_KV_DEVICE_H
#include "kv.h"
#include "wave.h"

namespace ac {
namespace {

constexpr int kE4m3 = 0, kInt8 = 1;
constexpr int kBf16 = 0, kFp16 = 1;

using half8 = __attribute__((__vector_size__(8 * sizeof(_Float16)))) _Float16;
using half2v = __attribute__((__vector_size__(2 * sizeof(_Float16)))) _Float16;
using bf8 = __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16;
using bf2 = __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16;
using f32x4 = __attribute__((__vector_size__(16))) float;
using f32x2 = __attribute__((__vector_size__(8))) float;
using u32x4 = __attribute__((__vector_size__(16))) uint32_t;
using u32x2 = __attribute__((__vector_size__(8))) uint32_t;

template <int DTYPE>
__device__ inline float to_float(uint16_t x) {
    if constexpr (DTYPE == kBf16) {
        return __builtin_bit_cast(float, (uint32_t)x << 16);
    } else {
        return (float)__builtin_bit_cast(_Float16, x);
    }
}

// to nearest, ties to even: half a step (bf16 2^-8, fp16 2^-11) is the only
// rounding between the 32-bit result and the output
template <int DTYPE>
__device__ inline uint32_t pack2(float a, float b) {
    const f32x2 v = {a, b};
    if constexpr (DTYPE == kBf16) {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf2));
    } else {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, half2v));
    }
}

__device__ inline float pow2(int e) {  // normal range only
    return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
}

__device__ inline int exp_of_pow2(float s) {
    return (int)((__builtin_bit_cast(uint32_t, s) >> 23) & 255u) - 127;
}

// Least e with amax <= largest code * 2^e (448 = 1.75 * 2^8, 127 =
// 1.984375 * 2^6), at least kKvExpMin; amax is finite and not negative.
template <int CODES>
__device__ inline int scale_exp(float amax) {
    const uint32_t b = __builtin_bit_cast(uint32_t, amax);
    const int k = CODES == kE4m3 ? 8 : 6;
    const uint32_t top = CODES == kE4m3 ? 0x600000u : 0x7E0000u;
    const int e = (int)(b >> 23) - 127 - k + ((b & 0x7FFFFFu) > top ? 1 : 0);
    return e < kKvExpMin ? kKvExpMin : e;
}

// A code's value.
template <int CODES, int BYTE>
__device__ inline float code_value(uint32_t w) {
    if constexpr (CODES == kE4m3) {
        return __builtin_amdgcn_cvt_f32_fp8((int)w, BYTE);
    } else {
        return (float)(int8_t)(w >> (8 * BYTE));
    }
}

// Four values in units of their scale to the nearest codes (ties to even),
// what lies outside to the largest code.  A NaN stays one in e4m3 and is 0
// in int8.
template <int CODES>
__device__ inline uint32_t to_codes4(float a, float b, float c, float d) {
    if constexpr (CODES == kE4m3) {
        auto lim = [](float x) {
            const float y = __builtin_amdgcn_fmed3f(x, -448.0f, 448.0f);
            return x != x ? x : y;
        };
        int r = __builtin_amdgcn_cvt_pk_fp8_f32(lim(a), lim(b), 0, false);
        r = __builtin_amdgcn_cvt_pk_fp8_f32(lim(c), lim(d), r, true);
        return (uint32_t)r;
    } else {
        auto q = [](float x) {
            const float y = __builtin_rintf(__builtin_amdgcn_fmed3f(x, -127.0f, 127.0f));
            return (uint32_t)(x != x ? 0 : (int)y) & 255u;
        };
        return q(a) | (q(b) << 8) | (q(c) << 16) | (q(d) << 24);
    }
}

// Four codes times 2^shift, as codes again.
template <int CODES>
__device__ inline uint32_t requant4(uint32_t w, float f) {
    return to_codes4<CODES>(code_value<CODES, 0>(w) * f, code_value<CODES, 1>(w) * f,
                            code_value<CODES, 2>(w) * f, code_value<CODES, 3>(w) * f);
}

// Number of a workgroup of grid_of's grids.
__device__ inline uint32_t block_number() { return blockIdx.y * gridDim.x + blockIdx.x; }

constexpr uint64_t kNoPage = ~0ull;

// A page's offset, or kNoPage where the table's entry is none: outside the
// arena, or not on the arena's 32-byte grid.
__device__ inline uint64_t page_offset(const KvCache &c, uint32_t b, uint64_t j) {
    const int64_t off = c.pages[(uint64_t)b * c.stride + j];
    const uint64_t need = kv_page_bytes(c.heads, c.dim);
    const bool bad = off < 0 || (off & 31) || need > c.arena_bytes || (uint64_t)off > c.arena_bytes - need;
    return bad ? kNoPage : (uint64_t)off;
}

__device__ inline uint8_t *page_at(const KvCache &c, uint32_t b, uint64_t j) {
    const uint64_t off = page_offset(c, b, j);
    return off == kNoPage ? nullptr : c.arena + off;
}

// What lane i (the same i in every lane) holds, in scalar registers.
__device__ inline uint64_t lane_u64(uint64_t x, int i) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, i) |
           (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), i) << 32;
}
// Waits here for a loaded value (and not at its first use, inside a loop that
// has younger loads under way).
template <typename T>
__device__ inline void arrived(T x) {
    asm volatile("" ::"v"(x));
}
__device__ inline float lane_f32(float x, int i) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), i));
}

__device__ inline float *page_scales(const KvCache &c, uint8_t *page, uint32_t h) {
    return reinterpret_cast<float *>(page + (uint64_t)c.heads * 2 * kKvPage * c.dim) + 2 * h;
}

// First token and number of new tokens of sequence b; none where `starts`
// does not ascend inside [0, tokens] or brings more than max_new.
__device__ inline void new_tokens(const int32_t *starts, uint64_t tokens, uint32_t max_new,
                                  uint32_t b, uint64_t *first, int *count, bool *bad) {
    if (!starts) {
        *first = b;
        *count = 1;
        *bad = false;
        return;
    }
    const int64_t s = starts[b], e = starts[b + 1];
    *bad = s < 0 || e < s || (uint64_t)e > tokens || e - s > (int64_t)max_new;
    *first = *bad ? 0 : (uint64_t)s;
    *count = *bad ? 0 : (int)(e - s);
}

// The top bit of each of four e4m3 codes that is a NaN (0x7F or 0xFF).
__device__ inline uint32_t nan_codes(uint32_t w) {
    return ~(((w & 0x7F7F7F7Fu) ^ 0x7F7F7F7Fu) + 0x7F7F7F7Fu) & 0x80808080u;
}

// op over the four lanes that share lane % 16, in each of them.  The swaps
// exchange rows of 16 (halves of 32) lanes of two registers: of a value with
// itself, the results are the one row (half) and the other, in both.
template <typename Op>
__device__ inline float across_groups(float x, Op op) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t p0 = p[0], p1 = p[1];
    const float y = op(__builtin_bit_cast(float, p0), __builtin_bit_cast(float, p1));
    const uint32_t v = __builtin_bit_cast(uint32_t, y);
    const auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    const uint32_t q0 = q[0], q1 = q[1];
    return op(__builtin_bit_cast(float, q0), __builtin_bit_cast(float, q1));
}

// The largest magnitudes among codes, byte by byte: magnitudes ascend with
// their codes' bits, so whole bytes are compared, two to a 16-bit lane, and
// scaled once at the end.  A NaN counts as 0.
struct ByteMax {
    uint32_t even = 0, odd = 0;  // bytes 0 and 2, bytes 1 and 3
};
__device__ inline uint32_t max_u16x2(uint32_t a, uint32_t b) {
    using u16x2 = __attribute__((__vector_size__(4))) uint16_t;
    const u16x2 x = __builtin_bit_cast(u16x2, a), y = __builtin_bit_cast(u16x2, b);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(x, y));
}
template <int CODES>
__device__ inline void byte_max(ByteMax &m, uint32_t w) {
    uint32_t mag;
    if constexpr (CODES == kE4m3) {
        mag = w & 0x7F7F7F7Fu & ~((nan_codes(w) >> 7) * 255u);
    } else {
        const uint32_t neg = (w >> 7) & 0x01010101u;
        mag = (w ^ (neg * 255u)) + neg;  // -128 is no code of append's, but stays 128
    }
    m.even = max_u16x2(m.even, mag & 0x00FF00FFu);
    m.odd = max_u16x2(m.odd, (mag >> 8) & 0x00FF00FFu);
}
template <int CODES>
__device__ inline float magnitude(uint32_t byte) {
    if constexpr (CODES == kE4m3)
        return code_value<kE4m3, 0>(byte);
    else
        return (float)byte;
}

// Largest of the wave's values (each at least 0), in every lane.
__device__ inline float wave_max0(float x) {
    return wave_reduce(x, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace
}  // namespace ac

#endif
