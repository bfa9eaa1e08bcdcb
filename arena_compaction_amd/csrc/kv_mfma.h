// kv_mfma.h -- codes of the 8-bit cache as operands of matrix instructions.
//
// Scores are products of 16-bit queries with codes brought to the queries'
// own type, which is exact (e4m3 has 4 significant bits, int8 7), and
// weights x values are products in float16, whose 11 bits round a weight
// eight times finer than bfloat16 would; sums are float32 throughout.
#ifndef ARENA_COMPACTION_KV_MFMA_H
#define ARENA_COMPACTION_KV_MFMA_H
#include "kv_device.h"

namespace ac {
namespace {

// Eight codes (two dwords, ascending) as eight 16-bit numbers.
template <int CODES, int DTYPE>
__device__ inline u32x4 widen8(uint32_t lo, uint32_t hi) {
    u32x4 r;
    if constexpr (CODES == kE4m3) {
        if constexpr (DTYPE == kFp16) {
            r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
            r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
            r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
            r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
        } else {
            r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
            r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
            r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
            r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
        }
    } else if constexpr (DTYPE == kFp16) {
        // the byte u = code + 128 under the high byte 0x64 is the float16
        // 1024 + u; taking 1152 away leaves the code, exactly
        const uint32_t a = lo ^ 0x80808080u, b = hi ^ 0x80808080u;
        const half2v off = {(_Float16)1152.0f, (_Float16)1152.0f};
        const uint32_t w[4] = {__builtin_amdgcn_perm(0x64646464u, a, 0x04010400u),
                               __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u),
                               __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u),
                               __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u)};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, w[i]) - off);
    } else {
        // through float32; at most 7 bits, so its high half is the bfloat16
        const uint32_t w[2] = {lo, hi};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = w[i / 2] >> (16 * (i % 2));
            const uint32_t p = __builtin_bit_cast(uint32_t, (float)(int8_t)x);
            const uint32_t q = __builtin_bit_cast(uint32_t, (float)(int8_t)(x >> 8));
            r[i] = __builtin_amdgcn_perm(q, p, 0x07060302u);
        }
    }
    return r;
}

// c += a x b over 32 places: a is 16 x 32, b 32 x 16.  A lane holds 8 places
// of row (column) lane % 16, from 8 * (lane / 16) on; of c, column lane % 16
// and rows 4 * (lane / 16) to + 3.
template <int DTYPE>
__device__ inline f32x4 mfma16(const u32x4 &a, const u32x4 &b, const f32x4 &c) {
    if constexpr (DTYPE == kBf16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a),
                                                       __builtin_bit_cast(bf8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                      __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

// The first of the 8 dimensions that lane group g holds at step s of a
// product over D.  Two steps share 64 dimensions so that a lane's codes of
// both are 16 contiguous bytes; a last step of 32 stands alone.
template <int D>
__device__ inline constexpr int dim_of(int s, int g) {
    return s < D / 64 * 2 ? s / 2 * 64 + g * 16 + s % 2 * 8 : D / 64 * 64 + g * 8;
}

// The token of a page that row m of key tile tt stands for: chosen so that
// the four tiles' scores a lane receives (rows 4g to 4g + 3 of each) are the
// 16 consecutive tokens 16g to 16g + 15, the ones whose value codes it loads.
__device__ inline int token_of(int tt, int m) { return m / 4 * 16 + tt * 4 + m % 4; }

// Key codes of a page's strip: tile tt, two dwords a step.
template <int D>
__device__ inline void load_keys(const uint8_t *strip, int lane, uint32_t (&k)[4][D / 16]) {
    const int m = lane % 16, g = lane / 16;
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
        const uint8_t *row = strip + token_of(tt, m) * D;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const u32x4 w = *reinterpret_cast<const u32x4 *>(row + c * 64 + g * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) k[tt][4 * c + i] = w[i];
        }
        if constexpr (D % 64 != 0) {
            const u32x2 w = *reinterpret_cast<const u32x2 *>(row + D / 64 * 64 + g * 8);
            k[tt][D / 16 - 2] = w[0];
            k[tt][D / 16 - 1] = w[1];
        }
    }
}

// Eight 16-bit numbers; 2-byte alignment will do (gfx950 reads 16 bytes from
// any address, in one instruction).
__device__ inline u32x4 load_q8(const uint16_t *p) {
    u32x4 r;
    __builtin_memcpy(&r, p, 16);
    return r;
}

}  // namespace
}  // namespace ac

#endif
