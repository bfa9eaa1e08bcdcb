// kv_rotary.hip -- new tokens into the pages of the 8-bit cache, their keys
// rotated by their positions on the way (kv_turn.h), and their queries beside
// them: the kernel is kv_store.h's, whose grid has workgroups for the queries
// behind those of the heads.
//
// Prompts of 13,000 tokens, 8 heads of 128 and 32 query heads (295 MB) take 79
// us, 3.7 TB/s where a copy reaches 4.75: the vector pipe, which makes sines and
// cosines and turns the keys in 64 bits, is busy for 47% of the cycles, and few
// waves (2.2 a SIMD) hide part of it.  One token of 128 sequences takes 10.6 us, of
// which 8.5 are what appending takes (five dependent trips to memory); a
// workgroup a head, of which one lane in 16 has a token, took 14.
#include "kv_store.h"

namespace ac {
namespace {

template <int D, int CODES>
void rotary_go(const KvRotary &a, int dtype, dim3 grid, hipStream_t s) {
    if (dtype == kBf16)
        hipLaunchKernelGGL((k_kv_append<D, CODES, kBf16, true>), grid, dim3(a.lanes), 0, s, a);
    else
        hipLaunchKernelGGL((k_kv_append<D, CODES, kFp16, true>), grid, dim3(a.lanes), 0, s, a);
}

template <int D>
void rotary_codes(const KvRotary &a, int codes, int dtype, dim3 grid, hipStream_t s) {
    if (codes == kE4m3)
        rotary_go<D, kE4m3>(a, dtype, grid, s);
    else
        rotary_go<D, kInt8>(a, dtype, grid, s);
}

}  // namespace

hipError_t launch_kv_append_rotary(const KvRotary &call, int codes, int dtype, hipStream_t s) {
    KvRotary a = call;
    // A wave takes up to 4 tokens (of 256 dimensions 2 quads and so 5, where
    // they begin in a quad's last place).
    a.lanes = a.max_new <= 4 ? 64 : 2 * a.c.dim;
    const dim3 grid(kv_append_pages(a.max_new, a.c.stride), a.c.heads + (a.q_heads + kRotaryHeads - 1) / kRotaryHeads, a.c.batch);
    switch (a.c.dim) {
        case 64: rotary_codes<64>(a, codes, dtype, grid, s); break;
        case 96: rotary_codes<96>(a, codes, dtype, grid, s); break;
        case 128: rotary_codes<128>(a, codes, dtype, grid, s); break;
        case 192: rotary_codes<192>(a, codes, dtype, grid, s); break;
        case 256: rotary_codes<256>(a, codes, dtype, grid, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace ac
