// kv_append.hip -- new tokens into the pages of the 8-bit cache, as they are
// (the kernel is in kv_store.h).
#include "kv_store.h"

namespace ac {
namespace {

__global__ void k_kv_zero(unsigned long long *p) {
    if (threadIdx.x == 0 && blockIdx.x == 0) *p = 0;
}

template <int D, int CODES>
void append_go(const KvAppend &a, int dtype, dim3 grid, hipStream_t s) {
    if (dtype == kBf16)
        hipLaunchKernelGGL((k_kv_append<D, CODES, kBf16, false>), grid, dim3(2 * D), 0, s, a);
    else
        hipLaunchKernelGGL((k_kv_append<D, CODES, kFp16, false>), grid, dim3(2 * D), 0, s, a);
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
