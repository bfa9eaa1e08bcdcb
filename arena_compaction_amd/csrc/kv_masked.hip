// kv_masked.hip -- attention over the 8-bit cache under a mask (the kernels are
// in kv_few.h, kv_prompt.h and kv_weigh.h).
#include "kv_few.h"
#include "kv_prompt.h"
#include "kv_weigh.h"

namespace ac {

template hipError_t launch_kv_few<kMasked>(const KvAttend &a, int codes, int dtype, hipStream_t s);
template hipError_t launch_kv_prompt<kMasked>(const KvAttend &a, int codes, int dtype, hipStream_t s);
template hipError_t launch_kv_weigh<kMasked>(const KvAttend &a, int codes, int dtype, hipStream_t s);

}  // namespace ac
