// kv_capped.hip -- attention of many query rows over the 8-bit cache with
// capped scores, and a mask or none (the kernel is in kv_prompt.h).
#include "kv_prompt.h"

namespace ac {

template hipError_t launch_kv_prompt<kCapped>(const KvAttend &a, int codes, int dtype, hipStream_t s);

}  // namespace ac
