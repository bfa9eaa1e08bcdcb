// kv_prompt.hip -- attention of many query rows over the 8-bit cache, without
// terms (the kernel is in kv_prompt.h).
#include "kv_prompt.h"

namespace ac {

template hipError_t launch_kv_prompt<kPlain>(const KvAttend &a, int codes, int dtype, hipStream_t s);

}  // namespace ac
