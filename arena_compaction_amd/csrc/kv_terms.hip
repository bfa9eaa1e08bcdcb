// kv_terms.hip -- attention over the 8-bit cache with a distance bias, and with a
// cap and a mask or none (the kernels are in kv_few.h, kv_prompt.h and
// kv_weigh.h); of few rows also with a cap alone, and with any cap above kLowCap.
#include "kv_few.h"
#include "kv_prompt.h"
#include "kv_weigh.h"

namespace ac {

template hipError_t launch_kv_few<kTerms>(const KvAttend &a, int codes, int dtype, hipStream_t s);
template hipError_t launch_kv_prompt<kTerms>(const KvAttend &a, int codes, int dtype, hipStream_t s);
template hipError_t launch_kv_weigh<kTerms>(const KvAttend &a, int codes, int dtype, hipStream_t s);

}  // namespace ac
