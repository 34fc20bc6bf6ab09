// attend_bf16.hip -- the attention kernel for bfloat16 queries and cache.
#include "attend.h"

namespace psispec {

hipError_t launch_attend_bf16(const AttendKernelArgs& k, int dp, int mt, hipStream_t stream) {
  return attend::launch_typed<__bf16, false>(k, dp, mt, stream);
}

}  // namespace psispec
