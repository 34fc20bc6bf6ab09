// attend_bf16_f8.hip -- the attention kernel for bfloat16 queries, 8-bit cache.
#include "attend.h"

namespace psispec {

hipError_t launch_attend_bf16_f8(const AttendKernelArgs& k, int dp, int mt, hipStream_t stream) {
  return attend::launch_typed<__bf16, true>(k, dp, mt, stream);
}

}  // namespace psispec
