// attend_f16_f8.hip -- the attention kernel for float16 queries, 8-bit cache.
#include "attend.h"

namespace psispec {

hipError_t launch_attend_f16_f8(const AttendKernelArgs& k, int dp, int mt, hipStream_t stream) {
  return attend::launch_typed<_Float16, true>(k, dp, mt, stream);
}

}  // namespace psispec
