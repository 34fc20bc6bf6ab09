// attend_f16.hip -- the attention kernel for float16 queries and cache.
#include "attend.h"

namespace psispec {

hipError_t launch_attend_f16(const AttendKernelArgs& k, int dp, int mt, hipStream_t stream) {
  return attend::launch_typed<_Float16, false>(k, dp, mt, stream);
}

}  // namespace psispec
