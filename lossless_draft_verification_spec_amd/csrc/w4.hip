// w4.hip -- which kernel takes a 4-bit product.
#include "layers.h"

namespace psispec {

size_t w4_workspace_bytes(int rows, int n, int k, int mats) { return 0; }

hipError_t launch_w4(const W4Args& a, psispec_dtype dtype, int format, int mats, hipStream_t stream) {
  if (dtype == PSISPEC_BF16) return launch_w4_few_bf16(a, format, mats, stream);
  if (dtype == PSISPEC_F16) return launch_w4_few_f16(a, format, mats, stream);
  return launch_w4_few_f8(a, mats, stream);
}

}  // namespace psispec
