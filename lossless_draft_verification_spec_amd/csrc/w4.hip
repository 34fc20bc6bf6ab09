// w4.hip -- launches the kernel that takes a 4-bit product (w4_plan.h says which).
#include "layers.h"

namespace psispec {

size_t w4_workspace_bytes(int rows, int n, int k, int mats, int format) {
  const ManyPlan p = many_plan(rows, n, k, mats, format);
  return p.use ? p.bytes : 0;
}

hipError_t launch_w4(const W4Args& a, psispec_dtype dtype, int format, int mats, hipStream_t stream) {
  const bool many = many_plan(a.rows, a.n, a.k, mats, format).use;
  if (dtype == PSISPEC_BF16)
    return many ? launch_w4_many_bf16(a, format, mats, stream) : launch_w4_few_bf16(a, format, mats, stream);
  if (dtype == PSISPEC_F16)
    return many ? launch_w4_many_f16(a, format, mats, stream) : launch_w4_few_f16(a, format, mats, stream);
  return many ? launch_w4_many_f8(a, mats, stream) : launch_w4_few_f8(a, mats, stream);
}

}  // namespace psispec
