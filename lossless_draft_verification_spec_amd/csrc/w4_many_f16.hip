// w4_many_f16.hip -- the 4-bit products of many rows for F16 rows.
#include "w4_many.h"

namespace psispec {

template <int MATS>
static hipError_t go(const W4Args& a, int format, hipStream_t stream) {
  if (format == PSISPEC_W4_MX) return w4::launch_many<_Float16, 0, MATS>(a, stream);
  if (a.gpt == 1) return w4::launch_many<_Float16, 1, MATS>(a, stream);
  if (a.gpt == 2) return w4::launch_many<_Float16, 2, MATS>(a, stream);
  return w4::launch_many<_Float16, 4, MATS>(a, stream);
}
hipError_t launch_w4_many_f16(const W4Args& a, int format, int mats, hipStream_t stream) {
  return mats == 2 ? go<2>(a, format, stream) : go<1>(a, format, stream);
}

}  // namespace psispec
