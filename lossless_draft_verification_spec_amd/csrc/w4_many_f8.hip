// w4_many_f8.hip -- the 4-bit products of many rows for rows of 8 bits.
#include "w4_many.h"

namespace psispec {

hipError_t launch_w4_many_f8(const W4Args& a, int mats, hipStream_t stream) {
  return mats == 2 ? w4::launch_many<w4::F8, 0, 2>(a, stream) : w4::launch_many<w4::F8, 0, 1>(a, stream);
}

}  // namespace psispec
