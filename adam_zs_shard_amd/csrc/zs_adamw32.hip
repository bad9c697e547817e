// zs_adamw32.hip -- the AdamW step with 32-bit moments.

#include "zs_adamw_step.h"

namespace zs {

hipError_t launch_adamw32(const AwLaunch& L) {
  launch_step<32, false>(L);
  return hipGetLastError();
}

}  // namespace zs
