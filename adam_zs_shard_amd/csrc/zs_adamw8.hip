// zs_adamw8.hip -- the AdamW step with 8-bit moments.

#include "zs_adamw_step.h"

namespace zs {

hipError_t launch_adamw8(const AwLaunch& L) {
  if (L.rounding == ZS_ROUND_STOCHASTIC)
    launch_step<8, true>(L);
  else
    launch_step<8, false>(L);
  return hipGetLastError();
}

}  // namespace zs
