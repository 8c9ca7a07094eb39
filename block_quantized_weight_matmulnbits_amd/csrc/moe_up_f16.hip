// moe_up_f16.hip -- the gate and up projections of f16 layers of experts, their inputs as they are.
#include "moe.h"

namespace qmm {

hipError_t launch_moe_up_f16(const MoeArgs& a, const MoeWork& w) {
  return launch_moe_project<true, DT_F16, 1, 2>(a, w);
}

}  // namespace qmm
