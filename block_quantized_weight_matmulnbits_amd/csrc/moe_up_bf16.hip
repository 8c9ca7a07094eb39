// moe_up_bf16.hip -- the gate and up projections of bf16 layers of experts, their inputs as they are.
#include "moe.h"

namespace qmm {

hipError_t launch_moe_up_bf16(const MoeArgs& a, const MoeWork& w) {
  return launch_moe_project<true, DT_BF16, 1, 2>(a, w);
}

}  // namespace qmm
