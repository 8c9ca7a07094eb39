// moe_up_3.hip -- the gate and up projections of f32 layers of experts: 3 bf16 parts of
// every input.
#include "moe.h"

namespace qmm {

hipError_t launch_moe_up_3(const MoeArgs& a, const MoeWork& w) {
  return launch_moe_project<true, 3, 3>(a, w);
}

}  // namespace qmm
