// moe_up_1.hip -- the gate and up projections of bf16 layers of experts: 1 bf16 part of
// every input.
#include "moe.h"

namespace qmm {

hipError_t launch_moe_up_1(const MoeArgs& a, const MoeWork& w) {
  return launch_moe_project<true, 1, 2>(a, w);
}

}  // namespace qmm
