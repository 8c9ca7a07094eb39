// moe_up_2.hip -- the gate and up projections of f16 layers of experts: 2 bf16 parts of
// every input.
#include "moe.h"

namespace qmm {

hipError_t launch_moe_up_2(const MoeArgs& a, const MoeWork& w) {
  return launch_moe_project<true, 2, 2>(a, w);
}

}  // namespace qmm
