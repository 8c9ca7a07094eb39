// moe_down_3.hip -- the down projections of f32 layers of experts: 3 bf16 parts of
// every input.
#include "moe.h"

namespace qmm {

hipError_t launch_moe_down_3(const MoeArgs& a, const MoeWork& w) {
  return launch_moe_project<false, 3, 3>(a, w);
}

}  // namespace qmm
