// moe_down_2.hip -- the down projections of 16-bit layers of experts: 2 bf16 parts of
// every input.
#include "moe.h"

namespace qmm {

hipError_t launch_moe_down_2(const MoeArgs& a, const MoeWork& w) {
  return launch_moe_project<false, 2, 2>(a, w);
}

}  // namespace qmm
