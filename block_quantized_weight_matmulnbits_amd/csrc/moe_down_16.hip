// moe_down_16.hip -- the down projections of 16-bit layers of experts, inputs in two bf16 parts.
#include "moe.h"

namespace qmm {

hipError_t launch_moe_down_16(const MoeArgs& a, const MoeWork& w) {
  return launch_moe_project<false, DT_BF16, 2, 2>(a, w);
}

}  // namespace qmm
