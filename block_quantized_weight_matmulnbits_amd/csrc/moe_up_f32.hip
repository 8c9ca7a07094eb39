// moe_up_f32.hip -- the gate and up projections of f32 layers of experts, inputs in three bf16 parts.
#include "moe.h"

namespace qmm {

hipError_t launch_moe_up_f32(const MoeArgs& a, const MoeWork& w) {
  return launch_moe_project<true, DT_BF16, 3, 3>(a, w);
}

}  // namespace qmm
