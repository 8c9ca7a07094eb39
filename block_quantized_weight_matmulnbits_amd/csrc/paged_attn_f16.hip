// paged_attn_f16.hip -- the paged-attention kernels for f16 caches.
#include "paged_attn_rows.h"

namespace qmm {

hipError_t launch_rows_f16(const AttnArgs& a, const RowsPlan& plan, int blocks, int skip_above) {
  return launch_rows_type<DT_F16>(a, plan, blocks, skip_above);
}

}  // namespace qmm
