// paged_attn_bf16.hip -- the paged-attention kernels for bf16 caches.
#include "paged_attn_rows.h"

namespace qmm {

hipError_t launch_rows_bf16(const AttnArgs& a, const RowsPlan& plan, int blocks, int skip_above) {
  return launch_rows_type<DT_BF16>(a, plan, blocks, skip_above);
}

}  // namespace qmm
