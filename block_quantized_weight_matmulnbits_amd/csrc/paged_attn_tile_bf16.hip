// paged_attn_tile_bf16.hip -- paged attention of many new tokens, bf16 caches.
#include "paged_attn_tile.h"

namespace qmm {

hipError_t launch_tile_bf16(const AttnArgs& a, const TilePlan& plan, const RowsPlan& few) {
  return launch_tile_type<DT_BF16>(a, plan, few);
}

}  // namespace qmm
