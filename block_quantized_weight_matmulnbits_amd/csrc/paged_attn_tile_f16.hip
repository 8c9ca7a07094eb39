// paged_attn_tile_f16.hip -- paged attention of many new tokens, f16 caches.
#include "paged_attn_tile.h"

namespace qmm {

hipError_t launch_tile_f16(const AttnArgs& a, const TilePlan& plan, const RowsPlan& few) {
  return launch_tile_type<DT_F16>(a, plan, few);
}

}  // namespace qmm
