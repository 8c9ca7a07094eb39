// paged_attn.cpp -- how paged attention is cut into workgroups, and the
// workspace that this takes.
#include "paged.h"

namespace qmm {

namespace {

constexpr int DT_F32 = 0, DT_F16 = 1;
// Counters of the joins (paged_attn.h), and the workgroups that fill the chip:
// 256 compute units, four workgroups of the rows kernel on each, twice over.
constexpr int64_t COUNTERS = 16384, FILL = 2048;
// Keys of the smallest part: one block of 32 for each of the four waves.
constexpr int MIN_CHUNK = 128;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The split is a matter of sizes that the host knows: `keys` bounds what any
// row tile sees.  Tiles are counted in 16s of rows whatever the tile's height,
// so that the workspace holds every variant.
int64_t most_parts(int seqs, int max_new, int64_t keys, int group, int kv_heads, int blocks) {
  const int64_t rows = (int64_t)max_new * group, tiles16 = seqs * kv_heads * ceil_div(rows, 16);
  if (seqs * kv_heads * ceil_div(rows, 16 * blocks) > COUNTERS) return 1;
  const int64_t parts = ceil_div(FILL, tiles16 < 1 ? 1 : tiles16), whole = ceil_div(keys, MIN_CHUNK);
  return parts < whole ? parts : whole < 1 ? 1 : whole;
}

RowsPlan plan_rows(int seqs, int max_new, int64_t keys, int group, int kv_heads, int blocks) {
  RowsPlan p;
  p.row_tiles = (int)ceil_div((int64_t)max_new * group, 16 * blocks);
  const int64_t parts = most_parts(seqs, max_new, keys, group, kv_heads, blocks);
  const int64_t per = ceil_div(keys < 1 ? 1 : keys, parts);
  p.chunk = (int)(ceil_div(per, MIN_CHUNK) * MIN_CHUNK);
  p.splits = (int)ceil_div(keys < 1 ? 1 : keys, p.chunk);
  return p;
}

int padded(int dim) { return dim <= 64 ? 64 : dim <= 96 ? 96 : dim <= 128 ? 128 : dim <= 192 ? 192 : 256; }

}  // namespace

size_t attn_workspace_bytes(int seqs, int tokens, int max_new, int max_len, int q_heads,
                            int kv_heads, int dim) {
  const int group = q_heads / kv_heads;
  size_t most = 0;
  for (int blocks = 1; blocks <= 2; ++blocks) {
    // As many parts as there may be: a call with a window may have more of
    // them than one without, each shorter.
    const int64_t parts = most_parts(seqs, max_new, max_len, group, kv_heads, blocks);
    if (parts == 1) continue;
    const int64_t tiles = ceil_div((int64_t)max_new * group, 16 * blocks);
    const size_t rows = (size_t)seqs * tiles * kv_heads * parts * 16 * blocks;
    const size_t n = rows * (8 + 4 * (size_t)padded(dim));
    most = n > most ? n : most;
  }
  return COUNTERS * 4 + (most + 255) / 256 * 256;
}

hipError_t launch_paged_attention(const AttnArgs& a) {
  const CacheArgs& c = a.c;
  int64_t keys = c.max_len;
  const int blocks = (int64_t)c.max_new * a.group <= 16 ? 1 : 2;
  // A tile of rows sees at most the window of its first row and its own tokens.
  if (a.window > 0 && a.causal) {
    const int64_t seen = (int64_t)a.window + 32 / a.group + 1;
    keys = keys < seen ? keys : seen;
  }
  const RowsPlan p = plan_rows(c.seqs, c.max_new, keys, a.group, c.kv_heads, blocks);
  switch (a.dtype) {
    case DT_F32: return launch_rows_f32(a, p, blocks, INT32_MAX);
    case DT_F16: return launch_rows_f16(a, p, blocks, INT32_MAX);
    default: return launch_rows_bf16(a, p, blocks, INT32_MAX);
  }
}

}  // namespace qmm
