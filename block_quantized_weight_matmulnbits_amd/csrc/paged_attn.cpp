// paged_attn.cpp -- how paged attention is cut into workgroups, and the
// workspace that this takes.
#include "paged.h"

#ifndef V_FILL
#define V_FILL 512
#endif
#ifndef V_NO8
#define V_NO8 0
#endif
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

// Workgroups of the tiles kernel that fill the chip, one a compute unit, twice;
// its smallest part of the keys; the rows of a sequence that it takes.
constexpr int64_t TILE_FILL = V_FILL, TILE_MIN_CHUNK = 512, TILE_ROWS = 32;

// Whole rows are counted where the host knows them: the tokens of the batch.
TilePlan plan_tile(int seqs, int tokens, int max_new, int64_t keys, int group, int kv_heads, int dim,
                   int64_t* most_splits = nullptr) {
  TilePlan p;
  // Two blocks a wave halve what is read from LDS; one where registers end
  // (wide heads) or rows would be left over.
  p.blocks = V_NO8 ? 1 : dim <= 128 && (int64_t)max_new * group > 128 ? 2 : 1;
  const int64_t rows = 128 * p.blocks, whole = ceil_div((int64_t)tokens * group, rows);
  p.tiles = (int)(whole + seqs);
  // A single sequence is taken whatever it has; of several, those with few
  // rows are left to the rows kernel.
  p.skip_upto = seqs == 1 ? 0 : (int)(TILE_ROWS / group);
  int64_t parts = ceil_div(TILE_FILL, whole * kv_heads), most = keys / TILE_MIN_CHUNK;
  if (parts > most) parts = most;
  if (parts < 1 || (int64_t)p.tiles * kv_heads > COUNTERS / 2) parts = 1;
  if (most_splits) *most_splits = parts;
  p.chunk = (int)(ceil_div(ceil_div(keys < 1 ? 1 : keys, parts), 64) * 64);
  p.splits = (int)ceil_div(keys < 1 ? 1 : keys, p.chunk);
  return p;
}

int padded(int dim) { return dim <= 64 ? 64 : dim <= 96 ? 96 : dim <= 128 ? 128 : dim <= 192 ? 192 : 256; }

}  // namespace

size_t attn_workspace_bytes(int seqs, int tokens, int max_new, int max_len, int q_heads,
                            int kv_heads, int dim) {
  // The most that any call may take: every type, with a window or without.
  // With one, parts may be more than their plain count for max_len gives, but
  // never more than asked for.
  const int group = q_heads / kv_heads;
  const int64_t row_bytes = 8 + 4 * padded(dim), all = (int64_t)max_new * group;
  int64_t most = 0;
  auto rows = [&](int n) {
    for (int blocks = 1; blocks <= 2; ++blocks) {
      const int64_t parts = most_parts(seqs, n, max_len, group, kv_heads, blocks);
      const int64_t tiles = ceil_div((int64_t)n * group, 16 * blocks);
      const int64_t need = seqs * tiles * kv_heads * parts * 16 * blocks * row_bytes;
      if (parts > 1 && need > most) most = need;
    }
  };
  rows(max_new);
  if (all > TILE_ROWS) {
    int64_t parts;
    const TilePlan p = plan_tile(seqs, tokens, max_new, max_len, group, kv_heads, dim, &parts);
    const int64_t need = (int64_t)p.tiles * kv_heads * parts * 128 * p.blocks * row_bytes;
    if (parts > 1 && need > most) most = need;
    if (p.skip_upto > 0) rows(p.skip_upto);
  }
  return (size_t)(COUNTERS * 4 + (most + 255) / 256 * 256);
}

hipError_t launch_paged_attention(const AttnArgs& a) {
  const CacheArgs& c = a.c;
  const int64_t rows = (int64_t)c.max_new * a.group;
  // Few rows, 32-bit types (the tiles kernel's registers hold 16-bit queries)
  // and a scale of 0 (which it takes out of the maximum) run on the rows kernel.
  const bool tiles = a.dtype != DT_F32 && a.scale != 0.f && rows > TILE_ROWS;
  auto seen = [&](int64_t height) {
    // A tile of rows sees at most the window of its first row and its own tokens.
    int64_t keys = c.max_len;
    if (a.window > 0 && a.causal) {
      const int64_t most = (int64_t)a.window + height / a.group + 17;
      keys = keys < most ? keys : most;
    }
    return keys;
  };
  if (tiles) {
    const int height = c.dim <= 128 && rows > 128 ? 256 : 128;
    const TilePlan t = plan_tile(c.seqs, c.tokens, c.max_new, seen(height), a.group, c.kv_heads, c.dim);
    const hipError_t e = a.dtype == DT_F16 ? launch_tile_f16(a, t) : launch_tile_bf16(a, t);
    if (e != hipSuccess || t.skip_upto == 0) return e;
    // With one sequence there is none of the other kind, unless max_new is
    // only a bound.
    const int few = t.skip_upto < c.max_new ? t.skip_upto : c.max_new;
    const int blocks = few * a.group <= 16 ? 1 : 2;
    const RowsPlan p = plan_rows(c.seqs, few, seen(32), a.group, c.kv_heads, blocks);
    return a.dtype == DT_F16 ? launch_rows_f16(a, p, blocks, few) : launch_rows_bf16(a, p, blocks, few);
  }
  const int blocks = rows <= 16 ? 1 : 2;
  const RowsPlan p = plan_rows(c.seqs, c.max_new, seen(32), a.group, c.kv_heads, blocks);
  switch (a.dtype) {
    case DT_F32: return launch_rows_f32(a, p, blocks, INT32_MAX);
    case DT_F16: return launch_rows_f16(a, p, blocks, INT32_MAX);
    default: return launch_rows_bf16(a, p, blocks, INT32_MAX);
  }
}

}  // namespace qmm
