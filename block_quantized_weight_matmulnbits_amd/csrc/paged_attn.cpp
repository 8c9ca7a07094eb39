// paged_attn.cpp -- how paged attention is cut into workgroups, and the
// workspace that this takes.
#include "paged.h"

#include <algorithm>

namespace qmm {

namespace {

constexpr int DT_F32 = 0, DT_F16 = 1;

// Rows kernel.  Parts of a few hundred keys keep sequences of uneven lengths
// from leaving the chip half empty (64 sequences of 17 to 8191 keys: 288 us in
// parts of 2048, 235 of 1024, 229 of 512; two of 131071 and 90001: 199 of 1024,
// 205 of 512), so none is longer than ROWS_MAX_CHUNK; few rows are spread over
// more, shorter ones until the chip is filled, down to a block of 32 for each of
// the four waves.  Filled it is by three workgroups a compute unit, two times
// and a half over (as many tiles of rows are not split), or by one where a
// lane's registers leave room for no more.
constexpr int64_t ROWS_FILL = 2048, ROWS_FILL_WIDE = 256, ROWS_MIN_CHUNK = 128, ROWS_MAX_CHUNK = 1024,
                  ROWS_LONG_CHUNK = 4096;
// Tiles kernel: workgroups of 128 rows are resident twice on a compute unit
// (once for heads over 128), those of 256 once.  The kernel cuts long
// sequences into parts by the lengths that it finds (the price is in
// paged_attn_tile.h), where sequences may be uneven; the host only bounds them.
// Three chunks of 509 tokens over 5777 to 9001 keys take 248 us whole, 217 so;
// two of 700 over 10227 and 16000 391 and 330.  Even ones pay for the join that
// finds nothing (three of 512 over 4096 keys: 118 whole, 122), so that short
// ones, where less can be gained, are left whole (TILE_UNEVEN).
// Sequences with up to TILE_ROWS rows are left to the rows kernel.
constexpr int64_t UNITS = 256, TILE_UNEVEN = 2048, TILE_ROWS = 32;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int padded(int dim) {
  return dim <= 64 ? 64 : dim <= 96 ? 96 : dim <= 128 ? 128 : dim <= 192 ? 192 : 256;
}

// Cuts `keys` (a bound of what any row tile sees) into parts of a multiple of
// `step` keys; at most `parts`.
void cut(int64_t keys, int64_t parts, int64_t step, int* chunk, int* splits) {
  keys = std::max<int64_t>(keys, 1);
  parts = std::max<int64_t>(parts, 1);
  *chunk = (int)(ceil_div(ceil_div(keys, parts), step) * step);
  *splits = (int)ceil_div(keys, *chunk);
}

int64_t rows_parts(int seqs, int max_new, int64_t keys, int group, int kv_heads, int blocks,
                   bool wide) {
  const int64_t tiles = seqs * kv_heads * ceil_div((int64_t)max_new * group, 16 * blocks);
  // Wide rows leave a compute unit one workgroup at a time: with many of them
  // their beginnings and ends count (3 sequences of 300 f32 tokens over 900 to
  // 2000 keys: 474 us in parts of 1024, 323 of ROWS_LONG_CHUNK; 6 of 150 over
  // 300 to 5000: 867 and 946).
  if (wide && tiles >= 2 * ROWS_FILL_WIDE) return ceil_div(keys, ROWS_LONG_CHUNK);
  if (tiles >= ROWS_FILL) return 1;
  const int64_t fill = ceil_div(wide ? ROWS_FILL_WIDE : ROWS_FILL, std::max<int64_t>(tiles, 1));
  return std::max(ceil_div(keys, ROWS_MAX_CHUNK),
                  std::max<int64_t>(1, std::min(fill, ceil_div(keys, ROWS_MIN_CHUNK))));
}

int64_t resident(int blocks, int dim) { return UNITS * (blocks == 2 || dim > 128 ? 1 : 2); }

// Rows are counted over the whole batch where the host knows them: tokens.
// Two blocks of 128 rows a workgroup halve what is read from L2; one where
// registers end (wide heads) or rows would be left over.
TilePlan plan_tile(int seqs, int tokens, int max_new, int group, int dim) {
  TilePlan p{};
  p.blocks = dim <= 128 && (int64_t)max_new * group > 128 ? 2 : 1;
  p.tiles = (int)(ceil_div((int64_t)tokens * group, 128 * p.blocks) + seqs);
  // Where every sequence has as many tokens, none has fewer.
  p.skip_upto = (int64_t)seqs * max_new == tokens ? 0 : (int)(TILE_ROWS / group);
  return p;
}

// How many parts the keys of a tile may be cut into; the kernel, which knows
// the sequences' lengths, decides (to the most that is resident at once).  A
// long sequence among short ones takes more than its equal share of parts.
// bound: no fewer than for any number of keys up to `keys`.
int64_t tile_parts(int seqs, int tokens, int max_new, int64_t keys, int group, int kv_heads,
                   int blocks, int dim, bool bound = false) {
  // Tiles: of equal sequences, or else whole ones of the batch's rows.
  const int64_t height = 128 * blocks;
  const int64_t tiles = kv_heads * ((int64_t)seqs * max_new == tokens
                                        ? seqs * ceil_div((int64_t)max_new * group, height)
                                        : ceil_div((int64_t)tokens * group, height));
  const int64_t room = resident(blocks, dim);
  // Tiles of one sequence are as long as one another, and more than half of
  // what is resident gain nothing by parts; nor do short ones.
  const bool uneven = seqs > 1 && keys >= TILE_UNEVEN;
  if (tiles >= (uneven ? 2 * room : room / 2 + 1) ||
      keys < 2 * (PART_JOIN + PART_PARK * std::min(2 * tiles, room) / room))
    return 1;
  if (seqs > 1) return std::min<int64_t>(2 * room / tiles + 1, 64);
  if (bound) return std::min<int64_t>(room / tiles, 64);
  // One sequence: the same price as the kernel's, of equal parts.
  int64_t best = 1, least = keys;
  for (int64_t p = 2; p <= std::min<int64_t>(room / tiles, 64); ++p) {
    const int64_t price = ceil_div(keys, p) + PART_JOIN + PART_PARK * p * tiles / room;
    if (price < least) {
      best = p;
      least = price;
    }
  }
  return best;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// The workspace for `parts` parts of every row.
size_t parts_bytes(int64_t rows, int64_t parts, int dim) {
  return align256(rows * 4) + align256(rows * parts * 8) + (size_t)(rows * parts) * padded(dim) * 4;
}

void attn_parts(AttnArgs* a, char* ws, int64_t parts) {
  const int64_t rows = (int64_t)a->c.tokens * a->q_heads;
  a->part_count = (int32_t*)ws;
  a->part_stats = (float*)(ws + align256(rows * 4));
  a->part_out = (float*)(ws + align256(rows * 4) + align256(rows * parts * 8));
}

}  // namespace

size_t attn_workspace_bytes(int seqs, int tokens, int max_new, int max_len, int q_heads,
                            int kv_heads, int dim) {
  // The most that any call may take: every type, with a window or without (a
  // window makes parts shorter, never more than are asked for here).
  const int group = q_heads / kv_heads;
  const int64_t rows = (int64_t)tokens * q_heads;
  int64_t parts = 1;
  for (int blocks = 1; blocks <= 2; ++blocks)
    parts = std::max(parts, rows_parts(seqs, max_new, max_len, group, kv_heads, blocks, false));
  if ((int64_t)max_new * group > TILE_ROWS) {
    const TilePlan t = plan_tile(seqs, tokens, max_new, group, dim);
    parts = std::max(parts, tile_parts(seqs, tokens, max_new, max_len, group, kv_heads, t.blocks, dim, true));
    if (t.skip_upto > 0) parts = std::max(parts, ceil_div(max_len, ROWS_MAX_CHUNK));
  }
  return 256 + (parts > 1 ? align256(parts_bytes(rows, parts, dim)) : 0);
}

hipError_t launch_paged_attention(AttnArgs a, char* workspace) {
  const CacheArgs& c = a.c;
  const int64_t rows = (int64_t)c.max_new * a.group;
  // A tile of rows sees at most the window of its first row and its own tokens.
  auto seen = [&](int64_t height) {
    const int64_t most = (int64_t)a.window + height / a.group + 1;
    return a.window > 0 && a.causal ? std::min<int64_t>(c.max_len, most) : (int64_t)c.max_len;
  };
  // Few rows, 32-bit types (the tiles kernel's registers hold 16-bit queries),
  // a scale of 0 (which it takes out of the maximum) and strides past 32 bits
  // run on the rows kernel.
  const int64_t wide = std::max({c.k_page, c.v_page, c.k_token, c.v_token});
  const bool tiles = a.dtype != DT_F32 && a.scale != 0.f && wide < INT32_MAX / 2 && rows > TILE_ROWS;
  TilePlan t{};
  RowsPlan r{};
  int few = c.max_new, blocks = 1;
  if (tiles) {
    t = plan_tile(c.seqs, c.tokens, c.max_new, a.group, c.dim);
    const int64_t keys = seen(128 * t.blocks);
    t.splits = (int)tile_parts(c.seqs, c.tokens, c.max_new, keys, a.group, c.kv_heads, t.blocks,
                               c.dim);
    t.room = (int)(resident(t.blocks, c.dim) / c.kv_heads);
    if (t.splits > 1) t.tiles = std::max(t.tiles, (c.seqs > 1 && 2 * t.tiles > t.room ? 2 : 1) * t.room);
    few = t.skip_upto;
  }
  if (few > 0) {
    // 16-bit rows go 16 to a workgroup: two blocks keep a wave alone on its SIMD,
    // and what they save is read from L2 (20 sequences of 8 tokens, 4 heads a
    // group: 126 us in 32 rows, 91 in 16).  In 32 bits the matrix cores bound
    // them (300 tokens of 3 sequences each: 323 us in 32 rows, 453 in 16).
    blocks = a.dtype != DT_F32 || (int64_t)few * a.group <= 16 ? 1 : 2;
    const int64_t keys = seen(16 * blocks);
    r.row_tiles = (int)ceil_div((int64_t)few * a.group, 16 * blocks);
    // Beside tiles parts only keep the longest of them from being the last.
    int64_t parts = ceil_div(keys, ROWS_MAX_CHUNK);
    const bool wide = padded(c.dim) * (a.dtype == DT_F32 ? 4 : 2) * blocks > 768;
    if (!tiles) parts = rows_parts(c.seqs, few, keys, a.group, c.kv_heads, blocks, wide);
    cut(keys, parts, ROWS_MIN_CHUNK, &r.chunk, &r.splits);
  }
  const int splits = std::max(t.splits, r.splits);
  if (splits > 1) attn_parts(&a, workspace, splits);
  // Both kernels note how many parts each of their rows has.
  const bool join = splits > 1;
  if (tiles && few > 0 && join) {
    t.note = 1;
    r.note = 1;
  } else {
    t.note = t.splits > 1;
    r.note = r.splits > 1;
  }
  hipError_t e;
  if (tiles) {
    if (few > 0) t.few_groups = c.seqs * r.row_tiles * c.kv_heads * r.splits;
    e = a.dtype == DT_F16 ? launch_tile_f16(a, t, r) : launch_tile_bf16(a, t, r);
  } else {
    e = a.dtype == DT_F32 ? launch_rows_f32(a, r, blocks, INT32_MAX)
        : a.dtype == DT_F16 ? launch_rows_f16(a, r, blocks, INT32_MAX)
                            : launch_rows_bf16(a, r, blocks, INT32_MAX);
  }
  if (e == hipSuccess && join) e = launch_join(a, padded(c.dim), splits);
  return e;
}

}  // namespace qmm
