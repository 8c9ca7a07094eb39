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
  // As many tiles are not split.  In 16 bits that hardly matters where lengths
  // are spread evenly (from 17 to 8191 keys, 64 sequences over 32 key/value heads
  // 844 us whole and 834 in parts of 1024, 256 over 8 heads 846 and 861, both at
  // the copy's rate), but one of 131072 keys among 255 of 500 takes 3849 us whole
  // and 531 in parts, of a workspace of 545 MB: parts counted by the lengths on
  // the device, as the tiles kernel has them, are what is missing.  Wide ones lose
  // by parts (f32, heads of 128: 2048 tokens over 8192 keys 3.3 ms whole, 3.9 in
  // parts of 4096; four of 1024 over 2000 to 16384 8.5 and 13.3; 256 single
  // tokens, 8 heads of 256: 4.8 and 5.9).
  if (tiles >= ROWS_FILL) return 1;
  // Wide rows leave a compute unit one workgroup at a time: with many of them
  // their beginnings and ends count.  f32, in parts of 1024 and of
  // ROWS_LONG_CHUNK: 3 sequences of 300 tokens over 900 to 2000 keys 474 and 324
  // us; 4 of 500 over 600 to 3000, a head a group, 281 and 255; one of 1024 over
  // 6000 1589 and 1514; but 6 of 150 over 300 to 5000 856 and 945.
  if (wide && tiles >= 2 * ROWS_FILL_WIDE) return ceil_div(keys, ROWS_LONG_CHUNK);
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

// The workspace for `parts` parts of every row; 0 where no row has several.
size_t parts_bytes(int64_t rows, int64_t parts, int dim) {
  if (parts <= 1) return 0;
  return align256(rows * 4) + align256(rows * parts * 8) + (size_t)(rows * parts) * padded(dim) * 4;
}

void attn_parts(AttnArgs* a, char* ws, int64_t parts) {
  const int64_t rows = (int64_t)a->c.tokens * a->q_heads;
  a->part_count = (int32_t*)ws;
  a->part_stats = (float*)(ws + align256(rows * 4));
  a->part_out = (float*)(ws + align256(rows * 4) + align256(rows * parts * 8));
}

// What a call is cut by, beside the keys that its rows see.
struct Shape {
  int seqs, tokens, max_new, group, kv_heads, dim;
  bool f32, tiles;   // the queries' type; whether many rows may go to the tiles kernel
};
// Both kernels' shares of a call and the most parts that either cuts keys into.
struct Cut {
  bool tiles;
  TilePlan t{};
  int few, blocks;   // new tokens a sequence that the rows kernel takes, blocks of 16 rows
  int64_t few_keys, tile_parts, rows_parts;
  int64_t parts() const { return std::max(tile_parts, rows_parts); }
};
// The one place where parts are counted: for a launch, whose tiles of `height`
// rows see at most seen(height) keys, and (bound) for any launch of this shape
// whose tiles see no more.
template <typename Seen> Cut cut_of(const Shape& s, Seen seen, bool bound) {
  Cut p{};
  p.few = s.max_new;
  p.tile_parts = p.rows_parts = 1;
  p.tiles = s.tiles && !s.f32 && (int64_t)s.max_new * s.group > TILE_ROWS;
  if (p.tiles) {
    p.t = plan_tile(s.seqs, s.tokens, s.max_new, s.group, s.dim);
    p.tile_parts = tile_parts(s.seqs, s.tokens, s.max_new, seen(128 * p.t.blocks), s.group, s.kv_heads,
                              p.t.blocks, s.dim, bound);
    p.few = p.t.skip_upto;
  }
  if (p.few > 0) {
    // 16-bit rows go 16 to a workgroup: two blocks keep a wave alone on its SIMD,
    // and what they save is read from L2 (20 sequences of 8 tokens, 4 heads a
    // group: 126 us in 32 rows, 91 in 16).  In 32 bits the matrix cores bound
    // them (300 tokens of 3 sequences each: 323 us in 32 rows, 453 in 16).
    p.blocks = !s.f32 || (int64_t)p.few * s.group <= 16 ? 1 : 2;
    p.few_keys = seen(16 * p.blocks);
    const bool wide = padded(s.dim) * (s.f32 ? 4 : 2) * p.blocks > 768;
    // Beside tiles parts only keep the longest of them from being the last.
    p.rows_parts = p.tiles ? ceil_div(p.few_keys, ROWS_MAX_CHUNK)
                           : rows_parts(s.seqs, p.few, p.few_keys, s.group, s.kv_heads, p.blocks, wide);
  }
  return p;
}

}  // namespace

size_t attn_workspace_bytes(int seqs, int tokens, int max_new, int max_len, int q_heads,
                            int kv_heads, int dim) {
  // The most that any call may take: every type, by either kernel, with a
  // window (which leaves fewer keys to see) or without.
  int64_t parts = 1;
  for (int kind = 0; kind < 3; ++kind) {
    const Shape s{seqs, tokens, max_new, q_heads / kv_heads, kv_heads, dim, kind == 0, kind == 2};
    parts = std::max(parts, cut_of(s, [&](int64_t) { return (int64_t)max_len; }, true).parts());
  }
  return 256 + align256(parts_bytes((int64_t)tokens * q_heads, parts, dim));
}

hipError_t launch_paged_attention(AttnArgs a, char* workspace, size_t workspace_bytes) {
  const CacheArgs& c = a.c;
  // A tile of rows sees at most the window of its first row and its own tokens.
  auto seen = [&](int64_t height) {
    const int64_t most = (int64_t)a.window + height / a.group + 1;
    return a.window > 0 && a.causal ? std::min<int64_t>(c.max_len, most) : (int64_t)c.max_len;
  };
  // Few rows, 32-bit types (the tiles kernel's registers hold 16-bit queries),
  // a scale of 0 (which it takes out of the maximum) and strides past 32 bits
  // run on the rows kernel.
  const int64_t wide = std::max({c.k_page, c.v_page, c.k_token, c.v_token});
  const Cut p = cut_of(Shape{c.seqs, c.tokens, c.max_new, a.group, c.kv_heads, c.dim, a.dtype == DT_F32,
                             a.scale != 0.f && wide < INT32_MAX / 2}, seen, false);
  TilePlan t = p.t;
  RowsPlan r{};
  if (p.tiles) {
    t.splits = (int)p.tile_parts;
    t.room = (int)(resident(t.blocks, c.dim) / c.kv_heads);
    if (t.splits > 1) t.tiles = std::max(t.tiles, (c.seqs > 1 && 2 * t.tiles > t.room ? 2 : 1) * t.room);
  }
  if (p.few > 0) {
    r.row_tiles = (int)ceil_div((int64_t)p.few * a.group, 16 * p.blocks);
    cut(p.few_keys, p.rows_parts, ROWS_MIN_CHUNK, &r.chunk, &r.splits);
  }
  const int splits = std::max(t.splits, r.splits);
  // A launch has fewer than 2^32 threads: attention's, and the join's, which
  // for many rows are a group of lanes each (paged_attn_join.hip).
  const int64_t rows = (int64_t)c.tokens * a.q_heads;
  const int64_t tiles = p.tiles ? std::max<int64_t>(t.tiles, ceil_div((int64_t)c.tokens * a.group, 128 * t.blocks) + c.seqs) : 0;
  const int64_t few_groups = p.few > 0 ? (int64_t)c.seqs * r.row_tiles * c.kv_heads * r.splits : 0;
  const int64_t threads = (tiles * c.kv_heads + few_groups) * 256 * (p.tiles ? t.blocks : 1);
  const int64_t lanes = c.dim <= 64 ? 16 : c.dim <= 128 ? 32 : 64;
  if (threads > UINT32_MAX || (splits > 1 && rows * lanes + 255 > UINT32_MAX))
    return hipErrorInvalidConfiguration;
  if (parts_bytes(rows, splits, c.dim) > workspace_bytes)
    return hipErrorInvalidValue;   // not a byte is written past what was given
  if (splits > 1) attn_parts(&a, workspace, splits);
  // Both kernels note how many parts each of their rows has.
  const bool join = splits > 1;
  if (p.tiles && p.few > 0 && join) {
    t.note = 1;
    r.note = 1;
  } else {
    t.note = t.splits > 1;
    r.note = r.splits > 1;
  }
  hipError_t e;
  if (p.tiles) {
    t.few_groups = (int)few_groups;
    e = a.dtype == DT_F16 ? launch_tile_f16(a, t, r) : launch_tile_bf16(a, t, r);
  } else {
    e = a.dtype == DT_F32 ? launch_rows_f32(a, r, p.blocks, INT32_MAX)
        : a.dtype == DT_F16 ? launch_rows_f16(a, r, p.blocks, INT32_MAX)
                            : launch_rows_bf16(a, r, p.blocks, INT32_MAX);
  }
  if (e == hipSuccess && join) e = launch_join(a, padded(c.dim), splits);
  return e;
}

}  // namespace qmm
