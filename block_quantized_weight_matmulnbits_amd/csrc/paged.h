// paged.h -- host-side interface between the validated entry points of the
// paged cache (paged_api.cpp) and their kernel launchers (rope.hip,
// paged_attn*.hip, pages.hip).  Not installed.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace qmm {

// Division of a 32-bit index by a number fixed per launch: a multiply-high
// and two shifts (round-up reciprocal of 33 bits, exact for every n < 2^32).
struct FastDiv {
  uint32_t d = 1, mul = 0, s1 = 0, s2 = 0;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f;
  f.d = d;
  uint32_t l = 0;
  while (l < 32 && ((uint64_t)1 << l) < d) ++l;
  f.mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << l) - d)) / d + 1);
  f.s1 = l < 1 ? l : 1;
  f.s2 = l > 1 ? l - 1 : 0;
  return f;
}
#ifdef __HIPCC__
__host__ __device__ inline uint32_t div_by(uint32_t n, const FastDiv& f) {
  const uint32_t t = (uint32_t)(((uint64_t)n * f.mul) >> 32);
  return (t + ((n - t) >> f.s1)) >> f.s2;
}
#endif

// The cache's pages and the batch (device pointers; strides in elements).
struct CacheArgs {
  char* k = nullptr;              // [pages, kv_heads, page, dim]
  char* v = nullptr;
  int64_t k_page = 0, k_head = 0, k_token = 0;
  int64_t v_page = 0, v_head = 0, v_token = 0;
  int pages = 0, kv_heads = 0, page = 0, dim = 0;
  FastDiv by_page;
  const int32_t* starts = nullptr;  // [seqs + 1]
  const int32_t* lens = nullptr;    // [seqs]
  const int32_t* table = nullptr;   // [seqs, width]
  int64_t table_stride = 0;
  int seqs = 0, tokens = 0, width = 0, max_new = 0, max_len = 0;
};

struct RopeArgs {
  CacheArgs c;
  const char *q = nullptr, *k = nullptr, *v = nullptr;  // [tokens, heads, dim]
  char* out = nullptr;
  int64_t q_token = 0, q_head = 0, k_token = 0, k_head = 0, v_token = 0, v_head = 0;
  int64_t out_token = 0, out_head = 0;
  const double* inv_freq = nullptr;  // [half]
  const int32_t* positions = nullptr;
  double factor = 1.0;
  int q_heads = 0, half = 0, interleaved = 0, dtype = 0;
  hipStream_t stream = nullptr;
};
hipError_t launch_rope_append(const RopeArgs& a);

struct AttnArgs {
  CacheArgs c;
  const char* q = nullptr;
  char* out = nullptr;
  float* lse = nullptr;              // [tokens, q_heads] or null
  int64_t q_token = 0, q_head = 0, out_token = 0, out_head = 0, lse_token = 0, lse_head = 0;
  float scale = 1.f, softcap = 0.f;
  int q_heads = 0, group = 0, causal = 1, window = 0, dtype = 0;
  int q_wide = 0, out_wide = 0;      // 16-byte rows of q; four elements at once of out
  FastDiv by_group;
  // Parts of the keys, where there is more than one (attn_parts in
  // paged_attn.cpp): by row (token x head), the number of its parts; by part
  // and row, maximum (log2), sum, and the output before its division.
  int32_t* part_count = nullptr;
  float* part_stats = nullptr;       // [splits, rows, 2]
  float* part_out = nullptr;         // [splits, rows, padded dim]
  hipStream_t stream = nullptr;
};
size_t attn_workspace_bytes(int seqs, int tokens, int max_new, int max_len, int q_heads,
                            int kv_heads, int dim);
// Errors, with nothing enqueued: hipErrorInvalidValue where the parts would pass
// workspace_bytes, hipErrorInvalidConfiguration where a launch would be too large.
hipError_t launch_paged_attention(AttnArgs a, char* workspace, size_t workspace_bytes);
// Joins the parts of every row that has several (paged_attn_join.hip).
hipError_t launch_join(const AttnArgs& a, int padded_dim, int splits);

// A few rows of queries a workgroup (paged_attn_rows.h): keys are split over
// `splits` workgroups in runs of `chunk`, rows over `row_tiles`.
struct RowsPlan {
  int splits, chunk, row_tiles, note;   // note: leave each row's number of parts
};
// One instance file a type; blocks of 16 rows a tile, 1 or 2.  Sequences with
// more than skip_above new tokens are left to another kernel.
hipError_t launch_rows_f32(const AttnArgs& a, const RowsPlan& plan, int blocks, int skip_above);
hipError_t launch_rows_f16(const AttnArgs& a, const RowsPlan& plan, int blocks, int skip_above);
hipError_t launch_rows_bf16(const AttnArgs& a, const RowsPlan& plan, int blocks, int skip_above);

// What a workgroup of the tiles kernel takes beside its keys, in keys (of 30
// ns): to begin and end; to have its part joined; to park it, where every
// resident workgroup does.
constexpr int PART_OWN = 500, PART_JOIN = 200, PART_PARK = 300;

// Many rows of queries a workgroup (paged_attn_tile.h), 16-bit types: 128 or
// 256 rows (blocks 1 or 2), at most `tiles` tiles over all sequences with
// more than skip_upto new tokens.
struct TilePlan {
  int splits;   // parts of a tile's keys: no more than these; the kernel counts them
  int room;     // workgroups a key/value head that are resident at once
  int tiles, blocks, skip_upto, note;
  int few_groups;   // workgroups after them that take the other sequences (`few`)
};
hipError_t launch_tile_f16(const AttnArgs& a, const TilePlan& plan, const RowsPlan& few);
hipError_t launch_tile_bf16(const AttnArgs& a, const TilePlan& plan, const RowsPlan& few);

// The bookkeeping of the pages (strides and sizes of `data` in bytes).
struct PoolArgs {
  char* data = nullptr;             // [planes, pages, page_bytes]
  int64_t planes = 0, plane_stride = 0, page_stride = 0, page_bytes = 0;
  int32_t *refs = nullptr, *table = nullptr, *lens = nullptr;
  int64_t table_stride = 0;
  int pages = 0, slots = 0, width = 0, page = 0;
  FastDiv by_page;
  char* workspace = nullptr;
  hipStream_t stream = nullptr;
};
// Slots that one list may name (a bit each in LDS, to find repeated ones).
constexpr int64_t POOL_MAX_SLOTS = 1 << 18;
size_t pages_workspace_bytes(int64_t pages, int64_t count);
hipError_t launch_pages_free(const PoolArgs& p, const int32_t* seqs, int count);
hipError_t launch_pages_fork(const PoolArgs& p, const int32_t* parents, const int32_t* children,
                             int count, int32_t* status);
hipError_t launch_pages_reserve(const PoolArgs& p, const int32_t* seqs, const int32_t* grow,
                                int count, int32_t* status);
hipError_t launch_pages_copy(const PoolArgs& p, const int32_t* src, const int32_t* dst, int count);
hipError_t launch_pages_compact(const PoolArgs& p, int32_t* refs_out, int32_t* table_out,
                                int64_t table_out_stride, int32_t* live);

}  // namespace qmm
