// pages.hip -- the bookkeeping of a paged cache on the device: pages are given
// back, shared with a forked sequence, reserved for tokens to come, copied,
// and moved together at the front of the pool.
//
// A pool is `planes` arrays of `pages` pages (say the keys and the values of
// every layer), one reference count a page, and a table of slots: slot s
// holds ceil(lens[s] / page) pages, in order, then -1.  Counts and tables are
// whole numbers and new pages are the lowest free ones in list order, so a
// result does not depend on the order in which workgroups run.
//
// Tables and counts are small (kilobytes) and their steps depend on one
// another: one workgroup plans, through LDS and block-wide scans, and leaves
// the pages to copy in the workspace.  The copies are bound by HBM (each
// moved page read and written once in every plane) and run on the whole chip.
#include <hip/hip_runtime.h>

#include "../../include/qmm.h"
#include "paged.h"
#include "qmm_device.h"

namespace qmm {
namespace {

constexpr int PLAN_THREADS = 1024, PLAN_LDS = 1024;
constexpr int COPY_THREADS = 256, COPY_FLIGHT = 2;
// A compaction of at most so many pages and copying workgroups is one launch.
constexpr int NEAR_PAGES = 1024, NEAR_GRID = 4096;

// Workspace: the number of pages to copy, then the lists.
struct Plan {
  int32_t* moves;   // [1]
  int32_t* src;     // [max(count, pages)]
  int32_t* dst;
  int32_t* first;   // [count]: an entry's first new page in `fresh`
  int32_t* length;  // [count]: an entry's new length
  int32_t* fresh;   // [pages]: the pages taken
};
__host__ __device__ inline int64_t plan_round(int64_t n) { return (n + 63) / 64 * 64; }
__host__ __device__ inline Plan plan_of(char* ws, int64_t pages, int64_t count) {
  const int64_t most = plan_round(pages > count ? pages : count), n = plan_round(count);
  int32_t* w = (int32_t*)ws;
  Plan p;
  p.moves = w;
  p.src = w + 64;
  p.dst = p.src + most;
  p.first = p.dst + most;
  p.length = p.first + n;
  p.fresh = p.length + n;
  return p;
}

// Sum over the workgroup and the sum of the threads before this one.  Every
// thread calls it; `part` is LDS of one entry a wave.
__device__ __forceinline__ int block_scan(int v, int* part, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) part[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) {
    const int n = part[w];
    before += w < wave ? n : 0;
    all += n;
  }
  total = all;
  return before + x - v;
}

__device__ __forceinline__ int pages_for(int length, const PoolArgs& p) {
  return length <= 0 ? 0 : (int)div_by((uint32_t)length - 1u, p.by_page) + 1;
}

__global__ __launch_bounds__(256) void free_kernel(PoolArgs p, const int32_t* seqs) {
  const int s = seqs[blockIdx.x];
  if (s < 0 || s >= p.slots) return;
  int32_t* row = p.table + (int64_t)s * p.table_stride;
  for (int c = threadIdx.x; c < p.width; c += 256) {
    // Exchanged, so that a slot listed twice gives its pages back once.
    const int page = atomicExch(row + c, -1);
    if (page >= 0 && page < p.pages) atomicSub(p.refs + page, 1);
  }
  if (threadIdx.x == 0) p.lens[s] = 0;
}

// Pages src[i] -> dst[i] in every plane.  Work is cut into runs of two
// vectors a thread over (move, plane, vector), all in flight; a workgroup
// divides once for its run and by a launch constant from there.  A page is
// read and written once, so both pass the caches by (1 GB moved: 209 us with
// plain accesses, 197 without, 5.2 TB/s; four in flight: 208).
template <typename V>
__device__ __forceinline__ void copy_pages(const PoolArgs& p, const int32_t* src,
                                           const int32_t* dst, int64_t moves, uint32_t per_page,
                                           const FastDiv& by_vectors, const FastDiv& by_planes) {
  constexpr int RUN = COPY_FLIGHT * COPY_THREADS;
  const int64_t total = moves * p.planes * per_page;
  for (int64_t base = (int64_t)blockIdx.x * RUN; base < total; base += (int64_t)gridDim.x * RUN) {
    const int64_t pair0 = base / per_page;
    const uint32_t off0 = (uint32_t)(base - pair0 * per_page);
    V x[COPY_FLIGHT];
    V* to[COPY_FLIGHT];
#pragma unroll
    for (int u = 0; u < COPY_FLIGHT; ++u) {
      const uint32_t k = u * COPY_THREADS + threadIdx.x;
      to[u] = nullptr;
      if (base + k >= total) continue;
      const uint32_t more = div_by(off0 + k, by_vectors), off = off0 + k - more * per_page;
      const uint32_t pair = (uint32_t)(pair0 + more), m = div_by(pair, by_planes);
      const uint32_t plane = pair - m * (uint32_t)p.planes;
      const int a = src[m], b = dst[m];
      if (a < 0 || a >= p.pages || b < 0 || b >= p.pages || a == b) continue;
      char* at = p.data + plane * p.plane_stride;
      x[u] = __builtin_nontemporal_load((const V*)(at + a * p.page_stride) + off);
      to[u] = (V*)(at + b * p.page_stride) + off;
    }
#pragma unroll
    for (int u = 0; u < COPY_FLIGHT; ++u)
      if (to[u] != nullptr) __builtin_nontemporal_store(x[u], to[u]);
  }
}

// Four reference counts from `page` on (a multiple of 4), free past the pool's
// end as little as a used one.
__device__ __forceinline__ i32x4 refs_at(const PoolArgs& p, int page) {
  i32x4 r = {1, 1, 1, 1};
  if (page + 3 < p.pages && ((uintptr_t)p.refs & 15) == 0) return *(const i32x4*)(p.refs + page);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (page + k < p.pages) r[k] = p.refs[page + k];
  return r;
}

// Fork (FORK) or reserve.  Nothing is changed unless the whole list can be
// served: everything is checked and counted before the first write.
//
// Bound by latency: what depends on nothing is loaded first (the list, the
// status and the counts of the first 4096 pages), and lists of up to PLAN_LDS
// entries stay in LDS (48 forks out of 1536 pages: 11.4 us with both behind one
// another and in the workspace).
template <bool FORK>
__global__ __launch_bounds__(PLAN_THREADS) void take_kernel(PoolArgs p, const int32_t* parents,
                                                            const int32_t* seqs,
                                                            const int32_t* grow, int count,
                                                            int32_t* status, FastDiv by_width) {
  __shared__ uint32_t seen[POOL_MAX_SLOTS / 32];
  __shared__ int32_t near_first[PLAN_LDS], near_length[PLAN_LDS], near_have[PLAN_LDS],
      near_fresh[PLAN_LDS];
  __shared__ int part[PLAN_THREADS / 64];
  __shared__ int bad;
  const int tid = threadIdx.x;
  const Plan w = plan_of(p.workspace, p.pages, count);
  int32_t* first_of = count <= PLAN_LDS ? near_first : w.first;
  int32_t* length_of = count <= PLAN_LDS ? near_length : w.length;
  int32_t* have_of = count <= PLAN_LDS ? near_have : w.src;   // reserve has no copies
  const i32x4 front = refs_at(p, 4 * tid);
  const int before_status = status[0];
  int s = 0, arg = 0;
  if (tid < count) {
    s = seqs[tid];
    arg = FORK ? parents[tid] : grow[tid];
  }
  if (tid == 0) {
    *w.moves = 0;
    bad = 0;
  }
  for (int i = tid; i < (p.slots + 31) / 32; i += PLAN_THREADS) seen[i] = 0;
  __syncthreads();
  if (before_status != 0) return;   // an earlier call failed: nothing is done

  // Check the list and count the pages that each entry needs.
  int64_t needed = 0;
  for (int base = 0; base < count; base += PLAN_THREADS) {
    const int i = base + tid;
    int need = 0, code = 0, length = 0;
    if (i < count) {
      if (base > 0) {
        s = seqs[i];
        arg = FORK ? parents[i] : grow[i];
      }
      if (s < 0 || s >= p.slots || (FORK && (arg < 0 || arg >= p.slots))) {
        code = QMM_PAGES_BAD_ENTRY;
      } else {
        const int have = p.lens[s], other = FORK ? p.lens[arg] : 0;
        const uint32_t bit = 1u << (s & 31);
        if (atomicOr(&seen[s >> 5], bit) & bit) code = QMM_PAGES_BAD_ENTRY;
        if (FORK) {
          length = other;
          const int held = pages_for(length, p);
          if (have != 0 || length < 0 || held > p.width) code = QMM_PAGES_BAD_ENTRY;
          need = (int64_t)held * p.page != length;
        } else {
          const int64_t after = (int64_t)have + arg;
          length = (int)after;
          if (have < 0 || arg < 0 || after > INT32_MAX) {
            code = QMM_PAGES_BAD_ENTRY;
          } else {
            const int to = pages_for(length, p);
            if (to > p.width) code = QMM_PAGES_TOO_LONG;
            need = to - pages_for(have, p);
            have_of[i] = pages_for(have, p);
          }
        }
      }
      if (code) atomicMax(&bad, code);
    }
    if (code) need = 0;
    int sum;
    const int before = block_scan(need, part, sum);
    if (i < count) {
      length_of[i] = code ? 0 : length;
      if (needed + before <= p.pages) first_of[i] = (int)(needed + before);
    }
    needed += sum;
  }
  __syncthreads();
  const int64_t entries = FORK && !bad ? (int64_t)count * p.width : 0;
  for (int64_t e = tid; e < entries; e += PLAN_THREADS) {
    const int i = (int)div_by((uint32_t)e, by_width), c = (int)(e - (int64_t)i * p.width);
    if (c >= pages_for(length_of[i], p)) continue;
    const int page = p.table[(int64_t)parents[i] * p.table_stride + c];
    if (page < 0 || page >= p.pages) bad = QMM_PAGES_BAD_ENTRY;
  }

  // The lowest free pages, as many as are needed.
  int32_t* fresh = needed <= PLAN_LDS ? near_fresh : w.fresh;
  int found = 0;
  if (needed <= p.pages) {
    for (int base = 0; base < p.pages && found < needed; base += 4 * PLAN_THREADS) {
      const int page = base + 4 * tid;
      const i32x4 refs = base == 0 ? front : refs_at(p, page);
      int open = 0, sum;
#pragma unroll
      for (int k = 0; k < 4; ++k) open += refs[k] <= 0;
      int rank = found + block_scan(open, part, sum);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (refs[k] <= 0) {
          if (rank < needed) fresh[rank] = page + k;
          ++rank;
        }
      found += sum;
    }
  }
  __syncthreads();
  if (bad || found < needed) {
    if (tid == 0) {
      const int64_t lack = needed - found;
      status[0] = bad ? bad : QMM_PAGES_NONE_FREE;
      if (!bad) status[1] = (int)(lack > INT32_MAX ? INT32_MAX : lack);
    }
    return;
  }

  // The lengths are those that were counted above: a slot that another entry
  // fills here was empty then, and none of its row is read.
  for (int k = tid; k < (int)needed; k += PLAN_THREADS) {
    const int page = fresh[k];
    p.refs[page] = 1;
    if (!FORK) {
      // The last entry whose pages begin at or before the k-th has it.
      int lo = 0, hi = count - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (first_of[mid] <= k) lo = mid;
        else hi = mid - 1;
      }
      p.table[(int64_t)seqs[lo] * p.table_stride + have_of[lo] + k - first_of[lo]] = page;
    }
  }
  // Full pages are shared, a part-filled last one is copied into a new one.
  for (int64_t e = tid; e < entries; e += PLAN_THREADS) {
    const int i = (int)div_by((uint32_t)e, by_width), c = (int)(e - (int64_t)i * p.width);
    const int length = length_of[i], full = (int)div_by((uint32_t)length, p.by_page);
    int page = -1;
    if (c < pages_for(length, p)) {
      page = p.table[(int64_t)parents[i] * p.table_stride + c];
      if (c < full) {
        atomicAdd(p.refs + page, 1);
      } else {
        const int first = first_of[i];
        w.src[first] = page;
        page = fresh[first];
        w.dst[first] = page;
      }
    }
    p.table[(int64_t)seqs[i] * p.table_stride + c] = page;
  }
  for (int i = tid; i < count; i += PLAN_THREADS) p.lens[seqs[i]] = length_of[i];
  if (FORK && tid == 0) *w.moves = (int)needed;
}

// Compaction: the used pages at or past `live` (the number of used pages) move
// to the holes before it, the k-th to the k-th.  Fills the moves and the map of
// every page to its new place; every thread of the workgroup calls it.
struct Moves {
  int live, count;
};
__device__ __forceinline__ Moves plan_moves(const PoolArgs& p, int* part, int32_t* src, int32_t* dst,
                                            int32_t* map) {
  const int tid = threadIdx.x, stride = 4 * blockDim.x;
  const i32x4 front = refs_at(p, 4 * tid);
  int mine = 0;
  Moves m;
  for (int page = 4 * tid; page < p.pages; page += stride) {
    const i32x4 refs = page < stride ? front : refs_at(p, page);
#pragma unroll
    for (int k = 0; k < 4; ++k) mine += page + k < p.pages && refs[k] > 0;
  }
  block_scan(mine, part, m.live);
  int holes = 0;
  m.count = 0;
  for (int base = 0; base < p.pages; base += stride) {
    const int page = base + 4 * tid;
    const i32x4 refs = base == 0 ? front : refs_at(p, page);
    int mark = 0, sum;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = page + k < p.pages, used = in && refs[k] > 0;
      mark += (in && !used && page + k < m.live) + ((used && page + k >= m.live) << 16);
    }
    // At most 4096 of each, so both counts travel in one scan.
    const int before = block_scan(mark, part, sum);
    int hole = holes + (before & 0xFFFF), move = m.count + (before >> 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = page + k < p.pages, used = in && refs[k] > 0;
      if (in && !used && page + k < m.live) dst[hole++] = page + k;
      if (used && page + k >= m.live) src[move++] = page + k;
      else if (in) map[page + k] = page + k;
    }
    holes += sum & 0xFFFF;
    m.count += sum >> 16;
  }
  __syncthreads();
  for (int k = tid; k < m.count; k += blockDim.x) map[src[k]] = dst[k];
  return m;
}

__global__ __launch_bounds__(PLAN_THREADS) void compact_kernel(PoolArgs p, int32_t* live_out) {
  __shared__ int part[PLAN_THREADS / 64];
  const Plan w = plan_of(p.workspace, p.pages, 0);
  const Moves m = plan_moves(p, part, w.src, w.dst, w.fresh);
  if (threadIdx.x == 0) {
    *w.moves = m.count;
    *live_out = m.live;
  }
}

template <typename V>
__global__ __launch_bounds__(COPY_THREADS) void copy_kernel(PoolArgs p, const int32_t* src,
                                                            const int32_t* dst,
                                                            const int32_t* moves, int count,
                                                            uint32_t per_page, FastDiv by_vectors,
                                                            FastDiv by_planes) {
  copy_pages<V>(p, src, dst, moves ? *moves : count, per_page, by_vectors, by_planes);
}

// The copies of a compaction, with its counts and table written out anew.
// NEAR: a small pool, which every workgroup plans for itself, in LDS, instead of
// waiting for a launch that does (257 pages of 4 planes: 9.4 us in two launches,
// 8.3 in one; with 8 planes of 1000 pages the plans of 8192 workgroups cost more
// than the launch, 26 us against 21).
template <typename V, bool NEAR>
__global__ __launch_bounds__(COPY_THREADS) void move_kernel(PoolArgs p, int32_t* refs_out,
                                                            int32_t* table_out,
                                                            int64_t table_out_stride,
                                                            int32_t* live, uint32_t per_page,
                                                            FastDiv by_vectors, FastDiv by_planes,
                                                            FastDiv by_width) {
  __shared__ int part[COPY_THREADS / 64];
  __shared__ int32_t near_src[NEAR ? NEAR_PAGES : 1], near_dst[NEAR ? NEAR_PAGES : 1],
      near_map[NEAR ? NEAR_PAGES : 1];
  const Plan w = plan_of(p.workspace, p.pages, 0);
  const int32_t *src = NEAR ? near_src : w.src, *dst = NEAR ? near_dst : w.dst;
  const int32_t* map = NEAR ? near_map : w.fresh;
  int n, moves;
  if constexpr (NEAR) {
    const Moves m = plan_moves(p, part, near_src, near_dst, near_map);
    __syncthreads();
    n = m.live;
    moves = m.count;
    if (blockIdx.x == 0 && threadIdx.x == 0) *live = n;
  } else {
    n = *live;
    moves = *w.moves;
  }
  const int64_t threads = (int64_t)gridDim.x * COPY_THREADS;
  const int64_t id = (int64_t)blockIdx.x * COPY_THREADS + threadIdx.x;
  for (int64_t page = id; page < p.pages; page += threads) {
    const int refs = p.refs[page];
    if (refs > 0) refs_out[map[page]] = refs;
    if (page >= n) refs_out[page] = 0;
  }
  const int64_t entries = (int64_t)p.slots * p.width;
  for (int64_t e = id; e < entries; e += threads) {
    const int64_t s = div_by((uint32_t)e, by_width), c = e - s * p.width;
    const int page = p.table[s * p.table_stride + c];
    table_out[s * table_out_stride + c] = page >= 0 && page < p.pages ? map[page] : page;
  }
  copy_pages<V>(p, src, dst, moves, per_page, by_vectors, by_planes);
}

// Division by n, which may be 0 where there is nothing to divide.
FastDiv div_of(int64_t n) { return fast_div((uint32_t)(n > 0 ? n : 1)); }

// Calls f with a value of the widest vector that the pages' bytes allow.
template <typename F>
hipError_t by_vector(const PoolArgs& p, F f) {
  const uint64_t all = (uint64_t)(uintptr_t)p.data | (uint64_t)p.plane_stride |
                       (uint64_t)p.page_stride | (uint64_t)p.page_bytes;
  if (all % 16 == 0) return f(u32x4{});
  if (all % 4 == 0) return f(uint32_t{});
  return f(uint8_t{});
}

int copy_grid(const PoolArgs& p, int64_t moves, int64_t per_page) {
  const int64_t runs = (moves * p.planes * per_page + COPY_FLIGHT * COPY_THREADS - 1) / (COPY_FLIGHT * COPY_THREADS);
  return (int)(runs < 1 ? 1 : runs > 8192 ? 8192 : runs);
}

hipError_t launch_copy(const PoolArgs& p, const int32_t* src, const int32_t* dst,
                       const int32_t* moves, int count) {
  return by_vector(p, [&](auto v) {
    const int64_t per = p.page_bytes / (int64_t)sizeof(v);
    copy_kernel<decltype(v)><<<copy_grid(p, count, per), COPY_THREADS, 0, p.stream>>>(
        p, src, dst, moves, count, (uint32_t)per, div_of(per), div_of(p.planes));
    return hipGetLastError();
  });
}

}  // namespace

size_t pages_workspace_bytes(int64_t pages, int64_t count) {
  const int64_t most = plan_round(pages > count ? pages : count);
  return (size_t)(64 + 2 * most + 2 * plan_round(count) + plan_round(pages)) * 4;
}

hipError_t launch_pages_free(const PoolArgs& p, const int32_t* seqs, int count) {
  free_kernel<<<count, 256, 0, p.stream>>>(p, seqs);
  return hipGetLastError();
}

hipError_t launch_pages_fork(const PoolArgs& p, const int32_t* parents, const int32_t* children,
                             int count, int32_t* status) {
  take_kernel<true><<<1, PLAN_THREADS, 0, p.stream>>>(p, parents, children, nullptr, count, status,
                                                      fast_div((uint32_t)p.width));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.planes == 0 || p.page_bytes == 0) return e;
  const Plan w = plan_of(p.workspace, p.pages, count);
  return launch_copy(p, w.src, w.dst, w.moves, count);
}

hipError_t launch_pages_reserve(const PoolArgs& p, const int32_t* seqs, const int32_t* grow,
                                int count, int32_t* status) {
  take_kernel<false><<<1, PLAN_THREADS, 0, p.stream>>>(p, nullptr, seqs, grow, count, status,
                                                       fast_div((uint32_t)p.width));
  return hipGetLastError();
}

hipError_t launch_pages_copy(const PoolArgs& p, const int32_t* src, const int32_t* dst, int count) {
  return launch_copy(p, src, dst, nullptr, count);
}

hipError_t launch_pages_compact(const PoolArgs& p, int32_t* refs_out, int32_t* table_out,
                                int64_t table_out_stride, int32_t* live) {
  return by_vector(p, [&](auto v) {
    using V = decltype(v);
    const int64_t per = p.page_bytes / (int64_t)sizeof(v);
    const int grid = copy_grid(p, p.pages / 2 + 1, per);
    if (p.pages <= NEAR_PAGES && grid <= NEAR_GRID) {
      move_kernel<V, true><<<grid, COPY_THREADS, 0, p.stream>>>(
          p, refs_out, table_out, table_out_stride, live, (uint32_t)per, div_of(per),
          div_of(p.planes), div_of(p.width));
      return hipGetLastError();
    }
    compact_kernel<<<1, PLAN_THREADS, 0, p.stream>>>(p, live);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    move_kernel<V, false><<<grid, COPY_THREADS, 0, p.stream>>>(
        p, refs_out, table_out, table_out_stride, live, (uint32_t)per, div_of(per),
        div_of(p.planes), div_of(p.width));
    return hipGetLastError();
  });
}

}  // namespace qmm
