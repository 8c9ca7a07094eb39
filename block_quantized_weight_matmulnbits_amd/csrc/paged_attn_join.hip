// paged_attn_join.hip -- the join of attention's parts: where the keys of a row
// (a token's head) were split, its outputs and sums are brought to the largest
// of the parts' maxima, added in the order of the keys and divided.  A launch of
// its own costs the chip a few microseconds; counting arrivals inside the
// attention kernels instead had every workgroup write its L2 back, which took
// 1024 tiles of 256 rows 380 us more.  Bound by the reading of the parts.
#include "paged_attn.h"

namespace qmm {
namespace {

constexpr int JOIN_THREADS = 256, JOIN_MANY_THREADS = 1024;

// LANES lanes a row, four values each.  SHARED: a workgroup takes one row, its
// groups of lanes every so-many-th part; else every group takes a row.
template <int DT, int LANES, bool SHARED, int THREADS>
__global__ __launch_bounds__(THREADS) void join_kernel(AttnArgs a, int padded,
                                                            int splits) {
  using T = typename dt<DT>::T;
  constexpr int GROUPS = THREADS / LANES;
  __shared__ f32x4 part[SHARED ? GROUPS : 1][LANES];
  __shared__ float sums[SHARED ? GROUPS : 1];
  const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const int64_t rows = (int64_t)a.c.tokens * a.q_heads;
  const int64_t row = SHARED ? blockIdx.x : (int64_t)blockIdx.x * GROUPS + group;
  if (row >= rows) return;
  const float2* stats = (const float2*)a.part_stats + row;
  const int col = lane * 4;
  const bool mine = col < a.c.dim;
  const float* from = a.part_out + row * padded + col;
  constexpr int STEP = SHARED ? GROUPS : 1;
  const int k0 = SHARED ? group : 0;
  // Few rows: the first part of each group is loaded beside the number of
  // parts, not after it, and used only if there are so many.  Of many rows
  // most may have one part, and nothing to read.
  int count = SHARED ? splits : a.part_count[row];
  // A row of no sequence may hold anything here.
  if (count <= 1 || count > splits) return;
  float2 ml = make_float2(0.f, 0.f), other = ml;
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
  if (k0 < count) {
    ml = stats[k0 * rows];
    if (mine) y = *(const f32x4*)(from + k0 * rows * padded);
  }
  if (lane < count) other = stats[lane * rows];
  if constexpr (SHARED) {
    count = a.part_count[row];
    if (count <= 1 || count > splits) return;
  }
  float top = lane < count ? other.x : -INFINITY;
  for (int k = lane + LANES; k < count; k += LANES) top = fmaxf(top, stats[k * rows].x);
#pragma unroll
  for (int d = 1; d < LANES; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  const float ref = top == -INFINITY ? 0.f : top;
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
  float total = 0.f;
  if (k0 < count) {
    const float f = exp2_fast(ml.x - ref);
    total = f * ml.y;
    x = f * y;
  }
#pragma unroll 4
  for (int k = k0 + STEP; k < count; k += STEP) {
    const float2 m = stats[k * rows];
    const float f = exp2_fast(m.x - ref);
    total += f * m.y;
    if (mine) x += f * *(const f32x4*)(from + k * rows * padded);
  }
  if constexpr (SHARED) {
    part[group][lane] = x;
    if (lane == 0) sums[group] = total;
    __syncthreads();
    if (group != 0) return;
    for (int g = 1; g < GROUPS && g < count; ++g) {
      x += part[g][lane];
      total += sums[g];
    }
  }
  const int64_t tok = row / a.q_heads, h = row - tok * a.q_heads;
  if (mine) {
    const float inv = total == 0.f ? 0.f : 1.f / total;
    T* to = (T*)a.out + tok * a.out_token + h * a.out_head + col;
    T e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = dt<DT>::from_f32(x[j] * inv);
    if (a.out_wide) __builtin_memcpy(__builtin_assume_aligned(to, 4 * sizeof(T)), e, 4 * sizeof(T));
    else
#pragma unroll
      for (int j = 0; j < 4; ++j) to[j] = e[j];
  }
  if (a.lse != nullptr && lane == 0)
    a.lse[tok * a.lse_token + h * a.lse_head] =
        total == 0.f ? -INFINITY : (top + log2f(total)) * LN2;
}

template <int DT, int LANES>
hipError_t launch(const AttnArgs& a, int padded, int splits) {
  const int64_t rows = (int64_t)a.c.tokens * a.q_heads;
  // A workgroup a row that reads its parts side by side, larger for few rows,
  // which have many parts (64 rows of up to 128: 17 us in 256 threads, 10 in
  // 1024; 980 rows of 9: 4.6 in 256, 6.8 in 1024, 7.1 a group of lanes a row).
  if (rows <= 512)
    join_kernel<DT, LANES, true, JOIN_MANY_THREADS>
        <<<dim3((uint32_t)rows), JOIN_MANY_THREADS, 0, a.stream>>>(a, padded, splits);
  else if (rows <= 4096)
    join_kernel<DT, LANES, true, JOIN_THREADS>
        <<<dim3((uint32_t)rows), JOIN_THREADS, 0, a.stream>>>(a, padded, splits);
  else
    join_kernel<DT, LANES, false, JOIN_THREADS>
        <<<dim3((uint32_t)((rows + JOIN_THREADS / LANES - 1) / (JOIN_THREADS / LANES))), JOIN_THREADS,
           0, a.stream>>>(a, padded, splits);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_type(const AttnArgs& a, int padded, int splits) {
  return a.c.dim <= 64 ? launch<DT, 16>(a, padded, splits) : a.c.dim <= 128 ? launch<DT, 32>(a, padded, splits)
                                                                    : launch<DT, 64>(a, padded, splits);
}

}  // namespace

hipError_t launch_join(const AttnArgs& a, int padded_dim, int splits) {
  switch (a.dtype) {
    case DT_F32: return launch_type<DT_F32>(a, padded_dim, splits);
    case DT_F16: return launch_type<DT_F16>(a, padded_dim, splits);
    default: return launch_type<DT_BF16>(a, padded_dim, splits);
  }
}

}  // namespace qmm
