// moe.hip -- a layer of experts on block-quantized weights for a few tokens:
// the router's choice, the gate and up projections with SiLU, the down
// projection, and the sum over a token's experts.
//
// Four launches: the sum needs all of a token's experts, the down projection all of
// h, both projections the list of pairs by expert.  The first (4 to 8 us) and the
// last (3 to 5 us) are chains of dependent loads on a few workgroups; the first
// lays x out for the matrix cores beside the choice, which would otherwise be
// done by every workgroup again.
#include <algorithm>

#include "moe.h"

namespace qmm {
namespace {

constexpr int ROUTE_THREADS = 1024, ROUTE_WAVES = ROUTE_THREADS / 64;
constexpr int MAX_PAIRS = MOE_MAX_TOKENS * MOE_MAX_TOP_K;

size_t align256(size_t n) { return (n + 255) / 256 * 256; }
int padded(int n) { return (n + 255) / 256 * 256; }

// Lays the workspace out from `base` (null: only the size).
size_t lay_out(int tokens, int hidden, int inter, int experts, int top_k, int dtype, char* base,
               MoeWork* w) {
  const size_t pairs = (size_t)tokens * top_k;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = base + at;
    at += align256(bytes);
    return p;
  };
  w->x_cols = padded(hidden);
  w->h_cols = padded(inter);
  w->max_active = (int)std::min<size_t>(experts, pairs);
  w->ids = (int*)take(4 * pairs);
  w->weights = (float*)take(4 * pairs);
  w->order = (int*)take(4 * pairs);
  w->active = (MoeActive*)take(sizeof(MoeActive) * w->max_active);
  w->x = (uint16_t*)take(2 * (size_t)moe_x_parts(dtype) * tokens * w->x_cols);
  w->h = (uint16_t*)take(2 * (size_t)moe_h_parts(dtype) * pairs * w->h_cols);
  w->out = (float*)take(4 * pairs * (size_t)hidden);
  return at;
}

__device__ __forceinline__ float load_logit(const MoeArgs& a, int64_t i) {
  float v;
  if (a.logits_dtype == DT_F32) v = ((const float*)a.logits)[i];
  else if (a.logits_dtype == DT_F16) v = (float)((const _Float16*)a.logits)[i];
  else v = __uint_as_float((uint32_t)((const uint16_t*)a.logits)[i] << 16);
  return v != v ? -INFINITY : v;
}

// Orders as the values do (-0 as 0).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  auto over = [&](uint32_t u) { v = u > v ? u : v; };
  over((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));    // quad_perm 1,0,3,2
  over((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));    // quad_perm 2,3,0,1
  over((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));   // row_half_mirror
  over((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));   // row_mirror
  over((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));   // row_bcast:15
  over((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));   // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// One wave: token t's experts and their weights in lanes 0 .. top_k - 1; at most
// 64 PER experts.
template <int PER>
__device__ void choose(const MoeArgs& a, int t, int lane, int* id, float* weight) {
  *id = -1;
  *weight = 0.f;
  if (a.logits == nullptr) {
    if (lane < a.top_k) {
      *id = a.ids[t * a.top_k + lane];
      *weight = a.weights[t * a.top_k + lane];
    }
  } else {
    float v[PER];
    uint32_t key[PER], best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 64 * i;
      const bool there = 64 * i < a.experts && e < a.experts;
      v[i] = there ? load_logit(a, t * a.logits_stride + e) : -INFINITY;
      key[i] = there ? order_key(v[i]) : 0u;    // a key of a value is above 0
      best = key[i] > best ? key[i] : best;
    }
    best = wave_max_u32(best);
    auto value = [](uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); };
    const float top = value(best);
    // Infinite logits share everything equally.
    auto part = [&](float l) { return top == INFINITY ? (l == INFINITY ? 1.f : 0.f) : expf(l - top); };
    if (top > -INFINITY) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (v[i] > -INFINITY) sum += part(v[i]);
      sum = wave_sum(sum);
      float chosen = 0.f, mine = 0.f;
      for (int j = 0; j < a.top_k; ++j) {
        // The lowest index that has the largest key, which is then taken away.
        int e = 0;
        bool found = false;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const uint64_t has = __ballot(key[i] == best);
          if (!found && has) {
            found = true;
            e = 64 * i + __builtin_ctzll(has);
          }
        }
        const float l = value(best), p = l > -INFINITY ? part(l) : 0.f;
        chosen += p;
        if (lane == j) {
          *id = e;
          mine = p;
        }
        best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          key[i] = lane + 64 * i == e ? 0u : key[i];
          best = key[i] > best ? key[i] : best;
        }
        best = wave_max_u32(best);
      }
      *weight = mine / (a.normalize ? chosen : sum);
    }
  }
  if (*id < 0 || *id >= a.experts || *weight == 0.f || lane >= a.top_k) *id = -1;
}

// Workgroup 0 routes; the others lay x out for the matrix cores.
template <int DT, int BITS>
__global__ __launch_bounds__(ROUTE_THREADS) void route_kernel(MoeArgs a, MoeWork w) {
  using T = typename dt<DT>::T;
  constexpr int PARTS = moe_x_parts(DT);
  if (blockIdx.x > 0) {
    const int chunks = w.x_cols / 8;
    const int all = a.tokens * chunks;   // at most 2^23
    for (int i = ((int)blockIdx.x - 1) * ROUTE_THREADS + (int)threadIdx.x; i < all;
         i += ((int)gridDim.x - 1) * ROUTE_THREADS) {
      const int t = i / chunks, c = i % chunks * 8;
      const T* from = (const T*)a.x + t * a.x_stride;
      T v[8];
      if (c + 8 <= a.hidden) {
        __builtin_memcpy(v, from + c, sizeof(v));   // at any address
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c + j < a.hidden ? from[c + j] : T(0);
      }
      uint16_t e[PARTS][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = code_at<moe_whole(BITS, DT)>(j);
        uint16_t part[PARTS];
        if constexpr (DT == DT_F32) split_bf16<PARTS>(v[k], part);
        else part[0] = __builtin_bit_cast(uint16_t, v[k]);
#pragma unroll
        for (int p = 0; p < PARTS; ++p) e[p][j] = part[p];
      }
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
        __builtin_memcpy(__builtin_assume_aligned(w.x + ((int64_t)p * a.tokens + t) * w.x_cols + c, 16),
                         e[p], 16);
    }
    return;
  }
  __shared__ __attribute__((aligned(16))) int ids[MAX_PAIRS];
  __shared__ int upto[ROUTE_WAVES], starts[ROUTE_THREADS];
  __shared__ __attribute__((aligned(16))) int counts[ROUTE_THREADS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int pairs = a.tokens * a.top_k;
  if (threadIdx.x < 4 && pairs + threadIdx.x < MAX_PAIRS) ids[pairs + threadIdx.x] = -1;   // four are read at once
  counts[threadIdx.x] = 0;
  for (int i = threadIdx.x; i < w.max_active; i += ROUTE_THREADS) w.active[i] = MoeActive{0, 0, 0, 0};
  for (int t = wave; t < a.tokens; t += ROUTE_WAVES) {
    int id;
    float weight;
    if (a.experts <= 64) choose<1>(a, t, lane, &id, &weight);
    else if (a.experts <= 256) choose<4>(a, t, lane, &id, &weight);
    else choose<MOE_MAX_EXPERTS / 64>(a, t, lane, &id, &weight);
    if (lane < a.top_k) {
      ids[t * a.top_k + lane] = id;
      w.ids[t * a.top_k + lane] = id;
      w.weights[t * a.top_k + lane] = weight;
    }
  }
  __syncthreads();
  // How many pairs expert e, this thread's, has.
  const int e = threadIdx.x;
  for (int p = e; p < pairs; p += ROUTE_THREADS)
    if (ids[p] >= 0) atomicAdd(&counts[ids[p]], 1);
  __syncthreads();
  const int count = counts[e];
  // Pairs before this expert's.
  int sum = count;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 63) upto[wave] = sum;
  __syncthreads();
  int start = sum - count;
  for (int v = 0; v < wave; ++v) start += upto[v];
  starts[e] = start;
  if (count > 0) {
    // The place among the active ones: after those with more.
    int place = 0;
#pragma unroll 4
    for (int o = 0; o < a.experts; o += 4) {
      const i32x4 four = *(const i32x4*)(counts + o);
#pragma unroll
      for (int i = 0; i < 4; ++i) place += four[i] > count || (four[i] == count && o + i < e);
    }
    w.active[place] = MoeActive{e, start, count, 0};
  }
  __syncthreads();
  // A pair's place: after the same expert's pairs before it.
  for (int p = threadIdx.x; p < pairs; p += ROUTE_THREADS) {
    const int id = ids[p];
    if (id < 0) continue;
    int place = starts[id];
#pragma unroll 4
    for (int q = 0; q < p; q += 4) {
      const i32x4 four = *(const i32x4*)(ids + q);
#pragma unroll
      for (int i = 0; i < 4; ++i) place += four[i] == id && q + i < p;
    }
    w.order[place] = p;
  }
}

// y: the sum of a token's pairs, in their order.
template <int DT>
__global__ __launch_bounds__(256) void combine_kernel(MoeArgs a, MoeWork w) {
  const int t = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
  if (n >= a.hidden) return;
  float sum = 0.f;
  // Eight at once; what stands there for a pair without an expert is loaded and not
  // used.
  for (int j0 = 0; j0 < a.top_k; j0 += 8) {
    float v[8];
    int id[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int pair = t * a.top_k + min(j0 + j, a.top_k - 1);
      v[j] = w.out[(int64_t)pair * a.hidden + n];
      id[j] = w.ids[pair];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += j0 + j < a.top_k && id[j] >= 0 ? v[j] : 0.f;
  }
  ((typename dt<DT>::T*)a.y)[t * a.y_stride + n] = dt<DT>::from_f32(sum);
}

template <int DT, int BITS>
hipError_t launch(const MoeArgs& a, const MoeWork& w) {
  const int64_t chunks = (int64_t)a.tokens * w.x_cols / 8;
  const uint32_t stage = (uint32_t)std::min<int64_t>((chunks + ROUTE_THREADS - 1) / ROUTE_THREADS, 256);
  route_kernel<DT, BITS><<<dim3(1 + stage), ROUTE_THREADS, 0, a.stream>>>(a, w);
  hipError_t e = hipGetLastError();
  const int64_t x_part = (int64_t)a.tokens * w.x_cols, h_part = (int64_t)a.tokens * a.top_k * w.h_cols;
  const MoeSide up{true, (a.inter + 15) / 16, moe_x_parts(DT), moe_h_parts(DT), w.x, x_part, h_part, w.x_cols};
  const MoeSide down{false, (a.hidden + 31) / 32, moe_h_parts(DT), 0, w.h, h_part, 0, w.h_cols};
  // h is bf16 in every layer.
  if (e == hipSuccess)
    e = BITS == 8 ? (DT == DT_F16 ? launch_moe_whole8_f16(a, w, up) : launch_moe_whole8_bf16(a, w, up))
        : DT == DT_F32 ? launch_moe_whole4_bf16(a, w, up)
        : DT == DT_F16 ? launch_moe_f16(a, w, up)
                       : launch_moe_bf16(a, w, up);
  if (e == hipSuccess)
    e = BITS == 8 ? launch_moe_whole8_bf16(a, w, down)
        : DT == DT_F32 ? launch_moe_whole4_bf16(a, w, down)
                       : launch_moe_bf16(a, w, down);
  if (e != hipSuccess) return e;
  combine_kernel<DT><<<dim3((a.hidden + 255) / 256, a.tokens), 256, 0, a.stream>>>(a, w);
  return hipGetLastError();
}

}  // namespace

size_t moe_workspace_bytes(int tokens, int hidden, int inter, int experts, int top_k) {
  MoeWork w;
  return lay_out(tokens, hidden, inter, experts, top_k, DT_F32, nullptr, &w);
}

hipError_t launch_moe(const MoeArgs& a, char* workspace) {
  MoeWork w;
  lay_out(a.tokens, a.hidden, a.inter, a.experts, a.top_k, a.dtype, workspace, &w);
  const bool four = a.bits == 4;
  switch (a.dtype) {
    case DT_F32: return four ? launch<DT_F32, 4>(a, w) : launch<DT_F32, 8>(a, w);
    case DT_F16: return four ? launch<DT_F16, 4>(a, w) : launch<DT_F16, 8>(a, w);
    default: return four ? launch<DT_BF16, 4>(a, w) : launch<DT_BF16, 8>(a, w);
  }
}

}  // namespace qmm
