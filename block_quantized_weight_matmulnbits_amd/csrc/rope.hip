// rope.hip -- rotary positions of the query and key heads, fused with the
// append of keys and values to a paged cache.
//
// Token t of sequence s is its key number lens[s] - starts[s + 1] + t.  A
// pair (a, b) of a query or key head at position p turns by the angle
// p * inv_freq[i]:  (a cos - b sin, b cos + a sin), times `factor`.  The
// angle of a far position needs 64 bits (2^20 radians in 32 bits are off by
// 2^-4), so it is formed and reduced to [-pi/4, pi/4] in 64 bits, as are sine
// and cosine; both are rounded to 32 bits once and the heads are turned in 32.
//
// Bound by HBM: every head is read once and written once.  A token's angles
// are the same for all its heads, so a workgroup takes whole tokens, computes
// each angle once into LDS and turns every head from there.
#include <hip/hip_runtime.h>

#include "paged.h"
#include "qmm_device.h"

namespace qmm {
namespace {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_MAX_HALF = 256;

template <int BYTES> struct Chunk;
template <> struct Chunk<16> { using V = u32x4; };
template <> struct Chunk<8> { using V = u32x2; };
template <> struct Chunk<4> { using V = uint32_t; };
template <> struct Chunk<2> { using V = uint16_t; };

// Sine and cosine of x radians.  Cody and Waite's reduction: x minus the
// nearest multiple n of pi/2, held as two doubles whose products with n are
// formed by fused multiply-adds; then the Taylor series, whose first omitted
// terms are below 4e-13 on [-pi/4, pi/4].
__device__ __forceinline__ void sincos64(double x, double& s, double& c) {
  constexpr double PIO2_HI = 1.57079632679489655800e+00, PIO2_LO = 6.12323399573676603587e-17;
  const double n = __builtin_rint(x * 0.63661977236758134308);
  const double r = __builtin_fma(-n, PIO2_LO, __builtin_fma(-n, PIO2_HI, x));
  const double z = r * r;
  double ps = 1.0 / 6227020800.0, pc = 1.0 / 479001600.0;
  ps = __builtin_fma(ps, z, -1.0 / 39916800.0);
  pc = __builtin_fma(pc, z, -1.0 / 3628800.0);
  ps = __builtin_fma(ps, z, 1.0 / 362880.0);
  pc = __builtin_fma(pc, z, 1.0 / 40320.0);
  ps = __builtin_fma(ps, z, -1.0 / 5040.0);
  pc = __builtin_fma(pc, z, -1.0 / 720.0);
  ps = __builtin_fma(ps, z, 1.0 / 120.0);
  pc = __builtin_fma(pc, z, 1.0 / 24.0);
  ps = __builtin_fma(ps, z, -1.0 / 6.0);
  pc = __builtin_fma(pc, z, -0.5);
  const double sr = __builtin_fma(ps * z, r, r), cr = __builtin_fma(pc, z, 1.0);
  const int64_t quad = (int64_t)n;
  const double a = (quad & 1) ? cr : sr, b = (quad & 1) ? sr : cr;
  s = (quad & 2) ? -a : a;
  c = ((quad + 1) & 2) ? -b : b;
}

// Where one token goes.  page < 0: not appended (it has no valid slot).
struct Place {
  int page, at;
};

// TB tokens a workgroup; VEC elements a load.  An item is 2 VEC elements of
// one head: VEC pairs, or 2 VEC elements that are only copied.
template <int DT, int VEC, bool INTER, int TB>
__global__ __launch_bounds__(ROPE_THREADS) void rope_append_kernel(
    RopeArgs a, int items, FastDiv by_items, FastDiv by_head, int turning) {
  using T = typename dt<DT>::T;
  using V = typename Chunk<VEC * (int)sizeof(T)>::V;
  __shared__ float2 turn[TB][ROPE_MAX_HALF];
  __shared__ Place place[TB];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t0 = blockIdx.x * TB;
  const CacheArgs& c = a.c;

  // Each wave finds its token's sequence (the number of sequences that end at
  // or before it: their ends do not decrease) and, with the other waves of
  // the same token, its angles.
  // Thousands of tokens pass the caches by (16384 of 48 heads of 128: 86 us with
  // plain accesses, 82 without, 4.9 TB/s, what a large copy reaches here); a
  // few are about to be read again.
  constexpr bool STREAM = TB >= 4;
  constexpr int SHARE = TB >= 4 ? 1 : 4 / TB;   // waves of one token
  const int mine = wave / SHARE, t = t0 + mine;
  if (t < c.tokens) {
    int seq = 0;
    for (int base = 0; base < c.seqs; base += 64) {
      const int i = base + lane;
      const bool before = i < c.seqs && c.starts[i + 1] <= t;
      seq += __builtin_popcountll(__ballot(before));
    }
    int slot = -1, pos = 0;
    if (seq < c.seqs && t >= c.starts[seq]) {
      slot = c.lens[seq] - c.starts[seq + 1] + t;
      pos = slot;
    }
    if (a.positions != nullptr) pos = a.positions[t];
    if (lane == 0 && wave % SHARE == 0) {
      Place p{-1, 0};
      if (slot >= 0) {
        const int col = (int)div_by((uint32_t)slot, c.by_page);
        if (col < c.width) {
          p.page = c.table[(int64_t)seq * c.table_stride + col];
          p.at = slot - col * c.page;
          if (p.page >= c.pages) p.page = -1;
        }
      }
      place[mine] = p;
    }
    for (int i = (wave % SHARE) * 64 + lane; i < a.half; i += 64 * SHARE) {
      double s, co;
      sincos64((double)pos * a.inv_freq[i], s, co);
      turn[mine][i] = make_float2((float)(co * a.factor), (float)(s * a.factor));
    }
  }
  __syncthreads();

  const int left = c.tokens - t0, total = (left < TB ? left : TB) * items;
  const int step = ROPE_THREADS * gridDim.y;
  constexpr int U = TB >= 4 ? 4 : 1;   // items in flight per thread
  for (int first = blockIdx.y * ROPE_THREADS + tid; first < total; first += step * U) {
    V x[U][2];
    T* to[U];
    int at[U];   // first pair's angle, or -1: copied
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int idx = first + u * step;
      to[u] = nullptr;
      at[u] = -1;
      if (idx >= total) continue;
      const int tb = (int)div_by((uint32_t)idx, by_items), item = idx - tb * items;
      const int head = (int)div_by((uint32_t)item, by_head), n = item - head * (int)by_head.d;
      const int64_t tok = t0 + tb;
      const Place p = place[tb];
      const T* from;
      if (head < a.q_heads) {
        from = (const T*)a.q + tok * a.q_token + head * a.q_head;
        to[u] = (T*)a.out + tok * a.out_token + head * a.out_head;
      } else if (head < a.q_heads + c.kv_heads) {
        const int h = head - a.q_heads;
        from = (const T*)a.k + tok * a.k_token + h * a.k_head;
        to[u] = (T*)c.k + p.page * c.k_page + h * c.k_head + p.at * c.k_token;
      } else {
        const int h = head - a.q_heads - c.kv_heads;
        from = (const T*)a.v + tok * a.v_token + h * a.v_head;
        to[u] = (T*)c.v + p.page * c.v_page + h * c.v_head + p.at * c.v_token;
      }
      if (head >= a.q_heads && p.page < 0) { to[u] = nullptr; continue; }
      int64_t o0, o1;
      if (head < a.q_heads + c.kv_heads && n < turning) {
        at[u] = n * VEC;
        o0 = INTER ? n * 2 * VEC : n * VEC;
        o1 = INTER ? o0 + VEC : o0 + a.half;
      } else {
        // Past the turned part of a q or k head, items follow each other.
        o0 = n * 2 * VEC;
        o1 = o0 + VEC;
      }
      if constexpr (STREAM) {
        x[u][0] = __builtin_nontemporal_load((const V*)(from + o0));
        x[u][1] = __builtin_nontemporal_load((const V*)(from + o1));
      } else {
        x[u][0] = *(const V*)(from + o0);
        x[u][1] = *(const V*)(from + o1);
      }
      to[u] += o0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (to[u] == nullptr) continue;
      int64_t second = VEC;
      if (at[u] >= 0) {
        const int tb = (int)div_by((uint32_t)(first + u * step), by_items);
        T e[2 * VEC];
        __builtin_memcpy(e, &x[u][0], sizeof(V));
        __builtin_memcpy(e + VEC, &x[u][1], sizeof(V));
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float2 cs = turn[tb][at[u] + j];
          T& ea = e[INTER ? 2 * j : j];
          T& eb = e[INTER ? 2 * j + 1 : VEC + j];
          const float p = dt<DT>::to_f32(ea), q = dt<DT>::to_f32(eb);
          ea = dt<DT>::from_f32(p * cs.x - q * cs.y);
          eb = dt<DT>::from_f32(q * cs.x + p * cs.y);
        }
        __builtin_memcpy(&x[u][0], e, sizeof(V));
        __builtin_memcpy(&x[u][1], e + VEC, sizeof(V));
        if (!INTER) second = a.half;
      }
      if constexpr (STREAM) {
        __builtin_nontemporal_store(x[u][0], (V*)to[u]);
        __builtin_nontemporal_store(x[u][1], (V*)(to[u] + second));
      } else {
        *(V*)to[u] = x[u][0];
        *(V*)(to[u] + second) = x[u][1];
      }
    }
  }
}

template <int DT, int VEC, bool INTER>
hipError_t launch(const RopeArgs& a) {
  const CacheArgs& c = a.c;
  const int per_head = c.dim / (2 * VEC), items = (a.q_heads + 2 * c.kv_heads) * per_head;
  const int turning = a.half / VEC;
  const FastDiv by_items = fast_div(items), by_head = fast_div(per_head);
  // With tokens for every compute unit several times over, four of them share
  // a workgroup; fewer are spread over workgroups a part of the heads each.
  if (c.tokens >= 4096) {
    rope_append_kernel<DT, VEC, INTER, 4><<<dim3((c.tokens + 3) / 4), ROPE_THREADS, 0, a.stream>>>(
        a, items, by_items, by_head, turning);
  } else {
    const int parts = (items + ROPE_THREADS - 1) / ROPE_THREADS;
    const int y = c.tokens >= 1024 ? 1 : parts < 16 ? parts : 16;
    rope_append_kernel<DT, VEC, INTER, 1><<<dim3(c.tokens, y), ROPE_THREADS, 0, a.stream>>>(
        a, items, by_items, by_head, turning);
  }
  return hipGetLastError();
}

template <int DT, int VEC>
hipError_t launch_layout(const RopeArgs& a) {
  return a.interleaved ? launch<DT, VEC, true>(a) : launch<DT, VEC, false>(a);
}

// The widest load that every stride, pointer and the turned part allow.
int width_of(const RopeArgs& a, int size) {
  const CacheArgs& c = a.c;
  const int64_t counts[] = {a.q_token, a.q_head, a.k_token, a.k_head, a.v_token, a.v_head,
                            a.out_token, a.out_head, c.k_page, c.k_head, c.k_token, c.v_page,
                            c.v_head, c.v_token};
  const uintptr_t bases[] = {(uintptr_t)a.q, (uintptr_t)a.k, (uintptr_t)a.v, (uintptr_t)a.out,
                             (uintptr_t)c.k, (uintptr_t)c.v};
  int vec = 16 / size;
  for (; vec > 1; vec /= 2) {
    bool ok = a.half % vec == 0 && c.dim % (2 * vec) == 0;
    for (int64_t n : counts) ok = ok && n % vec == 0;
    for (uintptr_t p : bases) ok = ok && p % (uintptr_t)(vec * size) == 0;
    if (ok) break;
  }
  return vec;
}

template <int DT>
hipError_t launch_type(const RopeArgs& a) {
  switch (width_of(a, (int)sizeof(typename dt<DT>::T))) {
    case 8: if constexpr (sizeof(typename dt<DT>::T) == 2) return launch_layout<DT, 8>(a);
    case 4: return launch_layout<DT, 4>(a);
    case 2: return launch_layout<DT, 2>(a);
    default: return launch_layout<DT, 1>(a);
  }
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs& a) {
  switch (a.dtype) {
    case DT_F32: return launch_type<DT_F32>(a);
    case DT_F16: return launch_type<DT_F16>(a);
    default: return launch_type<DT_BF16>(a);
  }
}

}  // namespace qmm
