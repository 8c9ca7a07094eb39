// paged_attn.h -- device code shared by the paged-attention kernels: the
// matrix-core steps of each type, a sequence's share of a batch and the place
// of a key in the cache.
//
// Both kernels compute scores and outputs transposed, S^T = K Q^T and
// O^T = V^T P^T, so that a query row is a lane column of every accumulator:
// its maximum, sum and rescaling factor are one register a lane, and the
// probabilities that leave S^T are, lane by lane, the B operand of the second
// product once V's keys are taken in the same order.
#pragma once

#include <hip/hip_runtime.h>

#include "mfma_ops.h"
#include "paged.h"
#include "qmm_device.h"

namespace qmm {

typedef __attribute__((address_space(1))) const void* global_ptr;
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;

// What stands in for keys past a sequence's end and for the columns that pad
// a head to the kernel's width: a row of zeros.
__device__ __attribute__((aligned(256))) const uint32_t zero_row[256] = {};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// 16 bytes a lane from global memory to consecutive LDS addresses.
__device__ __forceinline__ void load_to_lds(const char* from, char* to) {
  __builtin_amdgcn_global_load_lds((global_ptr)from, (lds_ptr)to, 16, 0, 0);
}

// Four 16-bit elements a lane, transposed in each group of 16 lanes: lane i
// names 8 bytes of a 4 x 16 block (row i / 4, columns 4 (i % 4) ..) and gets
// column i of its four rows.
__device__ __forceinline__ s16x4 lds_read_tr(const char* from) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)from);
}

// Every load to LDS has landed (vmcnt 0), and nothing below moves above.
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt(0x0F70);
  asm volatile("" ::: "memory");
}

// The value of lane n of each 16 (n is a constant once loops are unrolled).
template <int N> __device__ __forceinline__ uint32_t row_lane(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x150 + N, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t row_broadcast(uint32_t v, int n) {
  switch (n) {
    case 0: return row_lane<0>(v);
    case 1: return row_lane<1>(v);
    case 2: return row_lane<2>(v);
    case 3: return row_lane<3>(v);
    case 4: return row_lane<4>(v);
    case 5: return row_lane<5>(v);
    case 6: return row_lane<6>(v);
    default: return row_lane<7>(v);
  }
}

// Maximum and sum over the four lanes that share a column (lane mod 16).
__device__ __forceinline__ float col_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float col_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// One sequence of the batch.  Counts and lengths that do not fit the batch's
// own bounds are cut to them, so that every access stays inside its buffer.
struct Seq {
  int t0, n, len;   // first token, tokens, keys
};
__device__ __forceinline__ Seq seq_of(const CacheArgs& c, int s) {
  Seq q;
  int a = c.starts[s], b = c.starts[s + 1];
  a = a < 0 ? 0 : a;
  b = b > c.tokens ? c.tokens : b;
  q.t0 = a;
  q.n = b - a;
  q.n = q.n < 0 ? 0 : q.n > c.max_new ? c.max_new : q.n;
  const int64_t room = (int64_t)c.width * c.page;
  int len = c.lens[s];
  len = len < 0 ? 0 : len > c.max_len ? c.max_len : len;
  q.len = len > room ? (int)room : len;
  return q;
}

// The page of key j (in range of the table); a bad entry reads page 0 or the
// last one, in bounds.
__device__ __forceinline__ int page_of(const CacheArgs& c, const int32_t* row, int j, int& at) {
  const int col = (int)div_by((uint32_t)j, c.by_page);
  at = j - col * c.page;
  const int page = row[col];
  return page < 0 ? 0 : page >= c.pages ? c.pages - 1 : page;
}

// Probabilities enter the second product in the values' type.  f16 has no more
// than 24 bits below 1, and many keys that each hold less may be all of a row's
// output where a key that holds nearly everything has a small value (an
// attention sink): they are taken 2^(15 - slack) larger, 2^15 at most, where
// `slack` is how far (log2) a score may pass its reference.  bf16 and f32 have
// the range.
template <int DT> constexpr int prob_shift(int slack) { return DT == DT_F16 ? 15 - slack : 0; }
constexpr float exp2_of(int n) { return n < 0 ? 0.5f * exp2_of(n + 1) : n > 0 ? 2.f * exp2_of(n - 1) : 1.f; }

// The score of a raw product in units of log2: capped or only scaled.
struct ScoreScale {
  float mul, cap;   // plain: scale * log2(e); capped: scale / cap, cap * log2(e)
};
// tanh x for |x| < TANH_NEAR: the odd polynomial of five terms past x that fits
// it best there (by reweighted least squares), to 4.6e-9 of its value; its
// roundings in 32 bits come to more.
constexpr float TANH_NEAR = 0.6f;
__device__ __forceinline__ float tanh_near(float x) {
  const float u = x * x;
  float p = __builtin_fmaf(u, -0.005895133130f, 0.020795948803f);
  p = __builtin_fmaf(u, p, -0.053783822805f);
  p = __builtin_fmaf(u, p, 0.133319243789f);
  p = __builtin_fmaf(u, p, -0.333332985640f);
  return __builtin_fmaf(x * u, p, x);
}
template <bool CAP>
__device__ __forceinline__ float score(float s, const ScoreScale& k) {
  const float x = s * k.mul;
  if constexpr (!CAP) return x;
  // Far from 0, tanh x = 1 - 2 / (e^2x + 1), off by 2^-23 at most.
  const float e = exp2_fast(x * (2.f * LOG2E));
  const float far = 1.f - 2.f * __builtin_amdgcn_rcpf(e + 1.f);
  return k.cap * (fabsf(x) < TANH_NEAR ? tanh_near(x) : far);
}

}  // namespace qmm
