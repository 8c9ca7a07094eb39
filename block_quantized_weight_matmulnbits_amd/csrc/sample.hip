// sample.hip -- the choice of the next token: logits, filtered by top-k, top-p
// and min-p, and a given number u in [0, 1) for each row.
//
// With w_i = exp((l_i - max l) / T), tokens ordered by logit (ties: the lowest
// index first): K = the first top_k; P = the shortest beginning of K that holds
// top_p of K's sum; of those, the ones with w_i >= min_p.  The token is the first
// one in the order of the indices whose running sum passes u times the whole.
//
// Sums decide which token a number falls on, so weights are formed in 64 bits and
// added as whole numbers, of which no order of addition changes a bit: w is held
// to 2^-SHIFT, SHIFT = 62 - log2(vocab) (45 bits for 131072 tokens).
//
// Nothing is sorted.  A row is cut into chunks and read three times (from HBM
// once: a batch's logits stay in the caches): for its maximum; for how many
// tokens, and how much weight, lie in each of 1024 buckets of their distance from
// it, which says in which bucket top-k and top-p end; and for the sum of each
// chunk before those buckets and a list of what is in them.  One workgroup a row
// then finds the last token that is kept, digit by digit of (logit, index) over
// the list, and the chunk and the token that u falls on.  The list is long only
// where thousands of logits are nearly equal; such a row is searched as a whole,
// eight bits of the places a scan (a flat row of 131072 under top-p 520 us, one of
// equal logits 1010; 64 of them 590 and 1130).
// Rows that fit the list are done in one launch.
//
// The bound is not memory: one row of 131072 (0.26 MB) takes 3.4 + 6.5 + 7.5 + 10.4
// us in its four launches, each a chain of dependent loads, scans and barriers; 64
// rows with settings of their own take 10 (1.7 TB/s) + 20 + 22 + 17 us, where the
// rows that filter by top-p or not at all need a 64-bit exp for every token and
// come to lie on the same compute units.  An exp with half of the 64-bit operations
// (32 roots of 2 in LDS and 6 terms) and lists gathered in LDS before one atomic were
// each slower by their own start.
#include <algorithm>

#include "decode.h"
#include "qmm_device.h"

namespace qmm {
namespace {

constexpr int BUCKETS = 1024, PER_UNIT = 32;   // buckets of 1 / 32 of a nat
constexpr int LIST = 4096;                     // tokens of a list
constexpr int RANKED = 256;                    // so many are compared each with each
constexpr int STEP = 2048;                     // tokens that a workgroup reads at once
constexpr int MAX_TILES = 64;
constexpr int64_t BATCH = 2048;                // rows that the workspace holds at once
constexpr int PASS_THREADS = 256, LAST_THREADS = 1024, LAST_WAVES = LAST_THREADS / 64;

// How a row is cut: tiles, of which sums are kept, and chunks of whole tiles, a
// workgroup's in the passes.
struct Cut {
  int tile, tiles, chunk, chunks;
};

// Where top-k and top-p end, as far as the buckets tell.
struct Ends {
  int k_bucket;                  // top-k's (BUCKETS: it keeps all)
  int p_from, p_upto;            // top-p's is one of these (BUCKETS: it keeps all)
  uint32_t listed;               // tokens in these buckets
  uint64_t k_count, k_weight;    // tokens and weight before k_bucket
  uint64_t p_weight;             // weight before p_from
  // Kept for certain; to be looked at.
  __device__ __forceinline__ bool before(int b) const { return b < (p_from < k_bucket ? p_from : k_bucket); }
  __device__ __forceinline__ bool at(int b) const { return b == k_bucket || (b >= p_from && b <= p_upto); }
};

// What the passes leave of a row.
struct RowWork {
  Ends ends;
  uint64_t first[MAX_TILES];     // the place of each chunk's first token
  uint64_t sums[MAX_TILES];      // weight of each tile's tokens before the listed ones
  uint64_t bucket_weight[BUCKETS];
  uint32_t bucket_count[BUCKETS];
  uint32_t listed;               // tokens in the list
  uint32_t unused;
  uint32_t list[LIST];           // indices
};

// Orders as the values do; a NaN below all, so that it is never chosen.
template <int DT>
__device__ __forceinline__ float logit(const char* row, int i) {
  const float v = dt<DT>::to_f32(((const typename dt<DT>::T*)row)[i]);
  return v != v ? -INFINITY : v;
}

// The place of a token in the order, larger first: the logit's bits (-0 as 0) in
// the order of the values, then the index.  16-bit logits need only their own.
constexpr int INDEX_BITS = 24;
template <int DT> constexpr int place_bits() { return INDEX_BITS + (DT == DT_F32 ? 32 : 16); }
template <int DT>
__device__ __forceinline__ uint64_t place_of(float v, int i) {
  uint32_t b;
  if constexpr (DT == DT_F16) {
    const uint32_t h = __builtin_bit_cast(uint16_t, (_Float16)(v + 0.f));
    b = h & 0x8000u ? ~h & 0xFFFFu : h | 0x8000u;
  } else {
    b = __float_as_uint(v + 0.f);
    b ^= (uint32_t)((int32_t)b >> 31) | 0x80000000u;
    if (DT == DT_BF16) b >>= 16;
  }
  return (uint64_t)b << INDEX_BITS | (uint32_t)((1 << INDEX_BITS) - 1 - i);
}
template <int DT> __device__ __forceinline__ float value_of(uint64_t place) {
  uint32_t b = (uint32_t)(place >> INDEX_BITS);
  if constexpr (DT == DT_F16)
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(b & 0x8000u ? b & 0x7FFFu : ~b));
  if (DT == DT_BF16) b <<= 16;
  b = b & 0x80000000u ? b & 0x7FFFFFFFu : ~b;
  return __uint_as_float(DT == DT_BF16 ? b & 0xFFFF0000u : b);
}
__device__ __forceinline__ int index_of(uint64_t place) {
  return (1 << INDEX_BITS) - 1 - (int)(place & ((1 << INDEX_BITS) - 1));
}

// exp(x) 2^shift for x <= 0 in 64 bits: 2^n times the Taylor polynomial of degree 12
// in |r| <= ln 2 / 2 (its rest is at most 1.04 2^-52 of the value).  Where the result
// would be far below 1 it is 0.
__device__ __forceinline__ double exp_f64(double x, int shift) {
  const bool far = !(x > -700.0);
  x = far ? 0.0 : x;
  const double n = rint(x * 1.4426950408889634074);
  // ln 2 in two parts, the first of 29 bits, so that n times it is exact.
  double r = __builtin_fma(n, -0x1.62e42ff000000p-1, x);
  r = __builtin_fma(n, 0x1.718432a1b0e26p-35, r);
  double p = 1.0 / 479001600.0;
  p = __builtin_fma(p, r, 1.0 / 39916800.0);
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return far ? 0.0 : ldexp(p, (int)n + shift);
}

// A row's settings and the weights of its tokens.
struct Row {
  float top;
  double over_t;         // 1 / T
  float per_bucket;      // buckets a unit of the logit
  int shift, k;          // k >= vocab: all
  double p, min_units, u;
  float little;          // logits below have less than min_p of the first's weight
  bool one;              // only the first token

  // The weight in units of 2^-shift, before it is rounded to a whole number.
  __device__ __forceinline__ double weight(float l) const {
    // Infinite logits share everything equally.
    const double d = l == top ? 0.0 : (double)l - (double)top;
    return exp_f64(d * over_t, shift);
  }
  // The nearest whole number of a w <= 2^62: its upper and lower 32 bits.
  static __device__ __forceinline__ uint64_t units(double w) {
    w = rint(w);
    const double hi = floor(w * 0x1p-32);
    return (uint64_t)(uint32_t)hi << 32 | (uint32_t)__builtin_fma(hi, -0x1p32, w);
  }
  // Does not fall as the logit does: a difference and a product, both rounded.
  __device__ __forceinline__ int bucket(float l) const {
    if (l == top) return 0;
    const float d = (top - l) * per_bucket;
    return d < (float)(BUCKETS - 1) ? (int)d : BUCKETS - 1;
  }
  __device__ __forceinline__ bool all(int vocab) const { return k >= vocab && p >= 1.0; }
};

__device__ Row row_of(const SampleArgs& a, int64_t row, float top, int shift) {
  Row r;
  r.top = top;
  const float t = a.temperature ? a.temperature[row] : 1.f;
  const bool greedy = !(t > 0.f);
  r.over_t = greedy ? 1.0 : 1.0 / (double)t;
  r.per_bucket = greedy ? (float)PER_UNIT : (float)PER_UNIT / t;
  r.shift = shift;
  r.k = a.top_k ? a.top_k[row] : 0;
  if (r.k <= 0 || r.k > a.vocab) r.k = a.vocab;
  if (greedy) r.k = 1;
  const float p = a.top_p ? a.top_p[row] : 1.f, m = a.min_p ? a.min_p[row] : 0.f;
  r.p = p < 1.f ? (p > 0.f ? p : 0.0) : 1.0;
  r.min_units = ldexp(m > 0.f ? (m < 1.f ? (double)m : 1.0) : 0.0, shift);
  r.u = a.uniform[row];
  r.one = r.k == 1;
  // exp((l - top) / T) < min_p without the exp: l below top + T log min_p, by more
  // than the roundings of either side (2^-49 of a weight near 1, a few of the log's 24
  // bits, of top and of T log min_p in 64 bits, of the bound in 32).  Infinities leave
  // all to the exp.  256 rows of 32000 with min_p alone: 36 us without, 30 with it.
  r.little = -INFINITY;
  if (a.min_p && m > 0.f) {
    const double off = (double)t * (double)logf(fminf(m, 1.f));
    const double bound = (double)top + off - 1e-6 * (fabs((double)top) + fabs(off)) - 1e-12 * (double)t;
    if (top < INFINITY && bound > -1e30) r.little = (float)bound;
  }
  return r;
}

__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const uint64_t u = __shfl_xor(v, o);
    v = u > v ? u : v;
  }
  return v;
}
// Sum over this lane and those before it.
__device__ __forceinline__ uint64_t wave_upto_u64(uint64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// body(i, logits, n) for the tokens [begin, end) of a row, n <= EIGHT side by side a
// thread (past n: minus infinity), and after(i0) for every STEP of them; AHEAD steps
// are loaded at once.
constexpr int EIGHT = 8;
template <int DT, int AHEAD, typename Body, typename After>
__device__ __forceinline__ void each_eight(const char* row, int begin, int end, Body body, After after) {
  using T = typename dt<DT>::T;
  for (int i0 = begin; i0 < end; i0 += STEP * AHEAD) {
    T e[AHEAD][EIGHT];
#pragma unroll
    for (int v = 0; v < AHEAD; ++v) {
      const int i = i0 + v * STEP + (int)threadIdx.x * EIGHT;
      if (i + EIGHT <= end) {
        __builtin_memcpy(e[v], (const T*)row + i, sizeof(e[v]));   // at any address
      } else {
#pragma unroll
        for (int j = 0; j < EIGHT; ++j) e[v][j] = ((const T*)row)[i + j < end ? i + j : end - 1];
      }
    }
#pragma unroll
    for (int v = 0; v < AHEAD; ++v) {
      const int i = i0 + v * STEP + (int)threadIdx.x * EIGHT;
      const int n = min(EIGHT, end - i);
      if (n > 0) {
        float l[EIGHT];
#pragma unroll
        for (int j = 0; j < EIGHT; ++j) {
          l[j] = dt<DT>::to_f32(e[v][j]);
          l[j] = j < n && l[j] == l[j] ? l[j] : -INFINITY;
        }
        body(i, l, n);
      }
      if (i0 + v * STEP < end) after(i0 + v * STEP);
    }
  }
}

template <int DT>
__device__ __forceinline__ const char* row_at(const SampleArgs& a, int64_t row) {
  return a.logits + row * a.stride * (int64_t)sizeof(typename dt<DT>::T);
}
// The first token of a row, from the chunks' (every wave for itself).
__device__ __forceinline__ uint64_t first_of(const RowWork& w, int chunks) {
  const int lane = threadIdx.x & 63;
  return wave_max_u64(lane < chunks ? w.first[lane] : 0);
}

// The first pass: the first token of each chunk, and a clean slate.
template <int DT>
__global__ __launch_bounds__(PASS_THREADS) void first_kernel(SampleArgs a, RowWork* work, Cut cut) {
  const int64_t row = blockIdx.x / cut.chunks;
  const int c = blockIdx.x % cut.chunks, begin = c * cut.chunk, end = min(begin + cut.chunk, a.vocab);
  RowWork& w = work[row];
  // A thread meets its tokens in their order: the first of equal ones stays.
  float top = -INFINITY;
  int at = begin;
  each_eight<DT, 4>(row_at<DT>(a, row), begin, end, [&](int i, const float (&l)[EIGHT], int) {
#pragma unroll
    for (int j = 0; j < EIGHT; ++j) {
      at = l[j] > top ? i + j : at;
      top = fmaxf(top, l[j]);
    }
  }, [](int) {});
  uint64_t best = top == -INFINITY ? place_of<DT>(top, begin) : place_of<DT>(top, at);
  __shared__ uint64_t waves[PASS_THREADS / 64];
  best = wave_max_u64(best);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = best;
  for (int b = c * PASS_THREADS + threadIdx.x; b < BUCKETS; b += cut.chunks * PASS_THREADS) {
    w.bucket_weight[b] = 0;
    w.bucket_count[b] = 0;
  }
  if (c == 0 && threadIdx.x == 0) w.listed = 0;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int v = 1; v < PASS_THREADS / 64; ++v) best = waves[v] > best ? waves[v] : best;
    w.first[c] = best;
  }
}

// The second pass: the buckets, where a row is filtered.
template <int DT>
__global__ __launch_bounds__(PASS_THREADS) void bucket_kernel(SampleArgs a, RowWork* work, Cut cut, int shift) {
  const int64_t row = blockIdx.x / cut.chunks;
  const int c = blockIdx.x % cut.chunks, begin = c * cut.chunk, end = min(begin + cut.chunk, a.vocab);
  RowWork& w = work[row];
  const char* logits = row_at<DT>(a, row);
  const Row r = row_of(a, row, value_of<DT>(first_of(w, cut.chunks)), shift);
  if (r.top == -INFINITY || r.one || r.all(a.vocab)) return;
  __shared__ uint64_t weight[BUCKETS];
  __shared__ uint32_t count[BUCKETS];
  for (int b = threadIdx.x; b < BUCKETS; b += PASS_THREADS) {
    weight[b] = 0;
    count[b] = 0;
  }
  __syncthreads();
  const bool weigh = r.p < 1.0;
  // Eight exps at once: one after another, each waited for the last one's steps (7 f32
  // rows of 50021: 17.0 us, 15.9 so).
  each_eight<DT, 2>(logits, begin, end, [&](int, const float (&l)[EIGHT], int n) {
    int b[EIGHT];
#pragma unroll
    for (int j = 0; j < EIGHT; ++j) b[j] = r.bucket(l[j]);
#pragma unroll
    for (int j = 0; j < EIGHT; ++j)
      if (j < n) atomicAdd(&count[b[j]], 1u);
    if (!weigh) return;
    uint64_t units[EIGHT];
#pragma unroll
    for (int j = 0; j < EIGHT; ++j) units[j] = Row::units(r.weight(l[j]));
#pragma unroll
    for (int j = 0; j < EIGHT; ++j)
      if (units[j]) atomicAdd((unsigned long long*)&weight[b[j]], (unsigned long long)units[j]);
  }, [](int) {});
  __syncthreads();
  for (int b = threadIdx.x; b < BUCKETS; b += PASS_THREADS) {
    if (count[b]) atomicAdd(&w.bucket_count[b], count[b]);
    if (weight[b]) atomicAdd((unsigned long long*)&w.bucket_weight[b], (unsigned long long)weight[b]);
  }
}

// By a workgroup of the passes, BUCKETS / 256 buckets a thread.
__device__ Ends ends_of(const RowWork& w, const Row& r, int vocab) {
  constexpr int EACH = BUCKETS / PASS_THREADS, WAVES = PASS_THREADS / 64;
  __shared__ uint64_t wave_n[WAVES], wave_w[WAVES], say[3][3];
  __shared__ int where[3];
  __shared__ uint32_t listed[WAVES];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  uint64_t n[EACH], v[EACH], sum_n = 0, sum_w = 0;
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    n[j] = w.bucket_count[t * EACH + j];
    v[j] = w.bucket_weight[t * EACH + j];
  }
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    sum_n += n[j];
    sum_w += v[j];
  }
  uint64_t upto_n = wave_upto_u64(sum_n, lane), upto_w = wave_upto_u64(sum_w, lane);
  if (lane == 63) {
    wave_n[wave] = upto_n;
    wave_w[wave] = upto_w;
  }
  if (t < 3) {
    where[t] = BUCKETS;
    say[t][0] = say[t][1] = say[t][2] = 0;
  }
  __syncthreads();
  uint64_t all = 0;
#pragma unroll
  for (int k = 0; k < WAVES; ++k) {
    if (k < wave) {
      upto_n += wave_n[k];
      upto_w += wave_w[k];
    }
    all += wave_w[k];
  }
  const uint64_t from_n = upto_n - sum_n, from_w = upto_w - sum_w;
  // The bucket in which a running sum (of counts or weights) reaches `want`; what
  // lies before it, and its weight.
  auto reach = [&](const uint64_t (&x)[EACH], uint64_t from, uint64_t upto, uint64_t want, int slot) {
    if (!(from < want && upto >= want)) return;
    uint64_t at_n = from_n, at_w = from_w;
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      if (from < want && from + x[j] >= want) {
        where[slot] = t * EACH + j;
        say[slot][0] = at_n;
        say[slot][1] = at_w;
        say[slot][2] = v[j];
      }
      from += x[j];
      at_n += n[j];
      at_w += v[j];
    }
  };
  if (r.k < vocab) {
    reach(n, from_n, upto_n, r.k, 0);
    __syncthreads();
  }
  Ends e;
  e.k_bucket = where[0];
  e.k_count = say[0][0];
  e.k_weight = e.k_bucket < BUCKETS ? say[0][1] : all;
  e.p_from = e.p_upto = BUCKETS;
  e.p_weight = 0;
  if (r.p < 1.0) {
    // top-k's own sum lies between the weight before its bucket and with it.
    const double lo = ceil(r.p * (double)e.k_weight);
    const double hi = ceil(r.p * (double)(e.k_bucket < BUCKETS ? e.k_weight + say[0][2] : all));
    reach(v, from_w, upto_w, lo < 1.0 ? 1 : (uint64_t)lo, 1);
    reach(v, from_w, upto_w, hi < 1.0 ? 1 : (uint64_t)hi, 2);
    __syncthreads();
    e.p_from = where[1];
    e.p_upto = where[2];
    e.p_weight = say[1][1];
  }
  uint32_t sum = 0;
#pragma unroll
  for (int j = 0; j < EACH; ++j) sum += e.at(t * EACH + j) ? (uint32_t)n[j] : 0u;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) listed[wave] = sum;
  __syncthreads();
  e.listed = 0;
#pragma unroll
  for (int k = 0; k < WAVES; ++k) e.listed += listed[k];
  return e;
}

// The third pass: the weight of each chunk before the ends, and the list.
template <int DT>
__global__ __launch_bounds__(PASS_THREADS) void list_kernel(SampleArgs a, RowWork* work, Cut cut, int shift) {
  const int64_t row = blockIdx.x / cut.chunks;
  const int c = blockIdx.x % cut.chunks, begin = c * cut.chunk, end = min(begin + cut.chunk, a.vocab);
  RowWork& w = work[row];
  const char* logits = row_at<DT>(a, row);
  const Row r = row_of(a, row, value_of<DT>(first_of(w, cut.chunks)), shift);
  if (r.top == -INFINITY || r.one) return;
  const bool all = r.all(a.vocab);
  Ends e;
  if (!all) {
    e = ends_of(w, r, a.vocab);
    if (c == 0 && threadIdx.x == 0) w.ends = e;
    if (e.listed > LIST) return;   // the row is searched as a whole
  }
  __shared__ uint64_t waves[MAX_TILES][PASS_THREADS / 64];
  uint64_t sum = 0;
  each_eight<DT, 2>(logits, begin, end, [&](int i, const float (&l)[EIGHT], int n) {
    bool weigh[EIGHT], any = false;
#pragma unroll
    for (int j = 0; j < EIGHT; ++j) {
      const int b = all ? 0 : r.bucket(l[j]);
      const bool before = all || e.before(b);
      weigh[j] = before && l[j] > -INFINITY && !(l[j] < r.little);
      any |= weigh[j];
      if (!before && e.at(b) && j < n) {
        // In any order: the list is a set.
        const uint32_t at = atomicAdd(&w.listed, 1u);
        if (at < LIST) w.list[at] = i + j;
      }
    }
    if (!any) return;
    if (r.min_units > 0.0) {
      // Few of them: 256 rows with min_p take 34 us with eight exps at once, 30 so.
#pragma unroll
      for (int j = 0; j < EIGHT; ++j)
        if (weigh[j]) {
          const double x = r.weight(l[j]);
          if (x >= r.min_units) sum += Row::units(x);
        }
    } else {
#pragma unroll
      for (int j = 0; j < EIGHT; ++j) {
        const uint64_t n_units = Row::units(r.weight(l[j]));
        sum += weigh[j] ? n_units : 0;
      }
    }
  }, [&](int i0) {
    // The end of a tile, or of the row.
    if ((i0 - begin + STEP) % cut.tile != 0 && i0 + STEP < end) return;
    sum = wave_sum_u64(sum);
    if ((threadIdx.x & 63) == 0) waves[(i0 - begin) / cut.tile][threadIdx.x >> 6] = sum;
    sum = 0;
  });
  __syncthreads();
  const int t0 = begin / cut.tile, t = threadIdx.x;
  if (t < cut.chunk / cut.tile && t0 + t < cut.tiles) {
    uint64_t s = 0;
    for (int v = 0; v < PASS_THREADS / 64; ++v) s += waves[t][v];
    w.sums[t0 + t] = s;
  }
}

struct Search {
  uint64_t amounts[256];
  uint32_t counts[256];
  uint64_t waves[LAST_WAVES];
  uint64_t left, last;
  uint32_t digit, single, found;
};

// The place of the last token of the shortest beginning of the order whose
// amounts reach `want`, among the places from `from` on; 0 where all of them
// together do not.  each(body): body(place, amount) for every token to look at.
template <int DT, typename Each>
__device__ uint64_t threshold(Search& s, uint64_t from, uint64_t want, Each each) {
  uint64_t prefix = 0;
  for (int bit = place_bits<DT>() - 8; bit >= 0; bit -= 8) {
    __syncthreads();
    if (threadIdx.x < 256) {
      s.amounts[threadIdx.x] = 0;
      s.counts[threadIdx.x] = 0;
    }
    __syncthreads();
    each([&](uint64_t at, uint64_t amount) {
      if (at < from || at >> (bit + 8) != prefix || amount == 0) return;
      atomicAdd((unsigned long long*)&s.amounts[at >> bit & 255], (unsigned long long)amount);
      atomicAdd(&s.counts[at >> bit & 255], 1u);
    });
    __syncthreads();
    // The digit, from the largest down, at which the amounts reach `want`.
    if (threadIdx.x < 64) {
      const int lane = threadIdx.x;
      uint64_t own = 0, four[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) own += four[j] = s.amounts[255 - (lane * 4 + j)];
      const uint64_t upto = wave_upto_u64(own, lane), all = __shfl(upto, 63);
      if (lane == 0) s.found = all >= want;
      uint64_t before = upto - own;
      if (before < want && upto >= want) {
        int found = -1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (found < 0 && before + four[j] >= want) found = j;
          if (found < 0) before += four[j];
        }
        s.digit = 255 - (lane * 4 + found);
        s.left = want - before;
        s.single = s.counts[s.digit] == 1;
      }
    }
    __syncthreads();
    if (!s.found) return 0;
    prefix = prefix << 8 | s.digit;
    want = s.left;
    if (s.single && bit > 0) {
      // One token is left: it is the last.
      each([&](uint64_t at, uint64_t amount) {
        if (at >= from && at >> bit == prefix && amount != 0) s.last = at;
      });
      __syncthreads();
      return s.last;
    }
  }
  return prefix;
}

// The last launch, a workgroup a row.  WHOLE: the only one, for rows that fit the
// list.
template <int DT, bool WHOLE>
__global__ __launch_bounds__(LAST_THREADS) void last_kernel(SampleArgs a, RowWork* work, Cut cut, int shift) {
  __shared__ Search s;
  __shared__ float list[LIST];       // the logits of the listed tokens,
  __shared__ int index[WHOLE ? 1 : LIST];   // and their indices
  __shared__ uint64_t list_weight[WHOLE ? 1 : RANKED], list_place[WHOLE ? 1 : RANKED];
  __shared__ uint64_t sums[MAX_TILES];
  __shared__ uint64_t begin_sum;
  __shared__ int begin_tile;
  const int64_t row = blockIdx.x;
  const char* logits = row_at<DT>(a, row);
  const int vocab = a.vocab, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

  uint64_t first;
  if constexpr (WHOLE) {
    first = 0;
    for (int i = threadIdx.x; i < vocab; i += LAST_THREADS) {
      const float l = logit<DT>(logits, i);
      list[i] = l;
      const uint64_t at = place_of<DT>(l, i);
      first = at > first ? at : first;
    }
    first = wave_max_u64(first);
    if (lane == 0) s.waves[wave] = first;
    __syncthreads();
    for (int v = 0; v < LAST_WAVES; ++v) first = s.waves[v] > first ? s.waves[v] : first;
    __syncthreads();
  } else {
    first = first_of(work[row], cut.chunks);
  }
  const Row r = row_of(a, row, value_of<DT>(first), shift);
  auto answer = [&](int token, float logprob) {
    a.tokens[row] = token;
    if (a.logprobs) a.logprobs[row] = logprob;
  };
  if (r.top == -INFINITY || r.one) {
    // Nothing is left to choose from, or no choice.
    if (threadIdx.x == 0) {
      if (r.top == -INFINITY) answer(-1, -INFINITY);
      else answer(index_of(first), 0.f);
    }
    return;
  }

  // The place of the last token that is kept, and the chunks' sums.
  uint64_t from = 0;
  auto sum_all = [&](uint64_t v) {
    v = wave_sum_u64(v);
    __syncthreads();
    if (lane == 0) s.waves[wave] = v;
    __syncthreads();
    uint64_t t = 0;
    for (int k = 0; k < LAST_WAVES; ++k) t += s.waves[k];
    return t;
  };
  // Both filters over some tokens: every(body) calls body(i, logit) for each, of
  // which `in` says whether a filter's end may lie there.
  auto filter = [&](auto every, auto in_k, auto in_p, uint64_t k_want, uint64_t k_weight, uint64_t p_weight) {
    uint64_t k_from = 0;
    if (r.k < vocab)
      k_from = threshold<DT>(s, 0, k_want, [&](auto body) {
        every([&](int i, float l) {
          if (in_k(l)) body(place_of<DT>(l, i), (uint64_t)1);
        });
      });
    from = k_from;
    if (r.p < 1.0) {
      uint64_t sum = 0;
      every([&](int i, float l) {
        if (in_k(l) && place_of<DT>(l, i) >= k_from) sum += r.units(r.weight(l));
      });
      // A token is kept while the sum before it is below p times the whole: the
      // last one is where the sum reaches that.
      const double want = ceil(r.p * (double)(k_weight + sum_all(sum)));
      const uint64_t p_from = threshold<DT>(s, k_from, (want < 1.0 ? 1 : (uint64_t)want) - p_weight, [&](auto body) {
        every([&](int i, float l) {
          if (in_p(l)) body(place_of<DT>(l, i), r.units(r.weight(l)));
        });
      });
      from = p_from > from ? p_from : from;
    }
  };
  auto always = [](float) { return true; };
  auto whole_row = [&](auto body) {
    for (int i = threadIdx.x; i < vocab; i += LAST_THREADS) body(i, WHOLE ? list[WHOLE ? i : 0] : logit<DT>(logits, i));
  };
  auto kept = [&](float l, int i, double* x) {
    if (l < r.little || place_of<DT>(l, i) < from) return (uint64_t)0;
    *x = r.weight(l);
    return *x >= r.min_units ? Row::units(*x) : 0;
  };
  double x;
  int at = 0, upto = vocab;          // where the token is looked for
  uint64_t before = 0, total = 0;
  bool searched = WHOLE;
  if constexpr (WHOLE) {
    if (!r.all(vocab)) filter(whole_row, always, always, r.k, 0, 0);
  } else {
    RowWork& w = work[row];
    const bool all = r.all(vocab);
    Ends e;
    if (!all) e = w.ends;
    if (!all && e.listed > LIST) {
      filter(whole_row, always, always, r.k, 0, 0);
      searched = true;
    } else {
      if ((int)threadIdx.x < cut.tiles) sums[threadIdx.x] = w.sums[threadIdx.x];
      if (!all) {
        const int n = (int)e.listed;
        for (int j = threadIdx.x; j < n; j += LAST_THREADS) {
          const int i = w.list[j];
          const float l = logit<DT>(logits, i);
          index[j] = i;
          list[j] = l;
          if (n <= RANKED) {
            list_place[j] = place_of<DT>(l, i);
            list_weight[j] = Row::units(r.weight(l));
          }
        }
        if (threadIdx.x == 0) s.left = s.last = 0;
        __syncthreads();
        auto listed = [&](auto body) {
          for (int j = threadIdx.x; j < n; j += LAST_THREADS) body(index[j], list[j]);
        };
        auto in_k = [&](float l) { return r.bucket(l) == e.k_bucket; };
        auto in_p = [&](float l) { const int b = r.bucket(l); return b >= e.p_from && b <= e.p_upto; };
        if (n <= RANKED) {
          // Few: how many come before a token, and how much, counted one by one, by
          // as many neighbouring threads a token as there are.
          int group = 1;
          while (group < 64 && 2 * group * n <= LAST_THREADS) group *= 2;
          const int j = threadIdx.x / group, part = threadIdx.x % group;
          const bool mine = j < n;
          const float l = mine ? list[j] : 0.f;
          const uint64_t own = mine ? list_place[j] : 0;
          const bool k_mine = mine && in_k(l), p_mine = mine && in_p(l);
          uint32_t count = 0;
          uint64_t weight = 0;
          for (int o = part; o < n; o += group) {
            // Larger places lie in the same bucket or before it.
            const bool more = list_place[o] > own;
            count += more;
            weight += more ? list_weight[o] : 0;
          }
          for (int d = 1; d < group; d <<= 1) {
            count += __shfl_xor(count, d);
            weight += __shfl_xor(weight, d);
          }
          // Of a token in top-k's bucket, those in top-p's before it were counted, too.
          uint64_t p_count = 0;
          if (e.k_bucket < BUCKETS && e.p_from < e.k_bucket) {
            const bool one = mine && part == 0 && p_mine && !k_mine;
            p_count = sum_all(one ? 1 : 0);
          }
          const bool k_keep = !mine ? false : k_mine ? e.k_count + count - p_count < (uint64_t)r.k : true;
          const bool chosen = mine && part == 0;
          const uint64_t whole = e.k_weight + sum_all(chosen && k_mine && k_keep ? list_weight[j] : 0);
          const double want = ceil(r.p * (double)whole);
          const uint64_t reach = want < 1.0 ? 1 : (uint64_t)want;
          const bool keep = k_keep && (r.p < 1.0 ? p_mine && e.p_weight + weight < reach : k_mine);
          // The last place that is kept; all that are larger are, too.
          uint64_t least = chosen && keep ? ~own : 0, most = mine ? own : 0;
          least = wave_max_u64(least);
          most = wave_max_u64(most);
          if (lane == 0) {
            atomicMax((unsigned long long*)&s.left, (unsigned long long)least);
            atomicMax((unsigned long long*)&s.last, (unsigned long long)most);
          }
          __syncthreads();
          from = s.left ? ~s.left : s.last + 1;
        } else {
          filter(listed, in_k, in_p, r.k - e.k_count, e.k_weight, e.p_weight);
        }
        listed([&](int i, float l) {
          const uint64_t n = kept(l, i, &x);
          if (n) atomicAdd((unsigned long long*)&sums[i / cut.tile], (unsigned long long)n);
        });
      }
      __syncthreads();
      // The tile that u falls on.
      if (wave == 0) {
        const uint64_t own = lane < cut.tiles ? sums[lane] : 0, upto_here = wave_upto_u64(own, lane);
        const uint64_t everything = __shfl(upto_here, 63);
        const double target = fmin(fmax(r.u, 0.0), 1.0 - 0x1p-53) * (double)everything;
        const uint64_t here = __ballot((double)upto_here > target);
        if (lane == __builtin_ctzll(here)) {
          begin_tile = lane;
          begin_sum = upto_here - own;
        }
        if (lane == 0) s.last = everything;
      }
      __syncthreads();
      at = begin_tile * cut.tile;
      upto = min(at + cut.tile, vocab);
      before = begin_sum;
      total = s.last;
    }
  }
  // Tokens that are kept, a run for each wave; the first whose running sum passes
  // u times the whole lies in one wave's.
  const int run = (upto - at + LAST_WAVES * 64 - 1) / (LAST_WAVES * 64) * 64;
  const int begin = at + wave * run, end = min(begin + run, upto);
  auto token = [&](int i) { return WHOLE ? list[WHOLE ? i : 0] : logit<DT>(logits, i); };
  uint64_t sum = 0;
  for (int i = begin + lane; i < end; i += 64) sum += kept(token(i), i, &x);
  sum = wave_sum_u64(sum);
  __syncthreads();
  if (lane == 0) s.waves[wave] = sum;
  __syncthreads();
  if (searched) {
    for (int v = 0; v < LAST_WAVES; ++v) total += s.waves[v];
  }
  for (int v = 0; v < wave; ++v) before += s.waves[v];
  const double target = fmin(fmax(r.u, 0.0), 1.0 - 0x1p-53) * (double)total;
  if (!((double)before <= target && (double)(before + sum) > target)) return;
  for (int i0 = begin; i0 < end; i0 += 64) {
    const int i = i0 + lane;
    const uint64_t upto_here = before + wave_upto_u64(i < end ? kept(token(i), i, &x) : 0, lane);
    const uint64_t here = __ballot((double)upto_here > target);
    if (here) {
      if (lane == __builtin_ctzll(here)) answer(i, (float)(log(x) - log((double)total)));
      return;
    }
    before = __shfl(upto_here, 63);
  }
}

// Tiles of 2048 tokens where 64 of them hold the row.  Chunks: some four
// workgroups a compute unit, since each has to clear, add and read the buckets (64
// rows of 131072 with two, four, eight: 87, 70, 69 us under the profiler; 256 of 32000:
// 34, 32, 33).
Cut cut_of(int64_t rows, int64_t vocab) {
  Cut c;
  c.tile = (int)((vocab + MAX_TILES * STEP - 1) / (MAX_TILES * STEP) * STEP);
  c.tiles = (int)((vocab + c.tile - 1) / c.tile);
  const int64_t each = std::max<int64_t>(1, rows * c.tiles / 1024);
  c.chunk = (int)std::min<int64_t>(each, c.tiles) * c.tile;
  c.chunks = (int)((vocab + c.chunk - 1) / c.chunk);
  return c;
}

template <int DT>
hipError_t launch(const SampleArgs& all, RowWork* work) {
  int shift = 62;
  while (((int64_t)1 << (62 - shift)) < all.vocab) --shift;
  if (all.vocab <= LIST) {
    last_kernel<DT, true><<<dim3((uint32_t)all.rows), LAST_THREADS, 0, all.stream>>>(all, nullptr, Cut{}, shift);
    return hipGetLastError();
  }
  for (int64_t r0 = 0; r0 < all.rows; r0 += BATCH) {
    SampleArgs a = all;
    a.rows = std::min<int64_t>(BATCH, all.rows - r0);
    a.logits += r0 * a.stride * (int64_t)sizeof(typename dt<DT>::T);
    a.temperature = a.temperature ? a.temperature + r0 : nullptr;
    a.top_k = a.top_k ? a.top_k + r0 : nullptr;
    a.top_p = a.top_p ? a.top_p + r0 : nullptr;
    a.min_p = a.min_p ? a.min_p + r0 : nullptr;
    a.uniform += r0;
    a.tokens += r0;
    a.logprobs = a.logprobs ? a.logprobs + r0 : nullptr;
    const Cut c = cut_of(a.rows, a.vocab);
    const dim3 grid((uint32_t)(a.rows * c.chunks));
    first_kernel<DT><<<grid, PASS_THREADS, 0, a.stream>>>(a, work, c);
    if (a.top_k != nullptr || a.top_p != nullptr)
      bucket_kernel<DT><<<grid, PASS_THREADS, 0, a.stream>>>(a, work, c, shift);
    list_kernel<DT><<<grid, PASS_THREADS, 0, a.stream>>>(a, work, c, shift);
    last_kernel<DT, false><<<dim3((uint32_t)a.rows), LAST_THREADS, 0, a.stream>>>(a, work, c, shift);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t sample_workspace_bytes(int64_t rows, int64_t vocab) {
  return vocab <= LIST ? 256 : 256 + (size_t)std::min(rows, BATCH) * sizeof(RowWork);
}

hipError_t launch_sample(const SampleArgs& a, char* workspace) {
  RowWork* work = (RowWork*)workspace;
  switch (a.dtype) {
    case DT_F32: return launch<DT_F32>(a, work);
    case DT_F16: return launch<DT_F16>(a, work);
    default: return launch<DT_BF16>(a, work);
  }
}

}  // namespace qmm
