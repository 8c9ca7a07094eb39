// sample.hip -- the choice of the next token: logits, filtered by top-k, top-p
// and min-p, and a given number u in [0, 1) for each row.
//
// With w_i = exp((l_i - max l) / T), tokens ordered by logit (ties: the lowest
// index first): K = the first top_k; P = the shortest beginning of K that holds
// top_p of K's sum; of those, the ones with w_i >= min_p.  The token is the first
// one in the order of the indices whose running sum passes u times the whole.
//
// Nothing is sorted.  A threshold (the last token that is kept, as a key and an
// index) is found digit by digit, by counts for top-k and by sums for top-p, and
// the running sum by two passes of a row.  Sums decide which token a number
// falls on, so weights are formed in 64 bits and added as whole numbers, of
// which no order of addition changes a bit: w is held to 2^-SHIFT, SHIFT = 62 -
// log2(vocab) (45 bits for 131072 tokens).
#include "decode.h"
#include "qmm_device.h"

namespace qmm {
namespace {

constexpr int THREADS = 1024, WAVES = THREADS / 64;

// Orders as the values do; a NaN below all, so that it is never chosen, -0 as 0.
template <int DT>
__device__ __forceinline__ float logit(const char* row, int i) {
  const float v = dt<DT>::to_f32(((const typename dt<DT>::T*)row)[i]);
  return v != v ? -INFINITY : v;
}
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// exp(x) for x <= 0 in 64 bits: 2^n times a Taylor polynomial of 13 terms in
// |r| <= ln 2 / 2 (its rest is below 2^-54 of the value).  Where the result would
// leave the whole numbers' range it is 0.
__device__ __forceinline__ double exp_f64(double x) {
  if (!(x > -700.0)) return 0.0;
  const double n = rint(x * 1.4426950408889634074);
  // ln 2 in two parts, the first of 31 bits, so that n times it is exact.
  double r = __builtin_fma(n, -0x1.62e42ff000000p-1, x);
  r = __builtin_fma(n, 0x1.718432a1b0e26p-35, r);
  double p = 1.0 / 6227020800.0;
  p = __builtin_fma(p, r, 1.0 / 479001600.0);
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
  return ldexp(p, (int)n);
}

// A row's settings and the weight of its tokens.
struct Row {
  double top, over_t;    // the largest logit; the temperature
  int shift, k;
  double p, min_p, u;
  bool greedy;

  __device__ double weight(float l) const {
    // Infinite logits share everything equally.
    if (top == INFINITY) return l == INFINITY ? 1.0 : 0.0;
    return exp_f64(((double)l - top) / over_t);
  }
  __device__ uint64_t units(double w) const { return (uint64_t)rint(ldexp(w, shift)); }
};

__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

struct Shared {
  uint64_t sums[256];
  uint64_t waves[WAVES];
  uint64_t found, left;
  uint32_t digit;
  float top;
};

// A sum over the workgroup, for everybody.
__device__ uint64_t group_sum(Shared& s, uint64_t v) {
  v = wave_sum_u64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s.waves[threadIdx.x >> 6] = v;
  __syncthreads();
  uint64_t t = 0;
  for (int w = 0; w < WAVES; ++w) t += s.waves[w];
  return t;
}

// The place of a token in the order: larger first.
__device__ __forceinline__ uint64_t place_of(uint32_t key, int i) {
  return (uint64_t)key << 32 | (uint32_t)~i;
}

// The place of the last token of the shortest beginning of the order whose
// amounts reach `want`, among the places that are not below `from`; 0 where all
// of them together do not.  amount(i, place): 1, or the weight.
template <int DT, typename Amount>
__device__ uint64_t threshold(Shared& s, const char* row, int vocab, uint64_t from, uint64_t want,
                              Amount amount) {
  uint64_t prefix = 0;
  for (int bit = 56; bit >= 0; bit -= 8) {
    __syncthreads();
    if (threadIdx.x < 256) s.sums[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < vocab; i += THREADS) {
      const float l = logit<DT>(row, i);
      const uint64_t at = place_of(key_of(l), i);
      if (at < from || (bit < 56 && at >> (bit + 8) != prefix)) continue;
      const uint64_t n = amount(l);
      if (n) atomicAdd((unsigned long long*)&s.sums[at >> bit & 255], (unsigned long long)n);
    }
    __syncthreads();
    // The digit, from the largest down, at which the amounts reach `want`.
    if (threadIdx.x < 64) {
      uint64_t own = 0, four[4];
      for (int j = 0; j < 4; ++j) {
        four[j] = s.sums[255 - (threadIdx.x * 4 + j)];
        own += four[j];
      }
      uint64_t before = own;
      for (int o = 1; o < 64; o <<= 1) {
        const uint64_t v = __shfl_up(before, o);
        if ((int)threadIdx.x >= o) before += v;
      }
      const uint64_t all = __shfl(before, 63);
      before -= own;
      if (threadIdx.x == 0) {
        s.found = all >= want;
      }
      if (before < want && before + own >= want) {
        int j = 0;
        while (before + four[j] < want) before += four[j++];
        s.digit = 255 - (threadIdx.x * 4 + j);
        s.left = want - before;
      }
    }
    __syncthreads();
    if (!s.found) return 0;
    prefix = prefix << 8 | s.digit;
    want = s.left;
  }
  return prefix;
}

// One workgroup a row, which it reads again for every digit.
template <int DT>
__global__ __launch_bounds__(THREADS) void sample_row_kernel(SampleArgs a, int shift) {
  __shared__ Shared s;
  const int64_t row = blockIdx.x;
  const char* logits = a.logits + row * a.stride * (int64_t)sizeof(typename dt<DT>::T);
  const int vocab = a.vocab;

  uint32_t best = 0;
  for (int i = threadIdx.x; i < vocab; i += THREADS) {
    const uint32_t k = key_of(logit<DT>(logits, i));
    best = k > best ? k : best;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const uint32_t v = __shfl_xor(best, o);
    best = v > best ? v : best;
  }
  if ((threadIdx.x & 63) == 0) s.waves[threadIdx.x >> 6] = best;
  __syncthreads();
  for (int w = 0; w < WAVES; ++w) best = s.waves[w] > best ? (uint32_t)s.waves[w] : best;
  __syncthreads();

  Row r;
  r.top = value_of(best);
  const float t = a.temperature ? a.temperature[row] : 1.f;
  r.greedy = !(t > 0.f);
  r.over_t = r.greedy ? 1.0 : t;
  r.shift = shift;
  r.k = a.top_k ? a.top_k[row] : 0;
  if (r.k <= 0 || r.k > vocab) r.k = vocab;
  if (r.greedy) r.k = 1;
  const float p = a.top_p ? a.top_p[row] : 1.f, m = a.min_p ? a.min_p[row] : 0.f;
  r.p = p < 1.f ? (p > 0.f ? p : 0.0) : 1.0;
  r.min_p = m > 0.f ? (m < 1.f ? m : 1.0) : 0.0;
  r.u = a.uniform[row];
  if (r.top == -INFINITY) {
    // Nothing is left to choose from.
    if (threadIdx.x == 0) {
      a.tokens[row] = -1;
      if (a.logprobs) a.logprobs[row] = -INFINITY;
    }
    return;
  }

  uint64_t from = 0;
  if (r.k < vocab)
    from = threshold<DT>(s, logits, vocab, 0, r.k, [](float) { return (uint64_t)1; });
  auto units = [&](float l) { return r.units(r.weight(l)); };
  if (r.p < 1.0) {
    uint64_t sum = 0;
    for (int i = threadIdx.x; i < vocab; i += THREADS) {
      const float l = logit<DT>(logits, i);
      if (place_of(key_of(l), i) >= from) sum += units(l);
    }
    // A token is kept while the sum before it is below p times the whole: the
    // last one is where the sum reaches that.
    const double want = ceil(r.p * (double)group_sum(s, sum));
    const uint64_t at = threshold<DT>(s, logits, vocab, from, want < 1.0 ? 1 : (uint64_t)want, units);
    from = at > from ? at : from;
  }
  // Tokens that are kept, a run of the row for each wave.
  auto kept = [&](int i, double* w) {
    const float l = logit<DT>(logits, i);
    if (place_of(key_of(l), i) < from) return (uint64_t)0;
    *w = r.weight(l);
    return *w >= r.min_p ? r.units(*w) : 0;
  };
  const int run = (vocab + WAVES * 64 - 1) / (WAVES * 64) * 64, lane = threadIdx.x & 63,
            wave = threadIdx.x >> 6;
  const int begin = wave * run, end = begin + run < vocab ? begin + run : vocab;
  uint64_t sum = 0;
  double w;
  for (int i = begin + lane; i < end; i += 64) sum += kept(i, &w);
  const uint64_t total = group_sum(s, sum);
  const double target = fmin(fmax(r.u, 0.0), 1.0 - 0x1p-53) * (double)total;
  uint64_t before = 0;
  for (int v = 0; v < wave; ++v) before += s.waves[v];
  // The first token whose running sum passes the target lies in one wave's run.
  if (!((double)before <= target && (double)(before + s.waves[wave]) > target)) return;
  for (int i0 = begin; i0 < end; i0 += 64) {
    const int i = i0 + lane;
    const uint64_t own = i < end ? kept(i, &w) : 0;
    uint64_t upto = own;
    for (int o = 1; o < 64; o <<= 1) {
      const uint64_t v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    const uint64_t here = __ballot((double)(before + upto) > target);
    if (here) {
      if (lane == __builtin_ctzll(here)) {
        a.tokens[row] = i;
        if (a.logprobs) a.logprobs[row] = (float)(log(w) - log(ldexp((double)total, -shift)));
      }
      return;
    }
    before += __shfl(upto, 63);
  }
}

template <int DT>
hipError_t launch(const SampleArgs& a) {
  int shift = 62;
  while (((int64_t)1 << (62 - shift)) < a.vocab) --shift;
  sample_row_kernel<DT><<<dim3((uint32_t)a.rows), THREADS, 0, a.stream>>>(a, shift);
  return hipGetLastError();
}

}  // namespace

size_t sample_workspace_bytes(int64_t, int64_t) { return 256; }

hipError_t launch_sample(const SampleArgs& a, char*) {
  switch (a.dtype) {
    case DT_F32: return launch<DT_F32>(a);
    case DT_F16: return launch<DT_F16>(a);
    default: return launch<DT_BF16>(a);
  }
}

}  // namespace qmm
