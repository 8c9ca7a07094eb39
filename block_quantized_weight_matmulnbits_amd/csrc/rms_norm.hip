// rms_norm.hip -- root-mean-square norm with the residual's addition, and its
// output in 8 bits with scales, for the projection that comes next:
//   h = x + residual,  y = (h * i) * (weight + offset),
//   i = 1 / sqrt(mean(h^2) + eps),
// h in 32 bits, the mean and i in 64 bits (i then rounded to 32), each product
// rounded to 32 bits.  The statistic has bits to spare because codes hang on its
// last one: with it codes and scales are those of the definition bit for bit,
// whatever the order of the sum.  h and y leave rounded once; the codes are
// made of the unrounded y.  A scale is the block's maximum times the rounded
// reciprocal of the format's largest value: half a step of 32 bits beside the
// quotient.  An MX scale is the power of two at or below that, as
// qmm_lowp_quantize's is, which clips every block's maximum by up to a half; or, by
// the caller's choice, that of the Microscaling formats, at most twice as large,
// which clips by up to an eighth (normal y in E4M3 codes is off by 0.161 and 0.029,
// root mean square).
//
// Bound by HBM: x and the residual in, h and the codes out.  A row is read
// once and stays in registers, eight elements of a thread side by side, so that
// the blocks that share a scale are groups of neighbouring lanes and their
// maxima a few cross-lane steps.  Workgroups of a row's width go from row to row,
// the next one loaded ahead: 16384 rows of 4096 bf16 with residual and MX codes take
// 111 us (4.25 TB/s; 158 with a workgroup a row), 777 f32 rows of 5001 12.4 us (2.8 TB/s).
// One row takes 3.4 us on the device, of which most is the launch.
#include <algorithm>
#include <type_traits>

#include "decode.h"
#include "qmm_device.h"

namespace qmm {
namespace {

constexpr int CHUNK = 8;            // elements a thread holds side by side
constexpr int WIDEST_SHUFFLE = 64;  // lanes of a block whose maximum is shuffled

template <int DT>
__device__ __forceinline__ float element(const char* p, int64_t i) {
  return dt<DT>::to_f32(((const typename dt<DT>::T*)p)[i]);
}

// Elements [c, c + 8) of a row; zero past its end.  The vectors need no alignment
// but the element's (gfx950 reads and writes them at any address).
template <int DT> struct Chunk {
  typename dt<DT>::T e[CHUNK];
  __device__ __forceinline__ float operator[](int j) const { return dt<DT>::to_f32(e[j]); }
};
template <int DT>
__device__ __forceinline__ void load8(const char* row, int c, int cols, Chunk<DT>& v) {
  using T = typename dt<DT>::T;
  if (c + CHUNK <= cols) {
    __builtin_memcpy(v.e, (const T*)row + c, sizeof(v.e));
  } else {
#pragma unroll
    for (int j = 0; j < CHUNK; ++j) v.e[j] = c + j < cols ? ((const T*)row)[c + j] : T(0);
  }
}

template <int DT>
__device__ __forceinline__ void store8(char* row, int c, int cols, const float (&v)[CHUNK]) {
  using T = typename dt<DT>::T;
  T e[CHUNK];
#pragma unroll
  for (int j = 0; j < CHUNK; ++j) e[j] = dt<DT>::from_f32(v[j]);
  if (c + CHUNK <= cols) {
    __builtin_memcpy((T*)row + c, e, sizeof(e));
  } else {
#pragma unroll
    for (int j = 0; j < CHUNK; ++j)
      if (c + j < cols) ((T*)row)[c + j] = e[j];
  }
}

__device__ __forceinline__ void load_weight(const NormArgs& a, int c, float (&w)[CHUNK]) {
  auto take = [&](const auto& v) {
#pragma unroll
    for (int j = 0; j < CHUNK; ++j) w[j] = v[j];
  };
  if (a.weight == nullptr) {
#pragma unroll
    for (int j = 0; j < CHUNK; ++j) w[j] = 1.f;
  } else if (a.weight_dtype == DT_F32) {
    Chunk<DT_F32> v;
    load8<DT_F32>(a.weight, c, a.cols, v);
    take(v);
  } else if (a.weight_dtype == DT_F16) {
    Chunk<DT_F16> v;
    load8<DT_F16>(a.weight, c, a.cols, v);
    take(v);
  } else {
    Chunk<DT_BF16> v;
    load8<DT_BF16>(a.weight, c, a.cols, v);
    take(v);
  }
#pragma unroll
  for (int j = 0; j < CHUNK; ++j) w[j] += a.offset;
}

// Two FP8 codes (OCP E4M3 or E5M2): nearest, ties to even, saturating; a NaN is
// 0x7F, where there may be any.
__device__ __forceinline__ uint32_t fp8_pair(float x, float y, int format, bool odd) {
  const float most = format == 0 ? 448.f : 57344.f;
  const float a = __builtin_amdgcn_fmed3f(x, -most, most), b = __builtin_amdgcn_fmed3f(y, -most, most);
  uint32_t c = format == 0 ? __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false)
                           : __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false);
  c &= 0xFFFFu;
  if (odd) {
    if (x != x) c = (c & 0xFF00u) | 0x7Fu;
    if (y != y) c = (c & 0xFFu) | 0x7F00u;
  }
  return c;
}

// Sum over a wave by neighbour exchanges inside rows of 16, then over the rows.
__device__ __forceinline__ double wave_sum_f64(double v) {
  auto over = [&](auto ctrl, auto rows) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
    v += __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  };
  using std::integral_constant;
  over(integral_constant<int, 0xB1>{}, integral_constant<int, 0xF>{});    // quad_perm 1,0,3,2
  over(integral_constant<int, 0x4E>{}, integral_constant<int, 0xF>{});    // quad_perm 2,3,0,1
  over(integral_constant<int, 0x141>{}, integral_constant<int, 0xF>{});   // row_half_mirror
  over(integral_constant<int, 0x140>{}, integral_constant<int, 0xF>{});   // row_mirror
  over(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});   // row_bcast:15
  over(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});   // row_bcast:31
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// 1 / sqrt(x) to within a few of 64 bits: the hardware's estimate and two of
// Newton's steps.
__device__ __forceinline__ double rsqrt_f64(double x) {
  double r = __builtin_amdgcn_rsq(x);
  if (x > 0.0 && x < INFINITY) {
#pragma unroll
    for (int i = 0; i < 2; ++i) r = __builtin_fma(0.5 * r, __builtin_fma(-x * r, r, 1.0), r);
  }
  return r;
}

// The value of another lane of the same four (a DPP quad permutation).
template <int CTRL> __device__ __forceinline__ float neighbour(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}

// body(p) for each of a thread's pieces, unrolled where they are registers.
template <int NP, typename Body>
__device__ __forceinline__ void each_piece(int pieces, Body body) {
  if constexpr (NP > 0) {
#pragma unroll
    for (int p = 0; p < NP; ++p) body(p);
  } else {
    for (int p = 0; p < pieces; ++p) body(p);
  }
}

// KIND: the quant_kind, or none.  RT threads a row, NP chunks a thread in registers (0: rows too long for
// them are read again where needed).
template <int DT, int KIND, int RT, int NP>
__global__ __launch_bounds__(RT < 256 ? 256 : RT) void rms_norm_kernel(NormArgs a, double over_cols) {
  constexpr int ES = (int)sizeof(typename dt<DT>::T);
  constexpr int ROWS = RT < 256 ? 256 / RT : 1;
  constexpr int WAVES = RT / 64, HELD = NP > 0 ? NP : 1;
  __shared__ double sums[WAVES];
  __shared__ uint32_t tops[NP == 0 ? NORM_MAX_COLS / 1024 : RT * NP * CHUNK / 1024 + 1];
  const int t = threadIdx.x % RT, lane = threadIdx.x & 63, wave = t >> 6;
  // Chunks of the codes' row, which may be padded to whole blocks.
  const int chunks = ((KIND == QUANT_INT8 ? a.code_cols : a.cols) + CHUNK - 1) / CHUNK;
  const int pieces = NP > 0 ? NP : (chunks + RT - 1) / RT;
  const int log_block = 31 - __builtin_clz(a.block | 1);
  const bool wide = KIND == QUANT_INT8 && a.block > CHUNK * WIDEST_SHUFFLE;
  const int64_t first = (int64_t)blockIdx.x * ROWS + threadIdx.x / RT, apart = (int64_t)gridDim.x * ROWS;
  if (RT == 64 && first >= a.rows) return;

  // What is read of a row, as it is; weights are kept over the rows.
  Chunk<DT> x[HELD], r[HELD];
  auto load = [&](int64_t row, int p, Chunk<DT>& xe, Chunk<DT>& re) {
    const int c = (p * RT + t) * CHUNK;
    load8<DT>(a.x + row * a.x_stride * ES, c, a.cols, xe);
    if (a.residual) load8<DT>(a.residual + row * a.residual_stride * ES, c, a.cols, re);
  };
  auto add = [&](const Chunk<DT>& xe, const Chunk<DT>& re, float (&h)[CHUNK]) {
#pragma unroll
    for (int j = 0; j < CHUNK; ++j) h[j] = a.residual ? xe[j] + re[j] : xe[j];
  };
  float w[HELD][CHUNK];
  if constexpr (NP > 0) {
    each_piece<NP>(pieces, [&](int p) { load(first, p, x[p], r[p]); });
    each_piece<NP>(pieces, [&](int p) { load_weight(a, (p * RT + t) * CHUNK, w[p]); });
  }

  for (int64_t row = first; row < a.rows; row += apart) {
    float v[HELD][CHUNK];
    double ss = 0.0;
    each_piece<NP>(pieces, [&](int p) {
      float(&h)[CHUNK] = v[NP > 0 ? p : 0];
      if constexpr (NP == 0) load(row, p, x[0], r[0]);
      add(x[NP > 0 ? p : 0], r[NP > 0 ? p : 0], h);
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) ss = __builtin_fma((double)h[j], (double)h[j], ss);
    });
    // The next row is on its way while this one is written.
    if constexpr (NP > 0) {
      if (row + apart < a.rows) each_piece<NP>(pieces, [&](int p) { load(row + apart, p, x[p], r[p]); });
    }
    ss = wave_sum_f64(ss);
    if constexpr (WAVES > 1) {
      __syncthreads();               // the row before has been read
      if (lane == 0) sums[wave] = ss;
      if (wide)
        for (int b = t; b < a.blocks; b += RT) tops[b] = 0u;
      __syncthreads();
      ss = 0.0;
#pragma unroll
      for (int k = 0; k < WAVES; ++k) ss += sums[k];
    }
    const float inv = (float)rsqrt_f64(__builtin_fma(ss, over_cols, a.eps));

    // y of a piece; zero past the row's end.
    auto normed = [&](int p, float (&y)[CHUNK]) {
      const int c = (p * RT + t) * CHUNK;
      if constexpr (NP == 0) {
        load(row, p, x[0], r[0]);
        add(x[0], r[0], v[0]);
        load_weight(a, c, w[0]);
      }
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) y[j] = v[NP > 0 ? p : 0][j] * inv * w[NP > 0 ? p : 0][j];
      if (c + CHUNK > a.cols) {
#pragma unroll
        for (int j = 0; j < CHUNK; ++j) y[j] = c + j < a.cols ? y[j] : 0.f;
      }
    };
    // The largest magnitude, as the bits that order so, a NaN's above infinity's:
    // a code is a whole number, so that only the scale can say of a NaN.
    auto chunk_top = [&](const float (&y)[CHUNK]) {
      uint32_t m = 0u;
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) m = max(m, __float_as_uint(y[j]) & 0x7FFFFFFFu);
      return m;
    };
    if constexpr (WAVES > 1) {
      // Blocks that several waves share: their maxima meet in LDS.
      if (wide) {
        each_piece<NP>(pieces, [&](int p) {
          const int c = (p * RT + t) * CHUNK;
          float y[CHUNK];
          normed(p, y);
          if (c < a.code_cols) atomicMax(&tops[c >> log_block], chunk_top(y));
        });
        __syncthreads();
      }
    }

    each_piece<NP>(pieces, [&](int p) {
      const int c = (p * RT + t) * CHUNK;
      float y[CHUNK];
      normed(p, y);
      if (a.h) store8<DT>(a.h + row * a.h_stride * ES, c, a.cols, v[NP > 0 ? p : 0]);
      if (a.y) store8<DT>(a.y + row * a.y_stride * ES, c, a.cols, y);
      if constexpr (KIND == QUANT_NONE) return;
      uint32_t word[2] = {0u, 0u};
      if constexpr (KIND == QUANT_INT8) {
        uint32_t most = chunk_top(y);
        if (wide) {
          most = c < a.code_cols ? tops[c >> log_block] : 0u;
        } else {
          for (int o = 1; o < a.block / CHUNK; o <<= 1) most = max(most, (uint32_t)__shfl_xor((int)most, o));
        }
        const float s = __uint_as_float(most) * (1.f / 127.f);
        if (c < a.code_cols && (c & (a.block - 1)) == 0)
          ((float*)a.scales)[row * a.blocks + (c >> log_block)] = s;
        const bool coded = s > 0.f && s < INFINITY;
#pragma unroll
        for (int j = 0; j < CHUNK; ++j) {
          const float q = fminf(fmaxf(rintf(y[j] / s), -127.f), 127.f);
          word[j / 4] |= (coded ? (uint32_t)(int)q & 0xFFu : 0u) << (8 * (j % 4));
        }
      } else {
        float q[CHUNK];
        // A sum is NaN where one of its terms is (or infinities meet).
        float sum = 0.f;
        if constexpr (KIND == QUANT_MX) {
          float top = 0.f;                            // skips NaN, which has a code
#pragma unroll
          for (int j = 0; j < CHUNK; ++j) top = fmaxf(top, fabsf(y[j]));
          top = fmaxf(top, neighbour<0xB1>(top));     // four lanes a block
          top = fmaxf(top, neighbour<0x4E>(top));
          // The exponent of the scale that would put the maximum on the format's
          // (or on the power of two there); dividing by a power of two is exact.
          const float raw = top > 0.f ? top * a.top_factor : 1.f;
          const uint32_t e = (__float_as_uint(raw) >> 23) & 0xFFu;
          if (c < a.cols && c % 32 == 0)
            ((uint8_t*)a.scales)[row * a.blocks + c / 32] = (uint8_t)e;
          // e = 255 (an infinite maximum) is a NaN; e = 254 cannot be.
          const float back = __uint_as_float(e == 255u ? 0x7FC00000u : (254u - e) << 23);
#pragma unroll
          for (int j = 0; j < CHUNK; ++j) q[j] = y[j] * back;
        } else {
          const float s = *(const float*)a.scales;
#pragma unroll
          for (int j = 0; j < CHUNK; ++j) q[j] = s != 0.f ? y[j] / s : 0.f;
        }
#pragma unroll
        for (int j = 0; j < CHUNK; ++j) sum += q[j];
        const bool odd = __any(sum != sum);
#pragma unroll
        for (int j = 0; j < CHUNK; j += 2)
          word[j / 4] |= fp8_pair(q[j], q[j + 1], a.format, odd) << (8 * (j % 4));
      }
      uint8_t* to = a.codes + row * a.code_cols + c;
      if (c + CHUNK <= a.code_cols) {
        __builtin_memcpy(to, word, CHUNK);
      } else {
#pragma unroll
        for (int j = 0; j < CHUNK; ++j)
          if (c + j < a.code_cols) to[j] = (uint8_t)(word[j / 4] >> (8 * (j % 4)));
      }
    });
  }
}

template <int DT, int KIND, int RT, int NP>
hipError_t launch(const NormArgs& a) {
  constexpr int ROWS = RT < 256 ? 256 / RT : 1, THREADS = RT < 256 ? 256 : RT;
  // 2048 threads a compute unit, in workgroups that go from row to row.  Registers
  // hold fewer of them at once: three of 512 threads at 72, two of 768 at 68; the
  // others begin as these end.
  const int64_t groups = std::min<int64_t>((a.rows + ROWS - 1) / ROWS, 256 * 2048 / THREADS);
  rms_norm_kernel<DT, KIND, RT, NP><<<dim3((uint32_t)groups), THREADS, 0, a.stream>>>(a, 1.0 / a.cols);
  return hipGetLastError();
}

// A chunk a thread where a workgroup has as many.  Four do not fit the registers of
// 1024 threads (128): 512 bf16 rows of 32768 take 73 us with MX codes, as long as rows
// of 65536, which are read again.
template <int DT, int KIND>
hipError_t launch_size(const NormArgs& a) {
  const int chunks = ((KIND == QUANT_INT8 ? a.code_cols : a.cols) + CHUNK - 1) / CHUNK;
  if (chunks <= 64) return launch<DT, KIND, 64, 1>(a);
  if (chunks <= 256) return launch<DT, KIND, 256, 1>(a);
  if (chunks <= 512) return launch<DT, KIND, 512, 1>(a);
  if (chunks <= 768) return launch<DT, KIND, 768, 1>(a);
  if (chunks <= 1024) return launch<DT, KIND, 1024, 1>(a);
  if (chunks <= 2048) return launch<DT, KIND, 1024, 2>(a);
  if (chunks <= 4096) return launch<DT, KIND, 1024, 4>(a);
  return launch<DT, KIND, 1024, 0>(a);
}

template <int DT>
hipError_t launch_kind(const NormArgs& a) {
  switch (a.kind) {
    case QUANT_INT8: return launch_size<DT, QUANT_INT8>(a);
    case QUANT_MX: return launch_size<DT, QUANT_MX>(a);
    case QUANT_TENSOR: return launch_size<DT, QUANT_TENSOR>(a);
    default: return launch_size<DT, QUANT_NONE>(a);
  }
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a) {
  switch (a.dtype) {
    case DT_F32: return launch_kind<DT_F32>(a);
    case DT_F16: return launch_kind<DT_F16>(a);
    default: return launch_kind<DT_BF16>(a);
  }
}

}  // namespace qmm
