// moe.h -- a layer of experts on block-quantized weights: the workspace, and the
// projection of every active expert's tokens (both projections of the layer).
//
// A workgroup takes 32 rows of one expert's weights (16 of the gate and the same
// 16 of the up projection, or 32 of the down projection) for all of the expert's
// tokens, 16 RT at a time; its eight waves split K step by step (64 bytes of
// codes a row) and join through LDS.  Weights are read once, straight into
// registers, 16 bytes a lane; HBM is the bound.
//
// The matrix cores multiply bf16 parts of x with whole codes, so that weights are
// not rounded: a 4-bit code c is the bf16 value 16 + c (one shift and one
// and-or for two codes), an 8-bit one two such fields.  What the 16 and the zero
// point add to a block's sum is (16 + z) times the sum of x over the block,
// which one more product, with ones, gives in the same registers; then the
// block's sum is scaled, in fp32:
//   out += s * (sum (16 + c) x  -  (16 + z) sum x).
// A lane loads 16 consecutive bytes, one block of 32 codes for example, but a
// matrix instruction takes 32 codes of one block from the four lanes that share
// a row, so their 32-bit words are transposed first (4 swaps for 4 instructions).
// x is laid out once in the order that the codes have then.
#pragma once

#include <type_traits>

#include "decode.h"
#include "mfma_ops.h"
#include "qmm_device.h"

namespace qmm {

// An expert with tokens: its pairs are order[start .. start + count).
struct MoeActive {
  int expert, start, count, unused;
};

// The workspace.  Pair p = token * top_k + j is a token's j-th expert.
struct MoeWork {
  int* ids;              // [pairs] experts, -1: none
  float* weights;        // [pairs]
  int* order;            // pairs by expert
  MoeActive* active;     // by the expert's number
  int* n_active;
  uint16_t* x;           // [parts][tokens][hidden, padded]: bf16 parts of x
  uint16_t* h;           // [parts][pairs][inter, padded]: what enters the down projection
  float* out;            // [pairs][hidden]: weighted outputs of the pairs
  int x_cols, h_cols;    // padded to 128 with zeros
  int max_active;        // active experts at most
};

// bf16 parts that hold x (exactly) and h (16 bits of it, 24 of an f32 layer's).
constexpr int moe_x_parts(int dtype) { return dtype == DT_BF16 ? 1 : dtype == DT_F16 ? 2 : 3; }
constexpr int moe_h_parts(int dtype) { return dtype == DT_F32 ? 3 : 2; }

// The projections' launchers, one instance file a number of parts.
hipError_t launch_moe_up_1(const MoeArgs& a, const MoeWork& w);
hipError_t launch_moe_up_2(const MoeArgs& a, const MoeWork& w);
hipError_t launch_moe_up_3(const MoeArgs& a, const MoeWork& w);
hipError_t launch_moe_down_2(const MoeArgs& a, const MoeWork& w);
hipError_t launch_moe_down_3(const MoeArgs& a, const MoeWork& w);

// Which of eight consecutive codes stands at place i of a matrix-core operand:
// fields of a 32-bit word are taken from both of its halves at once.
template <int BITS> __host__ __device__ constexpr int code_at(int i) {
  return BITS == 4 ? i / 2 + 4 * (i % 2) : (i & 4) + (i / 2 % 2) + 2 * (i % 2);
}
template <int BITS> __device__ __forceinline__ int place_of_code(int k) {
  return BITS == 4 ? 2 * (k % 4) + k / 4 : (k & 4) + 2 * (k % 2) + (k / 2 % 2);
}

// v as a sum of bf16 values, of 8 bits each.
template <int PARTS>
__device__ __forceinline__ void split_bf16(float v, uint16_t (&part)[PARTS]) {
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    part[p] = MfmaOp<DT_BF16>::round(v);
    v -= bits16_to_f32<DT_BF16>(part[p]);
  }
}

#ifdef __HIPCC__

constexpr int MOE_WAVES = 8, MOE_THREADS = 64 * MOE_WAVES;

__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap_rows(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// UP: gate and up rows, to h; else the down projection, to out.  PARTS bf16
// parts of the input.  NS blocks a step of 64 bytes (1 also where a block is
// longer).  RT tiles of 16 tokens at once.
template <bool UP, int BITS, int PARTS, int H_PARTS, int SDT, int NS, int RT>
__global__ __launch_bounds__(MOE_THREADS, RT == 1 ? 4 : 2) void moe_project_kernel(MoeArgs a, MoeWork w,
                                                                                  int tiles) {
  constexpr int CODES = 64 * 8 / BITS, UNITS = CODES / 32;   // a step's, 32 a unit
  constexpr int HALVES = BITS == 4 && NS == 8 ? 2 : BITS == 8 && NS == 4 ? 2 : 1;  // blocks of 16: two a unit
  constexpr int FIELDS = BITS / 4;
  constexpr float FIELD0 = BITS == 4 ? 16.f : 272.f;
  constexpr bool AHEAD = RT * PARTS <= 2;    // x is loaded a step ahead, too
  using ST = typename dt<SDT>::T;
  using V8 = typename MfmaOp<DT_BF16>::V;

  const int tile = blockIdx.x % tiles, number = blockIdx.x / tiles;
  if (number >= *w.n_active) return;
  const MoeActive act = w.active[number];
  const MoeProj& m = UP ? a.up : a.down;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l15 = lane & 15, g = lane >> 4;
  const int width = UP ? a.inter : a.hidden;   // outputs
  const int n0 = tile * (UP ? 16 : 32);

  __shared__ float part_sum[MOE_WAVES][8][64];
  __shared__ float total[8][64];

  // Rows of the weights; those past the last one are read as it and dropped.
  const uint8_t* codes[2];
  const ST* scales[2];
  const uint8_t* zps[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    int n = n0 + l15 + (UP ? 0 : 16 * t);
    n = n < width ? n : width - 1;
    const int64_t row = (int64_t)act.expert * m.rows + (UP ? t * a.inter + n : n);
    codes[t] = m.codes + row * m.row_bytes;
    scales[t] = (const ST*)m.scales + row * m.blocks;
    zps[t] = m.zp ? m.zp + row * m.zp_row_bytes : nullptr;
  }
  const int row_bytes = (int)m.row_bytes, blocks = m.blocks;
  const int log_block = 31 - __builtin_clz(a.block);
  const int steps = (m.cols + CODES - 1) / CODES;
  const int x_cols = UP ? w.x_cols : w.h_cols;
  const int64_t x_part = (int64_t)(UP ? a.tokens : a.tokens * a.top_k) * x_cols;
  // Which eight of a unit's 32 codes a lane holds after the swaps.
  const int chunk = BITS == 4 ? g : (g >> 1) | (g & 1) << 1;
  const V8 ones = __builtin_bit_cast(V8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});

  for (int r0 = 0; r0 < act.count; r0 += 16 * RT) {
    // Row r of a tile is token (r % 4) * 4 + r / 4, so that up to four tokens
    // stand in the first of a lane's four results.
    const uint16_t* x[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      int j = r0 + 16 * rt + (l15 % 4) * 4 + l15 / 4;
      j = j < act.count ? j : r0;
      const int pair = w.order[act.start + j];
      x[rt] = (UP ? w.x + (int64_t)(pair / a.top_k) * x_cols : w.h + (int64_t)pair * x_cols) + 8 * chunk;
    }

    auto load_x = [&](int step, int unit, int rt, int p) {
      return *(const u32x4*)(x[rt] + p * x_part + step * CODES + 32 * unit);
    };
    struct Raw {
      u32x4 c[2];
      ST s[2][NS];
      uint32_t z[2];
      u32x4 x[AHEAD ? RT : 1][AHEAD ? PARTS : 1][AHEAD ? UNITS : 1];
    };
    auto load = [&](int step, Raw& d) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        // Codes past a row's end meet zeros of x: any will do.
        const int at = step * 64 + 16 * g;
        if constexpr (BITS == 4 && NS == 8) {
          u32x2 lo, hi;
          __builtin_memcpy(&lo, codes[t] + (at < row_bytes - 8 ? at : row_bytes - 8), 8);
          __builtin_memcpy(&hi, codes[t] + (at + 8 < row_bytes - 8 ? at + 8 : row_bytes - 8), 8);
          d.c[t] = u32x4{lo[0], lo[1], hi[0], hi[1]};
        } else {
          d.c[t] = *(const u32x4*)(codes[t] + (at < row_bytes - 16 ? at : row_bytes - 16));
        }
        const int b0 = (step * CODES) >> log_block;
        if (NS == 1 || b0 + NS <= blocks) {
          __builtin_memcpy(d.s[t], scales[t] + b0, sizeof(d.s[t]));
        } else {
#pragma unroll
          for (int b = 0; b < NS; ++b) d.s[t][b] = scales[t][b0 + b < blocks ? b0 + b : blocks - 1];
        }
        if (m.zp) {
          if constexpr (NS * BITS <= 8) {
            const int byte = BITS == 4 ? b0 >> 1 : b0;
            d.z[t] = zps[t][byte];
            if (BITS == 4 && NS == 1) d.z[t] >>= 4 * (b0 & 1);
          } else if (b0 + NS <= blocks) {
            d.z[t] = 0;
            __builtin_memcpy(&d.z[t], zps[t] + b0 * BITS / 8, NS * BITS / 8);
          } else {
            d.z[t] = 0;
            const int last = (int)m.zp_row_bytes - 1;
#pragma unroll
            for (int b = 0; b < NS * BITS / 8; ++b) {
              const int byte = b0 * BITS / 8 + b;
              d.z[t] |= (uint32_t)zps[t][byte < last ? byte : last] << (8 * b);
            }
          }
        }
      }
      if constexpr (AHEAD) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int p = 0; p < PARTS; ++p)
#pragma unroll
            for (int u = 0; u < UNITS; ++u) d.x[rt][p][u] = load_x(step, u, rt, p);
      }
    };

    f32x4 out[2][RT];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) out[t][rt] = f32x4{0.f, 0.f, 0.f, 0.f};

    // RESULTS of a lane's four are wanted.
    auto compute = [&](int step, Raw& d, auto results) {
      constexpr int RESULTS = decltype(results)::value;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint32_t c[4] = {d.c[t][0], d.c[t][1], d.c[t][2], d.c[t][3]};
        swap_halves(c[0], c[2]);
        swap_halves(c[1], c[3]);
        if constexpr (BITS == 4) {
          swap_rows(c[0], c[1]);
          swap_rows(c[2], c[3]);
        }
        d.c[t] = u32x4{c[0], c[1], c[2], c[3]};
      }
      constexpr f32x4 ZERO = {0.f, 0.f, 0.f, 0.f};
      constexpr int PER = HALVES == 2 ? 1 : UNITS / NS;    // units a block
      f32x4 acc[HALVES][2][FIELDS][RT], xs[HALVES][RT];
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        V8 wt[2][FIELDS];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int f = 0; f < FIELDS; ++f) {
            u32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // Codes at bits 3 .. 6 of each half: 16 + code in bf16.
              const uint32_t word = BITS == 4 ? d.c[t][u] : d.c[t][2 * u + i / 2];
              const int right = BITS == 4 ? 4 * i - 3 : 8 * (i % 2) + 4 * f - 3;
              const uint32_t at = right < 0 ? word << -right : word >> right;
              v[i] = (at & 0x00780078u) | 0x41804180u;
            }
            wt[t][f] = __builtin_bit_cast(V8, v);
          }
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            u32x4 xv;
            if constexpr (AHEAD) xv = d.x[rt][p][u];
            else xv = load_x(step, u, rt, p);
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
              const u32x4 mine = HALVES == 1 || (chunk >> 1) == h ? xv : u32x4{0u, 0u, 0u, 0u};
              const V8 v = __builtin_bit_cast(V8, mine);
              const bool fresh = (HALVES == 2 || u % PER == 0) && p == 0;
              xs[h][rt] = MfmaOp<DT_BF16>::run(v, ones, fresh ? ZERO : xs[h][rt]);
#pragma unroll
              for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int f = 0; f < FIELDS; ++f)
                  acc[h][t][f][rt] = MfmaOp<DT_BF16>::run(v, wt[t][f], fresh ? ZERO : acc[h][t][f][rt]);
            }
          }
        if (HALVES == 1 && (u + 1) % PER != 0) continue;
        // The end of a block.
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int b = HALVES == 2 ? 2 * u + h : u / PER;
            const float s = dt<SDT>::to_f32(d.s[t][b]);
            const float z = FIELD0 + (m.zp ? (float)(d.z[t] >> (BITS * b) & ((1u << BITS) - 1u))
                                           : (float)(1 << (BITS - 1)));
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
              for (int i = 0; i < RESULTS; ++i) {
                float v = acc[h][t][0][rt][i];
                if constexpr (FIELDS == 2) v = __builtin_fmaf(16.f, acc[h][t][FIELDS - 1][rt][i], v);
                v = __builtin_fmaf(-z, xs[h][rt][i], v);
                out[t][rt][i] = __builtin_fmaf(s, v, out[t][rt][i]);
              }
          }
      }
    };

    auto walk = [&](auto results) {
      Raw d, next;
      int step = wave;
      if (step < steps) load(step, d);
      for (; step < steps; step += MOE_WAVES) {
        if (step + MOE_WAVES < steps) load(step + MOE_WAVES, next);
        compute(step, d, results);
        d = next;
      }
    };
    if (UP && n0 >= width) {
      // Beyond the last column: zeros, which pad h.
    } else if (RT == 1 && act.count - r0 <= 4) {
      walk(std::integral_constant<int, 1>{});
    } else {
      walk(std::integral_constant<int, 4>{});
    }

#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (r0 + 16 * rt >= act.count) break;
      __syncthreads();
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) part_sum[wave][4 * t + i][lane] = out[t][rt][i];
      __syncthreads();
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < MOE_WAVES; ++k) v += part_sum[k][wave][lane];
      // This thread's sum: tile wave / 4, result wave % 4.
      const int j = r0 + 16 * rt + (wave % 4) * 4 + g;
      const int n = n0 + l15 + (UP ? 0 : 16 * (wave / 4));
      if constexpr (UP) {
        total[wave][lane] = v;
        __syncthreads();
        if (wave < 4 && j < act.count && n < w.h_cols) {
          const float up = total[4 + wave][lane];
          const float h = n < a.inter ? v / (1.f + expf(-v)) * up : 0.f;
          uint16_t part[H_PARTS];
          split_bf16<H_PARTS>(h, part);
          const int64_t pair = w.order[act.start + j];
#pragma unroll
          for (int p = 0; p < H_PARTS; ++p)
            w.h[((int64_t)p * a.tokens * a.top_k + pair) * w.h_cols + (n & ~7) + place_of_code<BITS>(n & 7)] =
                part[p];
        }
      } else if (j < act.count && n < a.hidden) {
        const int pair = w.order[act.start + j];
        w.out[(int64_t)pair * a.hidden + n] = v * w.weights[pair];
      }
    }
  }
}

template <bool UP, int BITS, int PARTS, int H_PARTS, int SDT, int NS>
hipError_t launch_rows(const MoeArgs& a, const MoeWork& w) {
  const int tiles = UP ? w.h_cols / 16 : (a.hidden + 31) / 32;
  const dim3 grid((uint32_t)tiles * w.max_active);
  if (a.tokens <= 16) moe_project_kernel<UP, BITS, PARTS, H_PARTS, SDT, NS, 1><<<grid, MOE_THREADS, 0, a.stream>>>(a, w, tiles);
  else if (a.tokens <= 32) moe_project_kernel<UP, BITS, PARTS, H_PARTS, SDT, NS, 2><<<grid, MOE_THREADS, 0, a.stream>>>(a, w, tiles);
  else moe_project_kernel<UP, BITS, PARTS, H_PARTS, SDT, NS, 4><<<grid, MOE_THREADS, 0, a.stream>>>(a, w, tiles);
  return hipGetLastError();
}

template <bool UP, int PARTS, int H_PARTS, int SDT>
hipError_t launch_blocks(const MoeArgs& a, const MoeWork& w) {
  if (a.bits == 4) {
    if (a.block == 16) return launch_rows<UP, 4, PARTS, H_PARTS, SDT, 8>(a, w);
    if (a.block == 32) return launch_rows<UP, 4, PARTS, H_PARTS, SDT, 4>(a, w);
    if (a.block == 64) return launch_rows<UP, 4, PARTS, H_PARTS, SDT, 2>(a, w);
    return launch_rows<UP, 4, PARTS, H_PARTS, SDT, 1>(a, w);
  }
  if (a.block == 16) return launch_rows<UP, 8, PARTS, H_PARTS, SDT, 4>(a, w);
  if (a.block == 32) return launch_rows<UP, 8, PARTS, H_PARTS, SDT, 2>(a, w);
  return launch_rows<UP, 8, PARTS, H_PARTS, SDT, 1>(a, w);
}

template <bool UP, int PARTS, int H_PARTS>
hipError_t launch_moe_project(const MoeArgs& a, const MoeWork& w) {
  switch (a.s_dtype) {
    case DT_F32: return launch_blocks<UP, PARTS, H_PARTS, DT_F32>(a, w);
    case DT_F16: return launch_blocks<UP, PARTS, H_PARTS, DT_F16>(a, w);
    default: return launch_blocks<UP, PARTS, H_PARTS, DT_BF16>(a, w);
  }
}

#endif  // __HIPCC__

}  // namespace qmm
