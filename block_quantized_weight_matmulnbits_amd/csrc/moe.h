// moe.h -- a layer of experts on block-quantized weights: the workspace, and the
// projection of every active expert's tokens (both projections of the layer).
//
// A workgroup takes 32 rows of one expert's weights (16 of the gate and the same
// 16 of the up projection, or 32 of the down projection) for all of the expert's
// tokens, up to 16 RT at a time; its four waves split K step by step (128 bytes of
// codes a row, a line of the caches) and join through LDS.  Weights are read once, straight into
// registers, 16 bytes a lane.  As many workgroups as are resident (three a compute
// unit, by the registers) go from item to item, and an item's first step is loaded
// while the one before it is joined: against a workgroup an item, one token over
// two experts took 52 us instead of 55, six of 64 narrow experts 68 instead of 72.
//
// HBM is the bound, at 0.81 of a large copy's rate where every weight of eight wide
// experts is read (hidden 4096, inter 14336, 16 tokens of f16, blocks of 32: up 135 us
// = 3.9 TB/s, down 75 us = 3.5), 0.7 for one token (29 us = 4.2 TB/s and 18 to 20 us
// = 3.2: 256 workgroups, whose beginning and end weigh more; K cut in three filled the
// chip and changed nothing), 0.5 for narrow ones (rows of 5 to 8 steps: two for
// a wave, so that joins and the wait for inputs show; 33 and 23 us).
//
// The matrix cores multiply x (an f32 one in three bf16 parts, h in two or three:
// a row each, so that few tokens fill the instruction's 16) with whole numbers,
// so that weights are not rounded, and a block's sum is scaled in fp32.  A 4-bit
// code c is the 16-bit value 16 + c (one shift and one and-or for two codes); what the 16 and the
// zero point add to a block's sum is (16 + z) times the sum of x over the block,
// which one more product, with ones, gives in the same registers:
//   out += s * (sum (16 + c) x  -  (16 + z) sum x).
// Those sums are up to some five times the result's size, which 16-bit types do
// not see; f32 layers, and 8-bit codes, for which the offset would be 256, enter
// as c - z.
// A lane loads 16 consecutive bytes, one block of 32 codes for example, but a
// matrix instruction takes 32 codes of one block from the four lanes that share
// a row, so their 32-bit words are transposed first (4 swaps for 4 instructions).
// x is laid out once in the order that the codes have then.
#pragma once

#include <algorithm>
#include <type_traits>

#include "decode.h"
#include "mfma_ops.h"
#include "qmm_device.h"

namespace qmm {

// An expert with tokens: its pairs are order[start .. start + count).  The ones
// with the most come first; entries without any have a count of 0.
struct MoeActive {
  int expert, start, count, unused;
};

// The workspace.  Pair p = token * top_k + j is a token's j-th expert.
struct MoeWork {
  int* ids;              // [pairs] experts, -1: none
  float* weights;        // [pairs]
  int* order;            // pairs by expert
  MoeActive* active;     // [max_active]
  uint16_t* x;           // [parts][tokens][hidden, padded]
  uint16_t* h;           // [parts][pairs][inter, padded]: what enters the down projection
  float* out;            // [pairs][hidden]: weighted outputs of the pairs
  int x_cols, h_cols;    // padded to 256 with zeros
  int max_active;        // active experts at most
};

// Parts that hold x (exactly: x itself, or three of bf16) and h (16 bits of it,
// or 24, in bf16, which has the range).
constexpr int moe_x_parts(int dtype) { return dtype == DT_F32 ? 3 : 1; }
constexpr int moe_h_parts(int dtype) { return dtype == DT_F32 ? 3 : 2; }

// One of the layer's two projections.
struct MoeSide {
  bool up;               // gate and up rows, to h; else the down projection, to out
  int tiles;             // workgroups an expert
  int parts, h_parts;    // of an input; of what goes to h
  const uint16_t* x;     // inputs: [parts][tokens or pairs][x_cols]
  int64_t x_part, h_part;  // elements of a part
  int x_cols;
};
// One instance file each: 16-bit inputs and 4-bit codes, offset; whole numbers.
hipError_t launch_moe_bf16(const MoeArgs& a, const MoeWork& w, const MoeSide& side);
hipError_t launch_moe_f16(const MoeArgs& a, const MoeWork& w, const MoeSide& side);
hipError_t launch_moe_whole4_bf16(const MoeArgs& a, const MoeWork& w, const MoeSide& side);
hipError_t launch_moe_whole8_bf16(const MoeArgs& a, const MoeWork& w, const MoeSide& side);
hipError_t launch_moe_whole8_f16(const MoeArgs& a, const MoeWork& w, const MoeSide& side);

// Whether weights enter the matrix cores as whole numbers c - z, or offset.
constexpr bool moe_whole(int bits, int dtype) { return bits == 8 || dtype == DT_F32; }
// Which of eight consecutive codes stands at place i of a matrix-core operand:
// offset ones are taken from both halves of a 32-bit word at once.
template <bool WHOLE> __host__ __device__ constexpr int code_at(int i) {
  return WHOLE ? i : i / 2 + 4 * (i % 2);
}
template <bool WHOLE> __device__ __forceinline__ int place_of_code(int k) {
  return WHOLE ? k : 2 * (k % 4) + k / 4;
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

constexpr int MOE_WAVES = 4, MOE_THREADS = 64 * MOE_WAVES;
// Workgroups of a compute unit, as far as registers go.
constexpr int moe_resident(int rt, int ns) { return rt == 1 && ns <= 8 ? 3 : 2; }

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

// Inputs of XDT (16-bit).  WHOLE: weights enter as c - z.  NS blocks a step of 128
// bytes (1 also where a block is longer).  RT tiles of 16 rows of inputs at once.
template <int XDT, int BITS, bool WHOLE, int SDT, bool ZP, int NS, int RT>
__global__ __launch_bounds__(MOE_THREADS, moe_resident(RT, NS)) void moe_project_kernel(
    MoeArgs a, MoeWork w, MoeSide side, int least, int most) {
  constexpr int CODES = 128 * 8 / BITS, UNITS = CODES / 32;  // a step's, 32 a unit
  constexpr int HALF = UNITS / 2;                            // units of 64 bytes
  constexpr int HALVES = NS == 2 * UNITS ? 2 : 1;            // blocks of 16: two a unit
  constexpr int PER = HALVES == 2 ? 1 : UNITS / NS;          // units a block
  constexpr bool EARLY = RT == 1;            // a step's inputs fit beside its weights
  constexpr int AHEAD = EARLY ? 2 : 0;       // units whose inputs are loaded a step ahead
  constexpr int S_WORDS = (NS * (SDT == DT_F32 ? 4 : 2) + 3) / 4;
  constexpr int Z_BYTES = (NS * BITS + 7) / 8, Z_WORDS = (Z_BYTES + 3) / 4;
  // 1 and 16 of XDT, twice, and the place of a code's lowest bit in 16 + code.
  constexpr uint32_t ONE = XDT == DT_BF16 ? 0x3F803F80u : 0x3C003C00u;
  constexpr uint32_t OFFSET = XDT == DT_BF16 ? 0x41804180u : 0x4C004C00u;
  constexpr int PLACE = XDT == DT_BF16 ? 3 : 6;
  using ST = typename dt<SDT>::T;
  using Op = MfmaOp<XDT>;
  using V8 = typename Op::V;

  const bool up = side.up;
  const MoeProj& m = up ? a.up : a.down;
  const int lane = threadIdx.x & 63, l15 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int width = up ? a.inter : a.hidden;   // outputs

  __shared__ float part_sum[MOE_WAVES][8][64];

  const uint32_t row_bytes = (uint32_t)m.row_bytes, zp_row_bytes = (uint32_t)m.zp_row_bytes;
  const int blocks = m.blocks;
  const int log_block = 31 - __builtin_clz(a.block);
  const int steps = (m.cols + CODES - 1) / CODES;
  const int whole_steps = min(row_bytes / 128u, (uint32_t)steps);
  const int parts = side.parts, fit = 16 / parts;   // tokens of a tile
  // Which eight of a unit's 32 codes a lane holds after the swaps.
  const int chunk = BITS == 4 ? g : (g >> 1) | (g & 1) << 1;
  const V8 ones = __builtin_bit_cast(V8, ONE * u32x4{1u, 1u, 1u, 1u});

  // Word i of the lane that loaded row l15's bytes from 16 g on; of any that loaded
  // the row.
  const int codes_from = (4 * l15 + g) * 4, row_from = 4 * l15 * 4;
  auto hand_on = [](int from, uint32_t v) { return (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v); };

  // An and-or takes one scalar operand at most.
  uint32_t mask = 0x000F000Fu << PLACE, offset = OFFSET;
  asm("" : "+s"(mask));
  asm("" : "+v"(offset));

  // The item at hand: 32 rows of an expert for its tokens from r0 on.
  const int items = side.tiles * w.max_active;
  int item = blockIdx.x, r0 = 0, start = 0, count = 0, n0 = 0;
  const char *codes = nullptr, *scales = nullptr, *zps = nullptr;
  uint32_t row[2];
  int x_pair[RT], x_at_part[RT], pair[RT];

  // The next item, r0 after the one at hand; false: there is none.
  auto enter = [&](int at_r0) {
    r0 = at_r0;
    if (r0 >= count) {
      if (count > 0) item += gridDim.x;
      r0 = 0;
      for (;; item += gridDim.x) {
        if (item >= items) return false;
        const MoeActive act = w.active[item / side.tiles];
        if (act.count == 0) return false;
        start = act.start;
        count = act.count;
        if (count < least || count > most) continue;
        n0 = item % side.tiles * (up ? 16 : 32);
        // The expert's weights (the host keeps their offsets below 2^31).  Four
        // neighbouring lanes load 64 bytes of a row side by side (lanes 16 apart, as
        // the matrix cores want them, are each a request of their own); LDS's crossbar
        // hands them on.  Rows past the last one are read as it and dropped.
        const int64_t first = (int64_t)act.expert * m.rows;
        codes = (const char*)m.codes + first * m.row_bytes;
        scales = m.scales + first * m.blocks * (int64_t)sizeof(ST);
        zps = (const char*)m.zp + first * m.zp_row_bytes;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          int n = n0 + lane / 4 + (up ? 0 : 16 * t);
          n = n < width ? n : width - 1;
          row[t] = up ? t * a.inter + n : n;
        }
        break;
      }
    }
    // A token takes a row for each of its parts.  Row r of a tile is place (r % 4) *
    // 4 + r / 4, so that the first places stand in the first of a lane's four
    // results; places beyond the last token repeat one of these.
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int place = (l15 % 4) * 4 + l15 / 4;
      auto there = [&](int at) { return at / parts < fit && r0 + rt * fit + at / parts < count; };
      // Neighbouring lanes ask for the same row where there are no more than four.
      const int at = there(place) ? place : there(l15 / 4) ? l15 / 4 : 0;
      const int j = there(at) ? r0 + rt * fit + at / parts : r0;
      x_at_part[rt] = there(at) ? at % parts : 0;
      x_pair[rt] = w.order[start + j];
      // The token that this thread sums up at the end.
      const int own = r0 + rt * fit + (int)(threadIdx.x >> 4);
      pair[rt] = w.order[start + (own < count ? own : r0)];
    }
    return true;
  };

    struct Inputs {
      u32x4 v[EARLY ? UNITS : 1][RT];
    };
    // A step's weights: two times 16 bytes of each row, its scales and zero points.
    struct Raw {
      u32x4 c[2][2];
      uint32_t s[2][S_WORDS], z[2][Z_WORDS];
    };
    // WHOLE_STEP: all of its blocks are the row's.  Nothing here goes by a branch,
    // which would have a wave wait for loads ahead with the ones that it needs.
    auto load = [&](int step, Raw& d, auto whole) {
      constexpr bool WHOLE_STEP = decltype(whole)::value;
      const int b0 = (step * CODES) >> log_block;
      const uint32_t byte = b0 * BITS / 8;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        // Codes past a row's end meet zeros of x: any will do.
        const uint32_t from = row[t] * row_bytes;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t at = step * 128 + 64 * k + 16 * (lane % 4);
          if constexpr (WHOLE_STEP) {
            __builtin_memcpy(&d.c[t][k], codes + (from + at), 16);
          } else if constexpr (BITS == 4 && HALVES == 2) {
            u32x2 lo, hi;
            __builtin_memcpy(&lo, codes + (from + min(at, row_bytes - 8)), 8);
            __builtin_memcpy(&hi, codes + (from + min(at + 8, row_bytes - 8)), 8);
            d.c[t][k] = u32x4{lo[0], lo[1], hi[0], hi[1]};
          } else {
            d.c[t][k] = *(const u32x4*)(codes + (from + min(at, row_bytes - 16)));
          }
        }
        const uint32_t s_from = row[t] * blocks;
        if constexpr (WHOLE_STEP) {
          d.s[t][0] = 0;
          __builtin_memcpy(d.s[t], scales + (s_from + b0) * (uint32_t)sizeof(ST), NS * sizeof(ST));
        } else {
#pragma unroll
          for (int k = 0; k < S_WORDS; ++k) d.s[t][k] = 0;
#pragma unroll
          for (int b = 0; b < NS; ++b) {
            uint32_t v = 0;
            __builtin_memcpy(&v, scales + (s_from + min(b0 + b, blocks - 1)) * (uint32_t)sizeof(ST), sizeof(ST));
            d.s[t][b * sizeof(ST) / 4] |= v << (8 * (b * sizeof(ST) % 4));
          }
        }
        if constexpr (ZP) {
          const uint32_t z_from = row[t] * zp_row_bytes;
#pragma unroll
          for (int k = 0; k < Z_WORDS; ++k) d.z[t][k] = 0;
          if constexpr (WHOLE_STEP) {
            __builtin_memcpy(d.z[t], zps + (z_from + byte), Z_BYTES);
          } else {
#pragma unroll
            for (int b = 0; b < Z_BYTES; ++b)
              d.z[t][b / 4] |= (uint32_t)(uint8_t)zps[z_from + min(byte + b, zp_row_bytes - 1)] << (8 * (b % 4));
          }
        }
      }
    };

    // An item's first step is on its way while the one before it is summed up.
    Raw d;
    // Opaque, or its addresses would be kept in registers over all items.
    int own = wave;
    asm volatile("" : "+s"(own));
    auto begin_item = [&](int at_r0) {
      if (!enter(at_r0)) return false;
      if (own < whole_steps) load(own, d, std::true_type{});
      return true;
    };

  for (bool more = begin_item(0); more;) {
    const uint16_t* x[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      x[rt] = side.x + x_at_part[rt] * side.x_part + (int64_t)(up ? x_pair[rt] / a.top_k : x_pair[rt]) * side.x_cols + 8 * chunk;

    f32x4 out[2][RT];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) out[t][rt] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto x_at = [&](int step, int u, int rt) { return *(const u32x4*)(x[rt] + step * CODES + 32 * u); };
    auto load_x = [&](int step, Inputs& in) {
#pragma unroll
      for (int u = AHEAD; u < UNITS; ++u)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) in.v[EARLY ? u : 0][rt] = x_at(step, u, rt);
    };
    auto load_x_ahead = [&](int step, Inputs& in) {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) in.v[EARLY ? u : 0][rt] = x_at(step, u, rt);
    };

    // RESULTS of a lane's four are wanted.
    auto compute = [&](int step, const Raw& d, const Inputs& in, auto results) {
      constexpr int RESULTS = decltype(results)::value;
      constexpr f32x4 ZERO = {0.f, 0.f, 0.f, 0.f};
      uint32_t c[2][4], sw[2][S_WORDS], zw[2][Z_WORDS];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int k = 0; k < S_WORDS; ++k) sw[t][k] = hand_on(row_from, d.s[t][k]);
        if constexpr (ZP) {
#pragma unroll
          for (int k = 0; k < Z_WORDS; ++k) zw[t][k] = hand_on(row_from, d.z[t][k]);
        }
      }
      auto zero_bits = [&](int t, int b) {
        const int odd = BITS == 4 && NS == 1 ? 4 * ((step * CODES) >> log_block & 1) : 0;
        return zw[t][b * BITS / 32] >> (BITS * b % 32 + odd) & ((1u << BITS) - 1u);
      };
      auto zero = [&](int t, int b) { return ZP ? (float)zero_bits(t, b) : (float)(1 << (BITS - 1)); };
      // 16 + z: a float of 16 whose last bit is 2^-19.
      auto zero_offset = [&](int t, int b) {
        return ZP ? __uint_as_float(zero_bits(t, b) << 19 | 0x41800000u) : 24.f;
      };
      // Eight of a unit's codes, as bf16.
      auto weights = [&](int t, int u) {
        u32x4 v;
        if constexpr (WHOLE) {
          float z = zero(t, HALVES == 2 ? 2 * u : u / PER);
          if constexpr (HALVES == 2) z = chunk >> 1 ? zero(t, 2 * u + 1) : z;
          const uint32_t word = c[t][BITS == 4 ? u % HALF : 2 * (u % HALF)];
          const uint32_t lo = BITS == 4 ? word & 0x0F0F0F0Fu : 0u, hi = BITS == 4 ? word >> 4 & 0x0F0F0F0Fu : 0u;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float p, q;
            if constexpr (BITS == 4) {
              p = (float)(lo >> (8 * i) & 255u);
              q = (float)(hi >> (8 * i) & 255u);
            } else {
              const uint32_t from = c[t][2 * (u % HALF) + i / 2] >> (16 * (i % 2));
              p = (float)(from & 255u);
              q = (float)(from >> 8 & 255u);
            }
            v[i] = Op::pack(p - z, q - z);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int left = PLACE - 4 * i;
            const uint32_t at = left >= 0 ? c[t][u % HALF] << (left & 31) : c[t][u % HALF] >> (-left & 31);
            v[i] = (at & mask) | offset;
          }
        }
        return __builtin_bit_cast(V8, v);
      };
      f32x4 acc[HALVES][2][RT], xs[HALVES][RT];
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        if (u % HALF == 0) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) c[t][i] = hand_on(codes_from, d.c[t][u / HALF][i]);
            swap_halves(c[t][0], c[t][2]);
            swap_halves(c[t][1], c[t][3]);
            if constexpr (BITS == 4) {
              swap_rows(c[t][0], c[t][1]);
              swap_rows(c[t][2], c[t][3]);
            }
          }
        }
        V8 wt[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) wt[t] = weights(t, u);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const u32x4 xv = EARLY ? in.v[EARLY ? u : 0][rt] : x_at(step, u, rt);
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            const u32x4 mine = HALVES == 1 || (chunk >> 1) == h ? xv : u32x4{0u, 0u, 0u, 0u};
            const V8 v = __builtin_bit_cast(V8, mine);
            const bool fresh = u % PER == 0;
            if constexpr (!WHOLE) xs[h][rt] = Op::run(v, ones, fresh ? ZERO : xs[h][rt]);
#pragma unroll
            for (int t = 0; t < 2; ++t) acc[h][t][rt] = Op::run(v, wt[t], fresh ? ZERO : acc[h][t][rt]);
          }
        }
        // Registers hold what one unit needs at a time.
        __builtin_amdgcn_sched_barrier(0);
        if ((u + 1) % PER != 0) continue;
        // The end of a block.
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int b = HALVES == 2 ? 2 * u + h : u / PER;
            const uint32_t raw = sw[t][b * sizeof(ST) / 4] >> (8 * (b * sizeof(ST) % 4));
            float s;
            if constexpr (SDT == DT_F32) s = __uint_as_float(raw);
            else s = bits16_to_f32<SDT>((uint16_t)raw);
            const float z = WHOLE ? 0.f : zero_offset(t, b);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
              for (int i = 0; i < RESULTS; ++i) {
                float v = acc[h][t][rt][i];
                if constexpr (!WHOLE) v = __builtin_fmaf(-z, xs[h][rt][i], v);
                out[t][rt][i] = __builtin_fmaf(s, v, out[t][rt][i]);
              }
          }
      }
    };

    auto walk = [&](auto results) {
      Inputs in;
      int step = own;
      if (step < whole_steps) {
        if constexpr (EARLY) load_x_ahead(step, in);
        for (; step + MOE_WAVES < whole_steps; step += MOE_WAVES) {
          // Loads are waited for in their order: inputs before weights ahead, and the
          // first inputs of a step before it, to cover for the others.
          Inputs next_in;
          if constexpr (EARLY) {
            load_x(step, in);
            __builtin_amdgcn_sched_barrier(0);
            load_x_ahead(step + MOE_WAVES, next_in);
          }
          __builtin_amdgcn_sched_barrier(0);
          Raw next;
          load(step + MOE_WAVES, next, std::true_type{});
          __builtin_amdgcn_sched_barrier(0);
          compute(step, d, in, results);
          d = next;
          if constexpr (EARLY) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) in.v[u][0] = next_in.v[u][0];
          }
        }
        if constexpr (EARLY) load_x(step, in);
        compute(step, d, in, results);
      }
      if (whole_steps < steps && wave == whole_steps % MOE_WAVES) {
        int last = whole_steps;
        asm volatile("" : "+s"(last));
        if constexpr (EARLY) {
          load_x_ahead(last, in);
          load_x(last, in);
        }
        load(last, d, std::false_type{});
        compute(last, d, in, results);
      }
    };
    const int places = (count - r0) * parts;
    if (RT == 1 && places <= 4) {
      walk(std::integral_constant<int, 1>{});
    } else if (RT == 1 && places <= 8) {
      walk(std::integral_constant<int, 2>{});
    } else {
      walk(std::integral_constant<int, 4>{});
    }

    // The sums' places and weights, before the next item's loads.
    const int from = r0, upto = count, at_n0 = n0;
    int to_pair[RT];
    float weight[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      to_pair[rt] = pair[rt];
      weight[rt] = up ? 0.f : w.weights[pair[rt]];
    }
    more = begin_item(r0 + fit * RT);

#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int first_token = from + rt * fit;
      if (first_token >= upto) break;
      __syncthreads();
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) part_sum[wave][4 * t + i][lane] = out[t][rt][i];
      __syncthreads();
      // This thread's sums: column l15 of both tiles for one token.
      const int j = threadIdx.x >> 4, n = at_n0 + l15;
      if (j >= fit || first_token + j >= upto) continue;
      float v[2] = {0.f, 0.f};
      for (int p = parts - 1; p >= 0; --p) {
        const int place = j * parts + p, at = place % 4 * 16 + l15;
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < MOE_WAVES; ++k) {
          s[0] += part_sum[k][place / 4][at];
          s[1] += part_sum[k][4 + place / 4][at];
        }
        v[0] += s[0];
        v[1] += s[1];
      }
      if (up) {
        float h = n < a.inter ? v[0] / (1.f + expf(-v[0])) * v[1] : 0.f;
        uint16_t* to = w.h + (int64_t)to_pair[rt] * w.h_cols + (n & ~7) + place_of_code<WHOLE>(n & 7);
        for (int p = 0; p < side.h_parts; ++p, to += side.h_part) {
          *to = MfmaOp<DT_BF16>::round(h);
          h -= bits16_to_f32<DT_BF16>(*to);
          // The last tile's pads the row with zeros.
          if (at_n0 + 16 >= width)
            for (int k = 16; at_n0 + k < w.h_cols; k += 16) to[k] = 0;
        }
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (n + 16 * t < a.hidden) w.out[(int64_t)to_pair[rt] * a.hidden + n + 16 * t] = v[t] * weight[rt];
      }
    }
  }
}

template <int XDT, int BITS, bool WHOLE, int SDT, bool ZP, int NS>
hipError_t launch_rows(const MoeArgs& a, const MoeWork& w, const MoeSide& side) {
  // Where an expert has more tokens than fit a tile of 16 rows, on the average,
  // the ones with so many are taken four tiles at a time; they come first among
  // the active ones, and are no more than `many`.  (For a few of them a tile after
  // another costs less than the launch.)  256 bf16 tokens over eight experts of 4096
  // x 14336, two each, take 1.41 ms so in blocks of 128, where sixteen calls of 16
  // take 3.1.  But with four blocks a step or more (of 64 and less in 4 bits, 16 in 8;
  // nearly all in f32 layers of 4 bits) the step's body is compiled as a call, whose
  // state goes through scratch memory: 23.3 ms in blocks of 32, and 4.4 for 64 tokens,
  // which four calls of 16 do in 0.9.
  const int fit = 16 / side.parts, pairs = a.tokens * a.top_k;
  const int many = pairs > fit * a.experts ? std::min(w.max_active, pairs / (fit + 1)) : 0;
  // As many workgroups as are resident, which go from item to item.
  auto grid = [&](int experts, int resident) { return dim3((uint32_t)std::min(side.tiles * experts, 256 * resident)); };
  if (many > 0)
    moe_project_kernel<XDT, BITS, WHOLE, SDT, ZP, NS, 4>
        <<<grid(many, moe_resident(4, NS)), MOE_THREADS, 0, a.stream>>>(a, w, side, fit + 1, INT32_MAX);
  moe_project_kernel<XDT, BITS, WHOLE, SDT, ZP, NS, 1>
      <<<grid(w.max_active, moe_resident(1, NS)), MOE_THREADS, 0, a.stream>>>(a, w, side, 1, many > 0 ? fit : INT32_MAX);
  return hipGetLastError();
}

template <int XDT, int BITS, bool WHOLE, int SDT, bool ZP>
hipError_t launch_blocks(const MoeArgs& a, const MoeWork& w, const MoeSide& side) {
  // Blocks of a step of 128 bytes.
  constexpr int CODES = 128 * 8 / BITS;
  switch (a.block) {
    case 16: return launch_rows<XDT, BITS, WHOLE, SDT, ZP, CODES / 16>(a, w, side);
    case 32: return launch_rows<XDT, BITS, WHOLE, SDT, ZP, CODES / 32>(a, w, side);
    case 64: return launch_rows<XDT, BITS, WHOLE, SDT, ZP, CODES / 64>(a, w, side);
    case 128: return launch_rows<XDT, BITS, WHOLE, SDT, ZP, CODES / 128>(a, w, side);
    default: return launch_rows<XDT, BITS, WHOLE, SDT, ZP, 1>(a, w, side);
  }
}

template <int XDT, int BITS, bool WHOLE>
hipError_t launch_moe_scales(const MoeArgs& a, const MoeWork& w, const MoeSide& side) {
  const bool zp = (side.up ? a.up : a.down).zp != nullptr;
  switch (a.s_dtype) {
    case DT_F32:
      return zp ? launch_blocks<XDT, BITS, WHOLE, DT_F32, true>(a, w, side)
                : launch_blocks<XDT, BITS, WHOLE, DT_F32, false>(a, w, side);
    case DT_F16:
      return zp ? launch_blocks<XDT, BITS, WHOLE, DT_F16, true>(a, w, side)
                : launch_blocks<XDT, BITS, WHOLE, DT_F16, false>(a, w, side);
    default:
      return zp ? launch_blocks<XDT, BITS, WHOLE, DT_BF16, true>(a, w, side)
                : launch_blocks<XDT, BITS, WHOLE, DT_BF16, false>(a, w, side);
  }
}

#endif  // __HIPCC__

}  // namespace qmm
