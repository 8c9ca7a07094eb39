// paged_attn_tile.h -- attention of many new tokens over a paged cache, for
// 16-bit types: the bound is the matrix cores.
//
// A workgroup of four or eight waves takes 128 or 256 query rows (new tokens
// times the heads of a group, packed) of one key/value head; every wave owns 32
// of them from the first key to the last and keeps their queries, running
// statistics and outputs in registers.  Keys come in steps of 32.  A step's
// three parts have nothing to wait for in one another: the scores of the next
// step (matrix cores), the exponentials of this one (vector units) and the
// product of the last one's probabilities with V (matrix cores).
//
// 4096 new tokens after 12288 cached ones (32 heads of 128 over 8, bf16): 884 to
// 940 us by the card, 1020 to 1090 TFLOP/s, where a large matrix product reaches
// 1290 (with a sequence's first tiles first 4 % more: the last ones, which see the
// most keys, are then the end of the launch).  At 940 us the matrix cores are
// busy 0.54 of the time at 1.81 GHz: the chip lowers its clock under the load
// (128 workgroups instead of 256 run at 2.15 GHz), so what is left is energy,
// most of it in LDS reads and exponentials.
//
// The last workgroups of a launch take the sequences with few rows, as the rows
// kernel does: they fill the compute units that the tiles leave (three chunks
// of 509 tokens and six single ones, tiles whole: 258 us in two launches, 246
// in one, 270 with the few rows first).
//
// K and V pass through LDS in groups of two steps, two groups of each: the
// global loads of a group are in flight for a whole group's work before they
// are written to LDS.  Rows are padded there (K by 16 bytes, V to an odd
// multiple of 64) so that the 16-byte operand reads of K and the transposing
// reads of V meet no bank twice (measured: no conflict; with V padded by 32
// bytes a quarter of the LDS cycles were).  V is one group behind K, as its use is.
#pragma once

#include "paged_attn.h"
#include "paged_attn_rows.h"
#include "qmm_internal.h"

namespace qmm {

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int DT> struct Mfma32;
template <> struct Mfma32<DT_BF16> {
  static __device__ __forceinline__ f32x16 run(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
template <> struct Mfma32<DT_F16> {
  static __device__ __forceinline__ f32x16 run(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};

// Maximum and sum over the two lanes that share a column (lane mod 32).
__device__ __forceinline__ float pair_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float pair_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Minimum over the wave: turns among 16 lanes, then rows of 16 exchanged.
__device__ __forceinline__ float wave_min(float v) {
#define QMM_TURN(N)                                                                              \
  v = fminf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), 0x120 + (N), \
                                                           0xF, 0xF, true)));
  QMM_TURN(1) QMM_TURN(2) QMM_TURN(4) QMM_TURN(8)
#undef QMM_TURN
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fminf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  return -pair_max(-v);
}

// DK: the head's width in scores (16s), DV: in outputs (32s).
template <int DK, int DV> struct TileLds {
  static constexpr int KROW = DK * 2 + 16, VROW = DV * 2 + (DV % 64 == 32 ? 0 : 64);
  static constexpr int KBUF = 64 * KROW, VBUF = 64 * VROW;
  static constexpr int BYTES = 2 * (KBUF + VBUF);
};

// The statistics rise above the reference maximum by at most this (log2)
// before outputs are rescaled to a new one: probabilities stay below 2^slack.
// What f16 has left of its range keeps the small ones (prob_shift): with 4 those
// of 2^-25 and more keep all their bits (4096 new tokens over 16384 keys: 1012 us
// without a shift, 1019 with a slack of 8, 1023 of 4, 1033 of 2).
template <int DT> constexpr int tile_slack() { return DT == DT_F16 ? 4 : 8; }

template <int DT, int DK, int DV, int WAVES, bool CAP>
__global__ __launch_bounds__(64 * WAVES, DV <= 128 ? 2 : 1) void attn_tile_kernel(
    AttnArgs a, TilePlan plan, RowsPlan few, ScoreScale scale) {
  using T = typename dt<DT>::T;
  using L = TileLds<DK, DV>;
  using Op = MfmaOp<DT>;
  constexpr int KS = DK / 16, DB = DV / 32, CH = DK / 8;   // score steps, output blocks, chunks
  // Blocks of 32 rows a wave.  Two halve the LDS reads, but their registers
  // leave a SIMD one wave, and nothing to run while it waits (1007 us, not 930).
  constexpr int NQ = 1;
  constexpr int SR = 64 / WAVES, IT = (SR * CH + 63) / 64;   // rows of a group that a wave loads
  constexpr int THREADS = 64 * WAVES, ROWS = 32 * NQ * WAVES;
  constexpr int SLACK = tile_slack<DT>(), SHIFT = prob_shift<DT>(SLACK);   // of sums and outputs
  constexpr float DOWN = exp2_of(-SHIFT);
  constexpr int FEW = DV;   // the width that the few-row workgroups pad to
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  __shared__ int found[8];
  __shared__ int odd;

  const CacheArgs& c = a.c;
  const uint32_t groups = (uint32_t)plan.tiles * c.kv_heads;
  if (blockIdx.x >= groups) {
    attn_rows<DT, FEW, 1, WAVES, CAP>(a, few, scale, plan.skip_upto, blockIdx.x - groups, lds);
    return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l31 = lane & 31, half = lane >> 5, l15 = lane & 15;

  // Heads fastest, so that one head's tiles meet in one L2; then the parts of
  // the sequences' tiles, which follow one another without gaps.  A sequence's
  // last tiles see the most keys and come first.
  const int kvh = blockIdx.x % c.kv_heads, want = blockIdx.x / c.kv_heads;
  if (wave == 0) {
    struct Job {
      Seq q;
      int tiles;
      uint32_t keys;   // that a tile sees at most
    };
    auto job_of = [&](int s) QMM_INLINE {
      Job j{};
      if (s >= c.seqs) return j;
      j.q = seq_of(c, s);
      if (j.q.n <= plan.skip_upto) return j;
      j.tiles = (j.q.n * a.group + ROWS - 1) / ROWS;
      j.keys = j.q.len < 1 ? 1 : j.q.len;
      const uint32_t most = (uint32_t)a.window + ROWS / a.group + 1;
      if (a.window && a.causal && j.keys > most) j.keys = most;
      return j;
    };
    const Job job = job_of(lane);
    auto jobs_at = [&](int s0) QMM_INLINE { return s0 == 0 ? job : job_of(s0 + lane); };
    auto parts_in = [](uint32_t keys, uint32_t n) { return (keys - 1) / n + 1; };
    // Parts of about 1 / rate keys: the same number wherever it is asked for.
    auto parts_at = [](uint32_t keys, float rate) {
      return max(1u, (uint32_t)ceilf((float)keys * rate));
    };
    // Every lane prices one length of parts, 7 % below its neighbour's, in keys
    // of one workgroup's time: the longest part where all are resident at
    // once, or else an equal share of all and half a part of waste at the end.
    // (One sequence alone: as many as the host found.)
    float rate = 0.f;
    if (plan.splits > 1 && c.seqs > 1) {
      uint32_t most = 1;
      for (int s0 = 0; s0 < c.seqs; s0 += 64) {
        const Job j = jobs_at(s0);
        for (uint64_t rest = __ballot(j.tiles > 0); rest; rest &= rest - 1)
          most = max(most, (uint32_t)__builtin_amdgcn_readlane(j.keys, __builtin_ctzll(rest)));
      }
      const float mine = exp2_fast(0.1f * lane) / (float)most;
      uint32_t units = 0;
      float keys = 0.f, part = 0.f;
      for (int s0 = 0; s0 < c.seqs; s0 += 64) {
        const Job j = jobs_at(s0);
        for (uint64_t rest = __ballot(j.tiles > 0); rest; rest &= rest - 1) {
          const int w = __builtin_ctzll(rest);
          const uint32_t t = __builtin_amdgcn_readlane(j.tiles, w);
          const uint32_t k = __builtin_amdgcn_readlane(j.keys, w), n = parts_at(k, mine);
          units += t * n;
          part = fmaxf(part, (float)k * __builtin_amdgcn_rcpf((float)n));
          keys += (float)t * (float)k;
        }
      }
      const uint32_t longest = parts_at(most, mine);
      const float full = (float)units / plan.room;
      const float cost = PART_OWN + (longest == 1 ? 0.f : PART_JOIN + PART_PARK * fminf(full, 1.f));
      float price = full <= 1.f ? part + cost : keys / plan.room + full * cost + 0.5f * part;
      if (longest > (uint32_t)plan.splits || units > (uint32_t)plan.tiles) price = INFINITY;
      const float best = wave_min(price);
      const uint64_t who = __ballot(price == best && price < INFINITY);
      if (who) rate = __shfl(mine, __builtin_ctzll(who));
    }
    int base = 0, seq = -1;
    for (int s0 = 0; s0 < c.seqs && seq < 0; s0 += 64) {
      const Job j = jobs_at(s0);
      const int parts = c.seqs == 1 ? plan.splits : parts_at(j.keys, rate), mine = j.tiles * parts;
      int sum = mine;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(sum, d);
        if (lane >= d) sum += y;
      }
      const int first = base + sum - mine;
      const uint64_t who = __ballot(want >= first && want < first + mine);
      if (who) {
        seq = s0 + __builtin_ctzll(who);
        if (lane == __builtin_ctzll(who)) {
          // Parts are turned by the tile's number, as in the rows kernel.
          const int turn = (want - first) / parts;
          found[1] = j.tiles - 1 - turn;
          found[2] = j.q.t0;
          found[3] = j.q.n;
          found[4] = j.q.len;
          found[5] = (want - first + turn) % parts;
          found[6] = parts;
          found[7] = parts_in(parts_in(j.keys, parts), 64) * 64;
        }
      }
      base += __shfl(sum, 63);
    }
    if (lane == 0) {
      found[0] = seq;
      odd = 0;
    }
  }
  __syncthreads();
  const int seq = __builtin_amdgcn_readfirstlane(found[0]);
  if (seq < 0) return;
  const int tile = __builtin_amdgcn_readfirstlane(found[1]);
  const Seq sq{__builtin_amdgcn_readfirstlane(found[2]), __builtin_amdgcn_readfirstlane(found[3]),
               __builtin_amdgcn_readfirstlane(found[4])};
  const int split = __builtin_amdgcn_readfirstlane(found[5]);
  const int parts = __builtin_amdgcn_readfirstlane(found[6]);
  const uint32_t chunk = __builtin_amdgcn_readfirstlane(found[7]);
  const int rows = sq.n * a.group, row0 = tile * ROWS;
  const int row1 = rows < row0 + ROWS ? rows : row0 + ROWS;
  const int pos0 = sq.len - sq.n;
  auto clip = [&](int j) { return j < 0 ? 0 : j > sq.len ? sq.len : j; };
  auto pos_of = [&](int r) { return pos0 + (int)div_by(r, a.by_group); };
  const int kmin = a.window ? clip(pos_of(row0) - a.window + 1) : 0;
  const int kmax = a.causal ? clip(pos_of(row1 - 1) + 1) : sq.len;
  int active = kmax > kmin ? (int)(((uint32_t)(kmax - kmin) - 1) / chunk + 1) : 1;
  active = active > parts ? parts : active;
  if (split >= active) return;
  const int begin = kmin + split * chunk;
  const int end = split == active - 1 ? kmax : begin + chunk;
  const int steps = end > begin ? (end - begin + 31) / 32 : 0;

  // The wave's rows: what all of them see, and each lane's own limits.
  const int wrow0 = row0 + wave * 32 * NQ;
  int all0 = begin, all1 = end;
  if (wrow0 < row1) {
    const int wrow1 = row1 < wrow0 + 32 * NQ ? row1 : wrow0 + 32 * NQ;
    if (a.window) all0 = max(all0, pos_of(wrow1 - 1) - a.window + 1);
    if (a.causal) all1 = min(all1, clip(pos_of(wrow0) + 1));
  }
  all0 = __builtin_amdgcn_readfirstlane(all0);
  all1 = __builtin_amdgcn_readfirstlane(all1);

  u32x4 qf[NQ][KS];
  int lo[NQ], hi[NQ];
#pragma unroll
  for (int b = 0; b < NQ; ++b) {
    const int r = wrow0 + 32 * b + l31;
    const bool ok = r < row1;
    const int i = ok ? (int)div_by(r, a.by_group) : 0, h = ok ? r - i * a.group : 0;
    const int pos = pos0 + i;
    lo[b] = max(begin, a.window ? pos - a.window + 1 : 0);
    hi[b] = !ok ? 0 : min(end, a.causal ? clip(pos + 1) : sq.len);
    const T* from = (const T*)a.q + (int64_t)(sq.t0 + i) * a.q_token +
                    (int64_t)(kvh * a.group + h) * a.q_head;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = (2 * s + half) * 8;
      T e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = T(0);
      if (ok && d < c.dim) {
        if (a.q_wide) {
          __builtin_memcpy(e, __builtin_assume_aligned(from + d, 16), 16);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j] = from[d + j];
        }
      }
      __builtin_memcpy(&qf[b][s], e, 16);
      // A negative scale is its amount and a turned sign of q.
      if (a.scale < 0.f) qf[b][s] ^= 0x80008000u;
    }
  }

  // Staging.  Group n of V holds the keys of steps 2 n and 2 n + 1, group n of
  // K those three steps on, 2 n + 3 and 2 n + 4; this wave loads SR rows of
  // each, from SR wave on.
  const int32_t* table = c.table + (int64_t)seq * c.table_stride;
  // A lane moves 16 bytes of IT rows of each.  Lanes past the rows, or past the
  // head's own width, repeat the first row or piece, so that nothing in the
  // loop is conditional.
  const int chunks = c.dim / 8;
  int srow[IT], kw[IT], vw[IT];
  uint32_t piece[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int x = i * 64 + lane;
    srow[i] = IT * 64 == SR * CH || x < SR * CH ? x / CH : 0;
    const int ch = x < SR * CH && x % CH < chunks ? x % CH : 0;
    piece[i] = ch * 16;
    kw[i] = (SR * wave + srow[i]) * L::KROW + ch * 16;
    vw[i] = 2 * L::KBUF + (SR * wave + srow[i]) * L::VROW + ch * 16;
  }
  // Every row's place in the cache is looked up by one lane, K's and V's, and
  // handed to those that load it: where 16 lanes load a row, it is one of
  // them, and the address comes by a broadcast among 16.
  constexpr bool BY16 = CH == 16;
  const bool isv = BY16 ? (l15 / IT) & 1 : (lane & 16) != 0;
  const int key0 = begin + SR * wave + (BY16 ? 4 * (l15 % IT) + (lane >> 4) : l15 % SR) + (isv ? 0 : 96);
  const uint32_t page_bytes = (uint32_t)(isv ? c.v_page : c.k_page) * 2u;
  const uint32_t token_bytes = (uint32_t)(isv ? c.v_token : c.k_token) * 2u;
  const uint64_t head = (uint64_t)(isv ? c.v : c.k) + (uint64_t)(kvh * (isv ? c.v_head : c.k_head) * 2);
  int page, at;   // of the lane's row in the groups that are looked up next
  // Keys outside the sequence read its first or last one.
  auto look_up = [&](int n) QMM_INLINE {
    int j = key0 + 64 * n;
    j = j > sq.len - 1 ? sq.len - 1 : j;
    j = j < 0 ? 0 : j;
    const int col = (int)div_by((uint32_t)j, c.by_page);
    at = j - col * c.page;
    page = table[col];
  };
  auto row_address = [&]() QMM_INLINE {
    const int p = page < 0 ? 0 : page >= c.pages ? c.pages - 1 : page;
    return head + (uint64_t)(uint32_t)p * page_bytes + (uint64_t)(uint32_t)at * token_bytes;
  };
  auto bring = [&](uint64_t rows, int i, int v) QMM_INLINE {   // the address of load i of K or V
    uint32_t x, y;
    if constexpr (BY16) {
      x = row_broadcast((uint32_t)rows, v * IT + i);
      y = row_broadcast((uint32_t)(rows >> 32), v * IT + i);
    } else {
      const int who = (16 * v + srow[i]) * 4;
      x = __builtin_amdgcn_ds_bpermute(who, (int)(uint32_t)rows);
      y = __builtin_amdgcn_ds_bpermute(who, (int)(uint32_t)(rows >> 32));
    }
    return ((uint64_t)y << 32 | x) + piece[i];
  };
  struct Stage {
    u32x4 x[IT];
  };
  auto load = [&](uint64_t rows, int v, Stage& st) QMM_INLINE {
#pragma unroll
    for (int i = 0; i < IT; ++i) st.x[i] = *(const __attribute__((address_space(1))) u32x4*)bring(rows, i, v);
  };
  auto kbuf = [&](int n) { return lds + (n & 1) * L::KBUF; };
  auto vbuf = [&](int n) { return lds + 2 * L::KBUF + (n & 1) * L::VBUF; };
  auto store_k = [&](int n, const Stage& st) QMM_INLINE {
#pragma unroll
    for (int i = 0; i < IT; ++i) *(u32x4*)(lds + (n & 1) * L::KBUF + kw[i]) = st.x[i];
  };
  auto store_v = [&](int n, const Stage& st) QMM_INLINE {
#pragma unroll
    for (int i = 0; i < IT; ++i) *(u32x4*)(lds + (n & 1) * L::VBUF + vw[i]) = st.x[i];
  };
  // Keys that not every row of the workgroup sees: a value that is not finite
  // would make NaN of a probability of 0.  It is replaced by 0 (as are keys
  // past the end), and added at the end to the rows that see it.
  const int safe0 = a.window ? max(begin, clip(pos_of(row1 - 1) - a.window + 1)) : begin;
  const int safe1 = a.causal ? min(end, clip(pos_of(row0) + 1)) : end;
  auto mend_v = [&](int n) QMM_INLINE {
    const int j0 = begin + 64 * n + SR * wave;
    if (j0 >= safe0 && j0 + SR <= safe1) return;
    bool any = false;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      char* to = lds + (n & 1) * L::VBUF + vw[i];
      u32x4 x = *(const u32x4*)to;
      const int j = j0 + srow[i];
      const bool in = j >= begin && j < end, safe = j >= safe0 && j < safe1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        constexpr uint32_t E = DT == DT_BF16 ? 0x7F80u : 0x7C00u;
        uint32_t y = in ? x[e] : 0u;
        const bool o0 = !safe && (y & E) == E, o1 = !safe && ((y >> 16) & E) == E;
        if (o0) y &= 0xFFFF0000u;
        if (o1) y &= 0x0000FFFFu;
        any |= o0 || o1;
        x[e] = y;
      }
      *(u32x4*)to = x;
    }
    if (__any(any)) odd = 1;
  };

  u32x4 kf[KS];                        // the next step's K operands
  f32x16 o[NQ][DB], s0[NQ], s1[NQ];   // scores of even and odd steps
  u32x4 p0[NQ][2], p1[NQ][2];         // probabilities of even and odd steps
  float m[NQ], mo[NQ], sub[NQ], l[NQ], top[NQ];
#pragma unroll
  for (int b = 0; b < NQ; ++b) {
    m[b] = -INFINITY;
    sub[b] = 0.f;
    l[b] = 0.f;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[b][d][i] = 0.f;
  }

  // One operand of a step's products from rows `row` .. of a buffer: K for 16
  // columns of the head, V for 16 keys u and 32 columns d.
  auto key = [&](const char* buf, int row, int k) QMM_INLINE {
    return *(const u32x4*)(buf + (row + l31) * L::KROW + half * 16 + k * 32);
  };
  auto value = [&](const char* buf, int row, int u, int d) QMM_INLINE {
    const char* at = buf + (row + 4 * half + l15 / 4) * L::VROW + (lane & 16) * 2 + (l15 % 4) * 8 +
                     16 * u * L::VROW + d * 64;
    const s16x4 x0 = lds_read_tr(at), x1 = lds_read_tr(at + 8 * L::VROW);
    return __builtin_bit_cast(u32x4, __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto zero = [&](f32x16& x) QMM_INLINE {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
  };
  auto scores = [&](const char* buf, int row, f32x16 (&out)[NQ]) QMM_INLINE {
#pragma unroll
    for (int b = 0; b < NQ; ++b) zero(out[b]);
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int b = 0; b < NQ; ++b) out[b] = Mfma32<DT>::run(key(buf, row, k), qf[b][k], out[b]);
  };
  auto tops = [&](const f32x16 (&x)[NQ]) QMM_INLINE {
#pragma unroll
    for (int b = 0; b < NQ; ++b) {
      float t = fmaxf(fmaxf(x[b][0], x[b][1]), x[b][2]);
#pragma unroll
      for (int i = 3; i < 15; i += 2) t = fmaxf(fmaxf(t, x[b][i]), x[b][i + 1]);
      top[b] = pair_max(fmaxf(t, x[b][15]));
    }
  };
  const float mul = CAP ? 1.f : fabsf(scale.mul);
  // Cap and mask the scores of step n, where it needs either.
  auto whole = [&](int n) { return begin + 32 * n >= all0 && begin + 32 * n + 32 <= all1; };
  auto finish = [&](int n, f32x16 (&x)[NQ]) QMM_INLINE {
    const int j0 = begin + 32 * n;
    const bool part = !whole(n);
    if (!CAP && !part) return;
    int base = j0 + 4 * half;
    asm volatile("" : "+v"(base));   // a branch, not selects in every step
    // Scores far below the cap, the usual ones, take the polynomial alone
    // (2048 new tokens over 8192 keys: 351 us, 502 with both in every step).
    bool far = false;
    if constexpr (CAP) {
#pragma unroll
      for (int b = 0; b < NQ; ++b) {
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(x[b][i]));
        far |= !(most * fabsf(scale.mul) < TANH_NEAR);
      }
      far = __any(far);
    }
#pragma unroll
    for (int b = 0; b < NQ; ++b) {
      if (CAP && far) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[b][i] = score<true>(x[b][i], ScoreScale{fabsf(scale.mul), scale.cap});
      } else if (CAP) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[b][i] = scale.cap * tanh_near(x[b][i] * fabsf(scale.mul));
      }
      if (!part) continue;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = base + 8 * (i / 4) + i % 4;
        if (!(j >= lo[b] && j < hi[b])) x[b][i] = -INFINITY;
      }
    }
    tops(x);
  };
  // A new reference maximum where a row passed the old one by the slack.  A
  // row's first is the maximum itself, so that a key which is seen alone has
  // the probability 1 and its value comes out as it is; from there it rises by
  // a whole number, so that the factor that the sum and the probabilities not
  // yet multiplied are taken down by is a power of two and rounds neither.
  // The output follows (mo) only where `all` is set, at one place of the loop:
  // until then it meets probabilities of its own reference alone.
  auto renew = [&](bool all, u32x4 (&p)[NQ][2]) QMM_INLINE {
    bool past = false;
#pragma unroll
    for (int b = 0; b < NQ; ++b) {
      top[b] *= mul;
      past |= top[b] > m[b] + SLACK || (all && mo[b] != m[b]);
    }
    if (__builtin_expect(!__any(past), 1)) return;
#pragma unroll
    for (int b = 0; b < NQ; ++b) {
      const float was = m[b], up = ceilf(fmaxf(top[b] - was, 0.f));   // a NaN raises nothing
      m[b] = was == -INFINITY ? fmaxf(top[b], was) : was + up;
      sub[b] = m[b] == -INFINITY ? 0.f : m[b] - SHIFT;
      const float back = was == -INFINITY ? 1.f : exp2_fast(-up);
      l[b] *= back;
      if (!all) continue;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          p[b][u][e] = Op::pack(bits16_to_f32<DT>((uint16_t)p[b][u][e]) * back,
                                bits16_to_f32<DT>((uint16_t)(p[b][u][e] >> 16)) * back);
      const float down = m[b] == -INFINITY ? 0.f : exp2_fast(mo[b] - m[b]);
#pragma unroll
      for (int d = 0; d < DB; ++d) o[b][d] *= down;
      mo[b] = m[b];
    }
  };
  // One score a lane, s[b][i], to its probability.  Pairs are rounded to the
  // values' type for the product: the matrix cores take no other pair.  The
  // sum keeps them in 32 bits.
  auto prob = [&](f32x16 (&s)[NQ], u32x4 (&q)[NQ][2], int i) QMM_INLINE {
#pragma unroll
    for (int b = 0; b < NQ; ++b) {
      s[b][i] = exp2_fast(__builtin_fmaf(s[b][i], mul, -sub[b]));
      l[b] += s[b][i];
      if (i & 1) q[b][i / 8][i % 8 / 2] = Op::pack(s[b][i - 1], s[b][i]);
    }
  };
  // Step n: scores of step n + 1 (to `next`), probabilities of this one (s to
  // q), output of step n - 1 (p).  The K operands were read during the step
  // before; as they are used, V's take their registers, and as those are used
  // the next step's K.  The order is the one written: a matrix instruction,
  // then the vector work that hides behind it.
  // A step with `stage` also moves the groups: those in registers (t + 1) to
  // LDS, the next ones' loads and the look-up of the ones after.
  Stage gk, gv;
  auto step = [&](bool stage, int t, int row, f32x16 (&s)[NQ], f32x16 (&next)[NQ],
                  const u32x4 (&p)[NQ][2], u32x4 (&q)[NQ][2]) QMM_INLINE {
    constexpr int VS = 2 * DB, SLOTS = KS + VS, LEAD = 2;
    const char *kb = kbuf(t), *vb = vbuf(t);
    uint64_t rows = 0;
    u32x4 vf[VS];
    float high[NQ];
#pragma unroll
    for (int b = 0; b < NQ; ++b) zero(next[b]);
#pragma unroll
    for (int v = 0; v < LEAD && v < VS; ++v) vf[v] = value(vb, row, v / DB, v % DB);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      if (j < KS) {
#pragma unroll
        for (int b = 0; b < NQ; ++b) next[b] = Mfma32<DT>::run(kf[j], qf[b][j], next[b]);
      } else {
        const int v = j - KS;
#pragma unroll
        for (int b = 0; b < NQ; ++b) o[b][v % DB] = Mfma32<DT>::run(vf[v], p[b][v / DB], o[b][v % DB]);
      }
      if (j + LEAD < VS) vf[j + LEAD] = value(vb, row, (j + LEAD) / DB, (j + LEAD) % DB);
      if (j >= KS) {
        const int x = j - KS, k = x >= LEAD ? x - LEAD : x + VS - LEAD;
        if (k < KS && (x < LEAD || k + LEAD < VS)) kf[k] = key(kb, row, k);
      }
#pragma unroll
      for (int i = 16 * j / SLOTS; i < 16 * (j + 1) / SLOTS; ++i) prob(s, q, i);
      if (stage) {
        if (j == SLOTS / 16) rows = row_address();
        if (j == SLOTS * 4 / 16) store_k(t + 1, gk);
        if (j == SLOTS * 5 / 16) store_v(t + 1, gv);
        if (j == SLOTS * 6 / 16) look_up(t + 3);
        if (j == SLOTS * 8 / 16) load(rows, 0, gk);
        if (j == SLOTS * 10 / 16) load(rows, 1, gv);
      }
      // The maximum of the next scores, in the last three slots.
#pragma unroll
      for (int b = 0; b < NQ; ++b) {
        if (j == SLOTS - 3) {
          high[b] = fmaxf(fmaxf(next[b][0], next[b][1]), next[b][2]);
          high[b] = fmaxf(fmaxf(high[b], next[b][3]), next[b][4]);
          high[b] = fmaxf(fmaxf(high[b], next[b][5]), next[b][6]);
        } else if (j == SLOTS - 2) {
          high[b] = fmaxf(fmaxf(high[b], next[b][7]), next[b][8]);
          high[b] = fmaxf(fmaxf(high[b], next[b][9]), next[b][10]);
          high[b] = fmaxf(fmaxf(high[b], next[b][11]), next[b][12]);
        } else if (j == SLOTS - 1) {
          high[b] = fmaxf(fmaxf(high[b], next[b][13]), next[b][14]);
          top[b] = pair_max(fmaxf(high[b], next[b][15]));
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // Held here: the compiler would move the exponentials past the branch.
#pragma unroll
    for (int b = 0; b < NQ; ++b)
      asm volatile("" : "+v"(q[b][0]), "+v"(q[b][1]), "+v"(l[b]));
  };

  // Columns that pad K's rows are not loaded.
  for (int x = threadIdx.x; x < 128 * (CH - chunks); x += THREADS)
    *(u32x4*)(lds + x % 128 / 64 * L::KBUF + x % 64 * L::KROW + (chunks + x / 128) * 16) =
        u32x4{0, 0, 0, 0};
  // K groups -2 and -1 hold steps 0, 1 and 2.  The first five groups' places
  // are looked up together, and then loaded together: each wait is a latency.
  Stage k2, k1;
  if (sq.len > 0) {
    uint64_t rows[4];
    int pages[4], ats[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      look_up(i - 2);
      pages[i] = page;
      ats[i] = at;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      page = pages[i];
      at = ats[i];
      rows[i] = row_address();
    }
    look_up(2);
    load(rows[0], 0, k2);
    load(rows[1], 0, k1);
    load(rows[2], 1, gv);
    load(rows[2], 0, gk);
    store_k(-2, k2);
    store_k(-1, k1);
    store_v(0, gv);
    mend_v(0);
    load(rows[3], 0, k1);
    load(rows[3], 1, gv);
  }
  __syncthreads();
  scores(kbuf(-2), 32, s0);
  tops(s0);
  finish(0, s0);
#pragma unroll
  for (int b = 0; b < NQ; ++b) {
    // A NaN is left to the sum.
    m[b] = fmaxf(top[b] * mul, -INFINITY);
    mo[b] = m[b];
    sub[b] = m[b] == -INFINITY ? 0.f : m[b] - SHIFT;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) prob(s0, p0, i);
  scores(kbuf(-1), 0, s1);
  tops(s1);
  finish(1, s1);
#pragma unroll
  for (int k = 0; k < KS; ++k) kf[k] = key(kbuf(-1), 32, k);
  __syncthreads();
  store_k(0, gk);
  gk = k1;
  const int iters = (steps + 1) / 2;
  for (int t = 0; t < iters; ++t) {
    __syncthreads();
    renew(true, p0);
    step(true, t, 0, s1, s0, p0, p1);
    mend_v(t + 1);
    if (CAP || !whole(2 * t + 2)) finish(2 * t + 2, s0);
    renew(false, p1);
    step(false, t, 32, s0, s1, p1, p0);
    if (CAP || !whole(2 * t + 3)) finish(2 * t + 3, s1);
  }

  // The output may still be a reference behind the sum.
#pragma unroll
  for (int b = 0; b < NQ; ++b) {
    const float down = m[b] == -INFINITY ? 0.f : exp2_fast(mo[b] - m[b]);
#pragma unroll
    for (int d = 0; d < DB; ++d) o[b][d] *= down;
  }

  // Values that were left out, for the rows that see them.
  if (odd) {
    for (int j = begin; j < end; ++j) {
      if (j >= safe0 && j < safe1) continue;
      int at;
      const int64_t page = page_of(c, table, j, at);
      const T* from = (const T*)c.v + page * c.v_page + kvh * c.v_head + at * c.v_token;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int col = 32 * d + 8 * (i / 4) + 4 * half + i % 4;
          const float x = col < c.dim ? dt<DT>::to_f32(from[col]) : 0.f;
          if (!(fabsf(x) < INFINITY))
#pragma unroll
            for (int b = 0; b < NQ; ++b)
              if (j >= lo[b] && j < hi[b]) o[b][d][i] += x;
        }
    }
  }

  // Write, or park this part of the keys.
#pragma unroll
  for (int b = 0; b < NQ; ++b) {
    const int r = wrow0 + 32 * b + l31;
    const float sum = pair_sum(l[b]);
    if (r >= row1) continue;
    const int i = (int)div_by(r, a.by_group), h = kvh * a.group + r - i * a.group;
    const int64_t tok = sq.t0 + i;
    if (plan.note && split == 0 && half == 0) a.part_count[tok * a.q_heads + h] = active;
    if (active == 1) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      T* to = (T*)a.out + tok * a.out_token + (int64_t)h * a.out_head;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = 32 * d + 8 * e + 4 * half;
          if (col >= c.dim) continue;
          const u32x2 w = {Op::pack(o[b][d][4 * e] * inv, o[b][d][4 * e + 1] * inv),
                           Op::pack(o[b][d][4 * e + 2] * inv, o[b][d][4 * e + 3] * inv)};
          if (a.out_wide) *(u32x2*)(to + col) = w;
          else __builtin_memcpy(to + col, &w, 8);
        }
      if (a.lse != nullptr && half == 0)
        a.lse[tok * a.lse_token + (int64_t)h * a.lse_head] =
            sum == 0.f ? -INFINITY : (m[b] + log2f(sum * DOWN)) * LN2;
    } else {
      const int64_t at = (int64_t)split * c.tokens * a.q_heads + tok * a.q_heads + h;
      if (half == 0) ((float2*)a.part_stats)[at] = make_float2(m[b], sum * DOWN);
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *(f32x4*)(a.part_out + at * DV + 32 * d + 8 * e + 4 * half) =
              f32x4{o[b][d][4 * e], o[b][d][4 * e + 1], o[b][d][4 * e + 2], o[b][d][4 * e + 3]} * DOWN;
    }
  }
}

template <int DT, int DK, int DV, int WAVES>
hipError_t launch_tile(const AttnArgs& a, const TilePlan& plan, const RowsPlan& few) {
  constexpr int THREADS = 64 * WAVES;
  const bool cap = a.softcap > 0.f;
  const ScoreScale k = cap ? ScoreScale{a.scale / a.softcap, a.softcap * LOG2E}
                           : ScoreScale{a.scale * LOG2E, 0.f};
  constexpr int need = (int)rows_lds_bytes(DV * 2, DV, WAVES);
  constexpr int bytes = TileLds<DK, DV>::BYTES > need ? TileLds<DK, DV>::BYTES : need;
  const void* fn = cap ? (const void*)attn_tile_kernel<DT, DK, DV, WAVES, true>
                       : (const void*)attn_tile_kernel<DT, DK, DV, WAVES, false>;
  const hipError_t e = ensure_dynamic_lds(fn, bytes);
  if (e != hipSuccess) return e;
  const dim3 grid((uint32_t)plan.few_groups + (uint32_t)plan.tiles * a.c.kv_heads);
  if (cap) attn_tile_kernel<DT, DK, DV, WAVES, true><<<grid, THREADS, bytes, a.stream>>>(a, plan, few, k);
  else attn_tile_kernel<DT, DK, DV, WAVES, false><<<grid, THREADS, bytes, a.stream>>>(a, plan, few, k);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_tile_type(const AttnArgs& a, const TilePlan& plan, const RowsPlan& few) {
  const int d = a.c.dim;
#define QMM_TILE(DK, DV)                                                     \
  if (d <= DK) return plan.blocks == 2 ? launch_tile<DT, DK, DV, 8>(a, plan, few) \
                                       : launch_tile<DT, DK, DV, 4>(a, plan, few);
  QMM_TILE(64, 64) QMM_TILE(80, 96) QMM_TILE(96, 96) QMM_TILE(128, 128)
#undef QMM_TILE
  if (d <= 192) return launch_tile<DT, 192, 192, 4>(a, plan, few);
  return launch_tile<DT, 256, 256, 4>(a, plan, few);
}

}  // namespace qmm
