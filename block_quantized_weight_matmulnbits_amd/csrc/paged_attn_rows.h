// paged_attn_rows.h -- attention of a few query rows over a paged cache.
//
// The query rows of a sequence that share a key/value head (its new tokens
// times the heads of the group) are packed side by side, 16 a matrix-core
// column block, so that every key and value is read once for all of them.
// With few rows the keys are the work, and the bound is HBM: they are split
// over workgroups in runs of `chunk` keys and, inside one, over its four waves
// in blocks of 32.  A wave needs no other until its last key: it keeps its own
// running maximum, sum and output, loads K straight into matrix-core operands
// (16 bytes a lane) and V through its own LDS (16 bytes a lane, asynchronous),
// from where 16-bit values are read back transposed.  The waves join through
// LDS; parts of the keys are left in the workspace for the join.
//
// 64 sequences of 17 to 8191 keys, a token each (32 heads of 128 over 8, bf16):
// 230 us with the join, 4.98 TB/s of keys and values, where a large copy moves
// 4.95.  Two sequences of 90001 and 131071 keys: 190 us, 4.8 TB/s.  Five guessed f32
// tokens for each of 7 sequences: 22 us, of which latencies in a row are most.
#pragma once

#include "paged_attn.h"
#include "qmm_internal.h"

namespace qmm {

constexpr int ROWS_WAVES = 4, ROWS_THREADS = 64 * ROWS_WAVES, ROWS_BLOCK = 32;
#define QMM_INLINE __attribute__((always_inline))

constexpr size_t rows_lds_bytes(int row_bytes, int dp, int waves) {
  const size_t v = (size_t)ROWS_BLOCK * row_bytes, o = (size_t)16 * (dp + 4) * 4;
  return waves * (v > o ? v : o);
}

// Waves a SIMD that the registers are cut for.
template <int DT, int DP, int NB> struct RowsWaves {
  static constexpr int RB = DP * (DT == DT_F32 ? 4 : 2);
  static constexpr int N = RB * NB <= 768 ? 2 : 1;
};

// One workgroup of WAVES waves, number `id` of the plan's.
template <int DT, int DP, int NB, int WAVES, bool CAP>
__device__ __forceinline__ void attn_rows(const AttnArgs& a, const RowsPlan& plan,
                                          const ScoreScale& scale, int skip_above, uint32_t id,
                                          char* lds) {
  constexpr bool F32 = DT == DT_F32;
  using T = typename dt<DT>::T;
  constexpr int ES = (int)sizeof(T), RB = DP * ES;   // bytes of a padded row
  constexpr int KS = RB / 64;                        // 64-byte steps along a row
  constexpr int DB = DP / 16;                        // output blocks of 16 columns
  // Heads up to this width run on a narrower variant.
  constexpr int NARROWER = DP == 64 ? 0 : DP == 96 ? 64 : DP == 128 ? 96 : DP == 192 ? 128 : 192;
  // The next block's keys are loaded ahead where registers hold them.
  constexpr bool AHEAD = RB <= 512;
  constexpr int VBYTES = ROWS_BLOCK * RB;
  constexpr int OSTRIDE = DP + 4;
  constexpr uint32_t EXP = DT == DT_BF16 ? 0x7F80u : 0x7C00u;   // a 16-bit value's exponent
  constexpr float UP = exp2_of(prob_shift<DT>(0));   // of the outputs until they leave
  __shared__ float2 wave_ml[WAVES][16];

  const CacheArgs& c = a.c;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l15 = lane & 15, g = lane >> 4;
  // Parts fastest, then heads.  Workgroups go round the eight XCDs by number,
  // and the last parts of short sequences have no work: turned by the rest of
  // the number, every XCD gets first parts and last ones alike (64 sequences
  // of 17 to 8191 keys, in parts of 1024: 296 us without, 235 with).
  const int split = (id % plan.splits + id / plan.splits) % plan.splits;
  id /= plan.splits;
  const int kvh = id % c.kv_heads;
  id /= c.kv_heads;
  // A sequence's last rows see the most keys and come first.
  const int tile = plan.row_tiles - 1 - (int)(id % plan.row_tiles), seq = id / plan.row_tiles;

  if (seq >= c.seqs) return;
  const Seq sq = seq_of(c, seq);
  const int rows = sq.n * a.group, row0 = tile * 16 * NB;
  if (row0 >= rows || sq.n > skip_above) return;
  const int row1 = rows < row0 + 16 * NB ? rows : row0 + 16 * NB;
  const int pos0 = sq.len - sq.n;
  const int first_pos = pos0 + (int)div_by(row0, a.by_group);
  const int last_pos = pos0 + (int)div_by(row1 - 1, a.by_group);
  auto clip = [&](int j) { return j < 0 ? 0 : j > sq.len ? sq.len : j; };
  // Keys that any row of the tile sees, and those that all of them see.
  const int kmin = a.window ? clip(first_pos - a.window + 1) : 0;
  const int kmax = a.causal ? clip(last_pos + 1) : sq.len;
  const int all0 = a.window ? clip(last_pos - a.window + 1) : 0;
  const int all1 = a.causal ? clip(first_pos + 1) : sq.len;

  int active = kmax > kmin ? (kmax - kmin + plan.chunk - 1) / plan.chunk : 1;
  active = active > plan.splits ? plan.splits : active;
  if (split >= active) return;
  const int begin = kmin + split * plan.chunk;
  const int end = split == active - 1 ? kmax : begin + plan.chunk;

  // Query rows as the B operand: column l15, 16 bytes of step 4 s + g.
  u32x4 qf[NB][KS];
  int lo[NB], hi[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int r = row0 + 16 * b + l15;
    const bool ok = r < row1;
    const int i = ok ? (int)div_by(r, a.by_group) : 0, h = ok ? r - i * a.group : 0;
    const int pos = pos0 + i;
    lo[b] = a.window ? pos - a.window + 1 : 0;
    hi[b] = !ok ? 0 : a.causal ? clip(pos + 1) : sq.len;
    const T* from = (const T*)a.q + (int64_t)(sq.t0 + i) * a.q_token +
                    (int64_t)(kvh * a.group + h) * a.q_head;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = (4 * s + g) * (16 / ES);
      T e[16 / ES];
#pragma unroll
      for (int j = 0; j < 16 / ES; ++j) e[j] = T(0);
      if (ok && d < c.dim) {
        if (a.q_wide) {
          __builtin_memcpy(e, __builtin_assume_aligned(from + d, 16), 16);
        } else {
#pragma unroll
          for (int j = 0; j < 16 / ES; ++j) e[j] = from[d + j];
        }
      }
      __builtin_memcpy(&qf[b][s], e, 16);
    }
  }

  const int32_t* table = c.table + (int64_t)seq * c.table_stride;
  char* vl = lds + wave * VBYTES;
  const char* zeros = (const char*)zero_row;

  // Rows of a block that this lane loads, keys 16 t + l15, from its first
  // piece on; a key past the end reads zeros.
  struct Rows {
    const char *k[2], *v[2];
  };
  auto rows_at = [&](int kb) {
    Rows r;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int j = kb + 16 * t + l15;
      r.k[t] = r.v[t] = zeros;
      if (j < end) {
        int at;
        const int64_t page = page_of(c, table, j, at);
        r.k[t] = c.k + (page * c.k_page + kvh * c.k_head + at * c.k_token) * ES;
        r.v[t] = c.v + (page * c.v_page + kvh * c.v_head + at * c.v_token) * ES;
      }
      r.k[t] += g * 16;
      r.v[t] += g * 16;
    }
    return r;
  };
  // Step s of a row; past the head's own width, where the padded one may pass
  // it, zeros.
  auto piece = [&](const char* row, int s) {
    if (64 * (s + 1) > NARROWER * ES && (4 * s + g) * 16 >= c.dim * ES) return zeros;
    return row + 64 * s;
  };
  auto load_k = [&](const Rows& r, u32x4 (&k)[2][KS]) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int s = 0; s < KS; ++s) k[t][s] = *(const u32x4*)piece(r.k[t], s);
  };

  f32x4 o[NB][DB];
  float m[NB], l[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    m[b] = -INFINITY;
    l[b] = 0.f;
#pragma unroll
    for (int d = 0; d < DB; ++d) o[b][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  u32x4 kf[2][KS];
  Rows rw;
  int kb = begin + ROWS_BLOCK * wave;
  if (AHEAD && kb < end) {
    rw = rows_at(kb);
    load_k(rw, kf);
  }
  for (; kb < end; kb += ROWS_BLOCK * WAVES) {
    if constexpr (!AHEAD) {
      rw = rows_at(kb);
      load_k(rw, kf);
    }
    // V of this block and K of the next are in flight together.
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int t = 0; t < 2; ++t) load_to_lds(piece(rw.v[t], s), vl + (s * 2 + t) * 1024);
    u32x4 kn[AHEAD ? 2 : 1][AHEAD ? KS : 1];
    const int next = kb + ROWS_BLOCK * WAVES;
    if constexpr (AHEAD) {
      if (next < end) {
        rw = rows_at(next);
        load_k(rw, kn);
      }
    }

    f32x4 sc[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t) sc[b][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if constexpr (F32) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sc[b][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                  __uint_as_float(kf[t][s][e]), __uint_as_float(qf[b][s][e]), sc[b][t], 0, 0, 0);
          } else {
            using V8 = typename MfmaOp<F32 ? DT_BF16 : DT>::V;
            sc[b][t] = MfmaOp<F32 ? DT_BF16 : DT>::run(__builtin_bit_cast(V8, kf[t][s]),
                                                       __builtin_bit_cast(V8, qf[b][s]), sc[b][t]);
          }
        }

    const bool full = kb >= all0 && kb + ROWS_BLOCK <= all1 && kb + ROWS_BLOCK <= end;
    float p[NB][2][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = score<CAP>(sc[b][t][i], scale);
          if (!full) {
            const int j = kb + 16 * t + 4 * g + i;
            x = j >= lo[b] && j < hi[b] && j < end ? x : -INFINITY;
          }
          p[b][t][i] = x;
          top = fmaxf(top, x);
        }
      const float was = m[b];
      m[b] = fmaxf(was, col_max(top));
      const float ref = m[b] == -INFINITY ? 0.f : m[b];
      if (__any(m[b] != was)) {
        const float back = exp2_fast(was - ref);
        l[b] *= back;
#pragma unroll
        for (int d = 0; d < DB; ++d) o[b][d] *= back;
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[b][t][i] = exp2_fast(p[b][t][i] - ref);
          l[b] += p[b][t][i];
        }
    }

    wait_loads();
    // Whether the block holds a value that is not finite.
    bool odd = false;
    if (!F32 || !full) {
      u16x2 top = {0, 0};
#pragma unroll
      for (int s = 0; s < 2 * KS; ++s) {
        const u32x4 x = *(const u32x4*)(vl + s * 1024 + lane * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (F32) odd |= (x[e] & 0x7F800000u) == 0x7F800000u;
          else top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, x[e] & (EXP | EXP << 16)));
        }
      }
      if constexpr (!F32) odd = top[0] == EXP || top[1] == EXP;
      odd = __any(odd);
    }
    // A masked key adds nothing, whatever its value holds: with a NaN or an
    // infinity in the block the product would make NaN of 0 times it.
    const bool apart = !full && odd;
    auto value_f32 = [&](int d, int t, int i) QMM_INLINE {
      return *(const float*)(vl + (d * 2 + t) * 1024 + (l15 / 4) * 256 + (4 * g + i) * 16 + (l15 % 4) * 4);
    };
    // 32 bits, where products bound many rows: nothing but products, of two
    // blocks of columns in turn, so that none waits for the one before it (900
    // tokens of 3 sequences, 32 heads of 128: 551 us as below, 474 so, both in parts of
    // 1024 keys).
    if (F32 && __builtin_expect(!apart, 1)) {
#pragma unroll
      for (int d = 0; d < DB; d += 2)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = d; e < d + 2; ++e) {
              const float x = value_f32(e, t, i);
#pragma unroll
              for (int b = 0; b < NB; ++b)
                o[b][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(x, p[b][t][i], o[b][e], 0, 0, 0);
            }
    }
    // A block with such values is taken key by key: the product of that key
    // alone, kept in the columns that see it.  In 16 bits the others pass
    // through the same code (a copy without the choices gained nothing).
    const int rounds = apart ? ROWS_BLOCK : F32 ? 0 : 1;
#pragma unroll 1
    for (int key = 0; key < rounds; ++key) {
      const int only = apart ? (key % 16) / 4 == g ? key / 16 * 4 + key % 4 : -1 : -2;
      bool sees[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b)
        sees[b] = !apart || (kb + key >= lo[b] && kb + key < hi[b] && kb + key < end);
      if constexpr (F32) {
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          f32x4 n[NB];
#pragma unroll
          for (int b = 0; b < NB; ++b) n[b] = o[b][d];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = only == 4 * t + i ? value_f32(d, t, i) : 0.f;
#pragma unroll
              for (int b = 0; b < NB; ++b)
                n[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(x, p[b][t][i], n[b], 0, 0, 0);
            }
#pragma unroll
          for (int b = 0; b < NB; ++b)
            if (sees[b]) o[b][d] = n[b];
        }
      } else {
        // The matrix cores take probabilities of the values' type only: they
        // enter as what that type holds and, in a product of its own, what it
        // leaves of 32 bits, so that the output is as near as its type allows.
        // The keys being the work, the second product costs little (64
        // sequences of 17 to 8191 keys: 232 us with one and with two, the root
        // mean square of the error 2.0e-4 and 1.8e-4, that of probabilities of
        // 32 bits; 20 sequences of 8 guessed tokens 64 and 65.6 us).
        constexpr int T16 = F32 ? DT_BF16 : DT;
        using Op = MfmaOp<T16>;
        u32x4 pb[NB], rest[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = p[b][e / 2][e % 2 * 2] * UP, y = p[b][e / 2][e % 2 * 2 + 1] * UP;
            pb[b][e] = Op::pack(x, y);
            rest[b][e] = Op::pack(x - bits16_to_f32<T16>((uint16_t)pb[b][e]),
                                  y - bits16_to_f32<T16>((uint16_t)(pb[b][e] >> 16)));
          }
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          const char* at = vl + (d / 2) * 2048 + (2 * (d % 2) + (l15 % 4) / 2) * 256 +
                           (4 * g + l15 / 4) * 16 + (l15 % 2) * 8;
          const s16x4 x0 = lds_read_tr(at), x1 = lds_read_tr(at + 1024);
          auto v = __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
          auto w = v;   // for the rest, which may be 0 or less: no infinity
          if (odd) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (apart && only != e) v[e] = 0;
              w[e] = ((uint32_t)v[e] & EXP) == EXP ? (short)0 : v[e];
            }
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            f32x4 n = Op::run(__builtin_bit_cast(typename Op::V, v),
                              __builtin_bit_cast(typename Op::V, pb[b]), o[b][d]);
            n = Op::run(__builtin_bit_cast(typename Op::V, w),
                        __builtin_bit_cast(typename Op::V, rest[b]), n);
            if (sees[b]) o[b][d] = n;
          }
        }
      }
    }
    if constexpr (AHEAD) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int s = 0; s < KS; ++s) kf[t][s] = kn[t][s];
    }
  }

  // Join the waves, one block of 16 rows at a time, and write or park it.
  float* ol = (float*)lds;
  auto emit = [&](int r, int d, f32x4 x, float inv) {
    const int i = (int)div_by(r, a.by_group), h = r - i * a.group;
    T* to = (T*)a.out + (int64_t)(sq.t0 + i) * a.out_token +
            (int64_t)(kvh * a.group + h) * a.out_head + d;
    T e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = dt<DT>::from_f32(x[j] * inv);
    if (a.out_wide) __builtin_memcpy(__builtin_assume_aligned(to, 4 * ES), e, 4 * ES);
    else
#pragma unroll
      for (int j = 0; j < 4; ++j) to[j] = e[j];
  };
  auto emit_lse = [&](int r, float top, float sum) {
    if (a.lse == nullptr) return;
    const int i = (int)div_by(r, a.by_group), h = r - i * a.group;
    a.lse[(int64_t)(sq.t0 + i) * a.lse_token + (int64_t)(kvh * a.group + h) * a.lse_head] =
        sum == 0.f ? -INFINITY : (top + log2f(sum)) * LN2;
  };
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    __syncthreads();
    const float sum = col_sum(l[b]);
    if (g == 0) wave_ml[wave][l15] = make_float2(m[b], sum);
#pragma unroll
    for (int d = 0; d < DB; ++d)
      *(f32x4*)(ol + (wave * 16 + l15) * OSTRIDE + 16 * d + 4 * g) = o[b][d];
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * (DP / 4); e += 64 * WAVES) {
      const int q = e / (DP / 4), d = e % (DP / 4) * 4, r = row0 + 16 * b + q;
      if (r >= row1 || d >= c.dim) continue;
      float top = -INFINITY, total = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) top = fmaxf(top, wave_ml[w][q].x);
      const float ref = top == -INFINITY ? 0.f : top;
      f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const float f = exp2_fast(wave_ml[w][q].x - ref);
        total += f * wave_ml[w][q].y;
        x += f * *(const f32x4*)(ol + (w * 16 + q) * OSTRIDE + d);
      }
      x *= 1.f / UP;
      if (plan.note) {
        const int i = (int)div_by(r, a.by_group);
        const int64_t row = (int64_t)(sq.t0 + i) * a.q_heads + kvh * a.group + r - i * a.group;
        const int64_t at = (int64_t)split * c.tokens * a.q_heads + row;
        if (split == 0 && d == 0) a.part_count[row] = active;
        if (active > 1) {
          *(f32x4*)(a.part_out + at * DP + d) = x;
          if (d == 0) ((float2*)a.part_stats)[at] = make_float2(top, total);
          continue;
        }
      }
      emit(r, d, x, total == 0.f ? 0.f : 1.f / total);
      if (d == 0) emit_lse(r, top, total);
    }
  }
}

template <int DT, int DP, int NB, bool CAP>
__global__ __launch_bounds__(ROWS_THREADS, (RowsWaves<DT, DP, NB>::N)) void attn_rows_kernel(
    AttnArgs a, RowsPlan plan, ScoreScale scale, int skip_above) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  attn_rows<DT, DP, NB, ROWS_WAVES, CAP>(a, plan, scale, skip_above, blockIdx.x, lds);
}

template <int DT, int DP, int NB>
hipError_t launch_rows(const AttnArgs& a, const RowsPlan& plan, int skip_above) {
  constexpr int ES = (int)sizeof(typename dt<DT>::T);
  constexpr size_t bytes = rows_lds_bytes(DP * ES, DP, ROWS_WAVES);
  const bool cap = a.softcap > 0.f;
  const ScoreScale k = cap ? ScoreScale{a.scale / a.softcap, a.softcap * LOG2E}
                           : ScoreScale{a.scale * LOG2E, 0.f};
  const void* fn = cap ? (const void*)attn_rows_kernel<DT, DP, NB, true>
                       : (const void*)attn_rows_kernel<DT, DP, NB, false>;
  const hipError_t e = ensure_dynamic_lds(fn, (int)bytes);
  if (e != hipSuccess) return e;
  const dim3 grid((uint32_t)a.c.seqs * plan.row_tiles * a.c.kv_heads * plan.splits);
  if (cap) attn_rows_kernel<DT, DP, NB, true><<<grid, ROWS_THREADS, bytes, a.stream>>>(a, plan, k, skip_above);
  else attn_rows_kernel<DT, DP, NB, false><<<grid, ROWS_THREADS, bytes, a.stream>>>(a, plan, k, skip_above);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_rows_type(const AttnArgs& a, const RowsPlan& plan, int blocks, int skip_above) {
  const int d = a.c.dim;
#define QMM_ROWS(DP)                                                                    \
  if (d <= DP) return DT != DT_F32 || blocks == 1                                       \
                          ? launch_rows<DT, DP, 1>(a, plan, skip_above)                 \
                          : launch_rows<DT, DP, DT == DT_F32 ? 2 : 1>(a, plan, skip_above);
  QMM_ROWS(64) QMM_ROWS(96) QMM_ROWS(128) QMM_ROWS(192) QMM_ROWS(256)
#undef QMM_ROWS
  return hipErrorInvalidValue;
}

}  // namespace qmm
