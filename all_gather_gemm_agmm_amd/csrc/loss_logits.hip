// Vocabulary loss, the passes over the logits (gfx950).  The logits
//     x[i, v] = sum_k A[i, k] * W[v, k]          (rows i of the shards, W n x k)
// of one piece of the vocabulary are tiles of the part-ring GEMM
// (gemm_m16_loop.inc); they never leave the registers as logits:
//
//  * loss_stats_kernel: per row and 64 or 128 columns (a wave's share of the
//    tile) the maximum m and sum exp(x - m), and the label's logit from the one
//    lane that holds it.  loss_combine_kernel merges them over columns:
//    lse = M + log(sum_p s_p exp(m_p - M)), loss = lse - target.
//  * loss_grad_kernel: d[i, v] = a_i exp(x - lse_i) - b_i [v = label_i] as
//    16-bit operands of the two gradient products, by rows [i][v] for
//    dA = d W and transposed [v][i] for dW = d^T A: one tile in LDS, stored
//    row by row, then once more through transposing reads.  Rounding d to 16
//    bits (the operands' own precision) is what lets the matrix cores compute
//    both gradients; the sums are fp32.  d is scaled by 1 / S, S the rows'
//    largest weight (loss_rows).  bf16 has the range of fp32.  fp16 has
//    not: each row of d is scaled by a further power of two (exact) that brings
//    its weight near 1, and by 2^14, which keeps a probability of 2^-27 a
//    normal number; dA's rows are scaled back in fp32.  dW sums over rows, so
//    its operand d^T has one scale, 2^14 / S: row i times s_i / S, a power of
//    two of at least 2^-24, as it leaves the tile.  What that takes from a small
//    row is at most S 2^-38 of a d, where dW's own steps are 2^-24 or more.  (A
//    copy of A that carried the rows' powers instead lost rows of weight 2^-20
//    to 2%, of 2^-27 wholly.)
//
// Bound: MFMA; with few rows HBM on W.  The exponentials cost 256 (256 x 256
// tile) per lane once per tile, 3-5% beside the k loop of a 4096-deep product.
// Measured: loss_stats_kernel, 8192 x 4096 bf16 over 131072 columns 5.9-6.3 ms,
// 1400-1490 TFLOP/s (a library's product alone: 1310-1580); 8 x 4096 fp16 over
// 131072 176-179 us, 6.0 TB/s of W.  loss_grad_kernel, 8192 x 4096 over 16384
// columns 0.84-0.90 ms, 1220-1310 TFLOP/s: it also writes d twice, 512 MiB.
// loss_combine_kernel, 8192 rows of 1024 partials 13 us, 5.2 TB/s.
// loss_prepare_kernel's copy of 40000 x 2500 elements (a row length that is no
// multiple of 8) 84 us, 4.8 TB/s; element by element it took 136.
//
// The maximum uses v_max, which passes over NaN, but a NaN logit makes its
// sum NaN, so a row with one has a NaN loss.  Infinite maxima are replaced
// by 0 inside exp: a row of -inf only gives lse = -inf, one with +inf gives +inf.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_kernels.h"
#include "gemm_device.h"

namespace agmm {

namespace {

typedef float f32x2_t __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

__device__ __forceinline__ float finite_or_zero(float m) {
  return __builtin_fabsf(m) == __builtin_inff() ? 0.0f : m;
}

template <int BM, int BN, int BK, int DT, int WAVES, int OCC, bool GRAD>
__device__ __forceinline__ void loss_body(const LossProblem& lp, char* smem) {
  constexpr bool BT = true, SPLIT = false;
  const GemmProblem& p = lp.gemm;
  using T = GemmTile<BM, BN, BK, DT, BT, 5, WAVES, kLoopParts>;
  constexpr int kBK = BK;
  constexpr int FM = T::TM / 16, FN = T::TN / 16;
  constexpr int STEPS = BK / 32;

#include "gemm_m16_loop.inc"

  const bool whole = m0 + BM <= M && n0 + BN <= N;
  const int wcol = n0 + wn * T::TN;          // first column of the wave
  if constexpr (!GRAD) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int row = m0 + wm * T::TM + 16 * i + i16;
      float mx = -__builtin_inff();
      if (whole) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx = fmaxf(mx, acc[i][j][e]);
      } else {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (wcol + 16 * j + 4 * g4 + e < N) mx = fmaxf(mx, acc[i][j][e]);
      }
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float off = finite_or_zero(mx);
      float sum = 0.0f;
      if (whole) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum += exp_of(acc[i][j][e] - off);
      } else {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (wcol + 16 * j + 4 * g4 + e < N) sum += exp_of(acc[i][j][e] - off);
      }
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (g4 == 0 && row < M) {
        float* d = lp.stats + ((int64_t)(cb * T::WN + wn) * M + row) * 2;
        d[0] = mx;
        d[1] = sum;
      }
      // the label's logit, in the one wave whose columns hold it
      const int64_t at = row < M ? lp.labels[row] - lp.label0 - wcol : -1;
      if (__any(at >= 0 && at < T::TN)) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (at == 16 * j + 4 * g4 + e && wcol + at < N) lp.target[row] = acc[i][j][e];
      }
    }
  } else {
    // the rows' values, all on their way at once
    f32x4_t rv[FM];
    int at[FM];       // the label's column within the wave's, or -1
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int row = min(m0 + wm * T::TM + 16 * i + i16, M - 1);
      rv[i] = *reinterpret_cast<const f32x4_t*>(lp.rows + 4 * (int64_t)row);
      const int64_t rel = lp.labels[row] - lp.label0 - wcol;
      at[i] = rel >= 0 && rel < T::TN ? (int)rel : -1;
    }
    __syncthreads();   // the LDS now holds d: chunk c (8 columns) of tile row r at c ^ (r mod 16)
    constexpr int RB = BN * 2, CH = RB / 16;
    // fp16: behind d, the rows' powers of two s_i / S
    constexpr bool kRowPowers = DT == kDtypeFp16;
    static_assert(BM * RB + BM * 2 <= T::LDS_BYTES, "d and the rows' powers of two");
    _Float16* const power = reinterpret_cast<_Float16*>(smem + BM * RB);
    const float all = kRowPowers ? lp.scale_all[0] : 1.0f;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = wm * T::TM + 16 * i + i16;
      const bool in = m0 + r < M;
      const float f = (DT == kDtypeFp16 ? 16384.0f : 1.0f) / rv[i][3];
      const float lse = rv[i][0], a = rv[i][1] * f, b = rv[i][2] * f;
      if (kRowPowers && wn == 0 && g4 == 0) power[r] = (_Float16)(rv[i][3] / all);
      const bool hit = __any(at[i] >= 0);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        float d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = a * exp_of(acc[i][j][e] - lse);
        if (hit)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (at[i] == 16 * j + 4 * g4 + e) d[e] -= b;
        if (!whole)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!in || wcol + 16 * j + 4 * g4 + e >= N) d[e] = 0.0f;
        const int c = wn * T::TN + 16 * j + 4 * g4;
        *reinterpret_cast<u32x2_t*>(smem + r * RB + (((c >> 3) ^ (r & 15)) << 4) + (c & 4) * 2) =
            u32x2_t{pack2<DT>(d[0], d[1]), pack2<DT>(d[2], d[3])};
      }
    }
    __syncthreads();
    if (lp.d) {
      // whole rows, 16 bytes per lane, eight on their way at a time
      constexpr int ROWS = T::THREADS / CH;          // rows per pass
      const int c = tid % CH;
      const bool cin = n0 + c * 8 < lp.ldd;
      uint16_t* out = static_cast<uint16_t*>(lp.d) + (int64_t)m0 * lp.ldd + n0 + c * 8;
#pragma unroll 8
      for (int r = tid / CH; r < BM; r += ROWS) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(smem + r * RB + ((c ^ (r & 15)) << 4));
        if (cin && m0 + r < M) *reinterpret_cast<u32x4_t*>(out + (int64_t)r * lp.ldd) = v;
      }
    }
    if (lp.dt) {
      // Transposing reads: a wave takes 16 columns x 32 rows at a time, lane
      // (g4, i16) the rows 8 g4 .. 8 g4 + 7 of column i16 (two reads of four
      // rows, each lane of a group giving the address of row i16 / 4, columns
      // 4 (i16 % 4) .. + 3 of the 4 x 16 block), 16 bytes of the column's row.
      constexpr int PASSES = (BM / 32) * (BN / 16) / (T::THREADS / 64);
      uint16_t* out = static_cast<uint16_t*>(lp.dt) + (int64_t)n0 * lp.ldt + m0;
#pragma unroll 8
      for (int q = 0; q < PASSES; ++q) {
        const int u = q * (T::THREADS / 64) + wave;
        const int nb = (u / (BM / 32)) * 16, mb = (u % (BM / 32)) * 32 + 8 * g4;
        u32x2_t half[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = mb + 4 * h + (i16 >> 2), c = nb + 4 * (i16 & 3);
          half[h] = read_tr(smem + r * RB + (((c >> 3) ^ (r & 15)) << 4) + (c & 4) * 2);
        }
        if constexpr (kRowPowers) {
          const f16x8_t f = *reinterpret_cast<const f16x8_t*>(power + mb);   // of rows mb .. mb + 7
          const f16x8_t v = __builtin_bit_cast(f16x8_t, u32x4_t{half[0][0], half[0][1], half[1][0], half[1][1]}) * f;
          const u32x4_t w = __builtin_bit_cast(u32x4_t, v);
          half[0] = u32x2_t{w[0], w[1]};
          half[1] = u32x2_t{w[2], w[3]};
        }
        if (n0 + nb + i16 < N && m0 + mb < lp.ldt)
          *reinterpret_cast<u32x4_t*>(out + (int64_t)(nb + i16) * lp.ldt + mb) =
              u32x4_t{half[0][0], half[0][1], half[1][0], half[1][1]};
      }
    }
  }
}

template <int BM, int BN, int DT, int OCC>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
void loss_stats_kernel(LossProblem lp) {
  __shared__ __attribute__((aligned(1024))) char smem[GemmTile<BM, BN, 64, DT, true, 5, 4, kLoopParts>::LDS_BYTES];
  loss_body<BM, BN, 64, DT, 4, OCC, false>(lp, smem);
}

template <int BM, int BN, int DT, int OCC>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
void loss_grad_kernel(LossProblem lp) {
  __shared__ __attribute__((aligned(1024))) char smem[GemmTile<BM, BN, 64, DT, true, 5, 4, kLoopParts>::LDS_BYTES];
  loss_body<BM, BN, 64, DT, 4, OCC, true>(lp, smem);
}

// Few rows: FM x FN blocks of 16 rows x 16 columns per workgroup.  The waves
// share out k, 64 elements (whole 128-byte lines) at a time, and load their
// operands straight into registers: 16-byte accesses to global memory may start
// at any word, which loads into LDS may not, so neither operand is copied first
// whatever k and the strides are.  UN pieces are on their way at a time.  The
// waves' sums are added in LDS in a fixed order, wave w taking row block w.
// ODD (a stride is odd): rows that start in the middle of a word are read from
// that word on, with one word more, and shifted; accesses that start there take
// three times as long (24 rows of 3121 over 5391 columns: 55 us, 30 shifted, 18
// at 3122).  Bound: HBM on W (8 rows of 3008 over 20000 columns 23 us, 5.2
// TB/s), with more rows the operands' way into the CUs.
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));

template <int DT, int FM, int FN, int UN, bool ODD, bool GRAD>
__global__ __launch_bounds__(256) void loss_few_kernel(LossProblem lp) {
  const GemmProblem& p = lp.gemm;
  __shared__ float part[4][FM][FN][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g4 = lane >> 4, i16 = lane & 15;
  const int M = p.m, N = p.n, K = p.k;
  const int cb = (int)blockIdx.x / p.order.num_rb, rb = (int)blockIdx.x - cb * p.order.num_rb;
  const int m0 = rb * 16 * FM, n0 = cb * 16 * FN;
  // rows and columns past the end read the last one and are never used
  const uint16_t *a[FM], *b[FN];
#pragma unroll
  for (int f = 0; f < FM; ++f) {
    const int i = min(m0 + 16 * f + i16, M - 1), g = i / p.rows.rows_per_group;
    a[f] = static_cast<const uint16_t*>(p.rows.a_group[g]) + (int64_t)(i - g * p.rows.rows_per_group) * p.rows.a_ld + 8 * g4;
  }
#pragma unroll
  for (int f = 0; f < FN; ++f)
    b[f] = static_cast<const uint16_t*>(p.b) + (int64_t)min(n0 + 16 * f + i16, N - 1) * p.ldb + 8 * g4;

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const auto multiply = [&](const u32x4_t (&fa)[FM], const u32x4_t (&fb)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = mfma16_builtin<DT>(fb[j], fa[i], acc[i][j]);
  };
  // halves 2u, 2u + 1 of piece c + u: elements 64 (c + u) + 32 h + 8 g4 on;
  // ODD: their words and the one behind
  constexpr int W = ODD ? 2 * UN : 1;
  typedef u32x4_t u32x4_word_t __attribute__((aligned(4)));
  const auto load = [&](int c, u32x4_t (&fa)[2 * UN][FM], u32x4_t (&fb)[2 * UN][FN], uint32_t (&wa)[W][FM], uint32_t (&wb)[W][FN]) {
    const auto one = [&](const uint16_t* x, u32x4_t& v, uint32_t& w) {
      if constexpr (ODD) {
        const char* q = reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(x) & ~uintptr_t(2));
        v = *reinterpret_cast<const u32x4_word_t*>(q);
        w = *reinterpret_cast<const uint32_t*>(q + 16);
      } else {
        v = *reinterpret_cast<const u32x4_word_t*>(x);
      }
    };
#pragma unroll
    for (int h = 0; h < 2 * UN; ++h) {
#pragma unroll
      for (int j = 0; j < FN; ++j) one(b[j] + (int64_t)c * 64 + 32 * h, fb[h][j], wb[ODD ? h : 0][j]);
#pragma unroll
      for (int i = 0; i < FM; ++i) one(a[i] + (int64_t)c * 64 + 32 * h, fa[h][i], wa[ODD ? h : 0][i]);
    }
  };
  const auto shift = [&](const uint16_t* x, u32x4_t& v, uint32_t w) {
    const uint32_t by = (uint32_t)reinterpret_cast<uintptr_t>(x) & 2;
    v = u32x4_t{__builtin_amdgcn_alignbyte(v[1], v[0], by), __builtin_amdgcn_alignbyte(v[2], v[1], by),
                __builtin_amdgcn_alignbyte(v[3], v[2], by), __builtin_amdgcn_alignbyte(w, v[3], by)};
  };
  const auto use = [&](u32x4_t (&fa)[2 * UN][FM], u32x4_t (&fb)[2 * UN][FN], const uint32_t (&wa)[W][FM], const uint32_t (&wb)[W][FN]) {
#pragma unroll
    for (int h = 0; h < 2 * UN; ++h) {
      if constexpr (ODD) {
#pragma unroll
        for (int j = 0; j < FN; ++j) shift(b[j], fb[h][j], wb[h][j]);
#pragma unroll
        for (int i = 0; i < FM; ++i) shift(a[i], fa[h][i], wa[h][i]);
      }
      multiply(fa[h], fb[h]);
    }
  };
  const int pieces = (ODD ? max(K - 2, 0) : K) / 64, groups = pieces / UN;   // the word behind lies in the row
  u32x4_t fa[2][2 * UN][FM], fb[2][2 * UN][FN];
  uint32_t wa[2][W][FM], wb[2][W][FN];
  if (wave < groups) load(wave * UN, fa[0], fb[0], wa[0], wb[0]);
  for (int c = wave; c < groups; c += 8) {
    // two groups per turn, the last one loaded again where there is none
    load((c + 4 < groups ? c + 4 : c) * UN, fa[1], fb[1], wa[1], wb[1]);
    use(fa[0], fb[0], wa[0], wb[0]);
    if (c + 4 >= groups) break;
    load((c + 8 < groups ? c + 8 : c) * UN, fa[0], fb[0], wa[0], wb[0]);
    use(fa[1], fb[1], wa[1], wb[1]);
  }
  // what is left: halves of 32 elements, shared out over the waves, those
  // past k elementwise and zero
  for (int at = groups * UN * 64 + 32 * wave; at < K; at += 128) {
    u32x4_t ta[FM], tb[FN];
    const int left = K - at - 8 * g4;
    const auto get = [&](const uint16_t* x) {
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (left >= 8) {
        v = *reinterpret_cast<const u32x4_any_t*>(x + at);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < left) v[e >> 1] |= (uint32_t)x[at + e] << (16 * (e & 1));
      }
      return v;
    };
#pragma unroll
    for (int j = 0; j < FN; ++j) tb[j] = get(b[j]);
#pragma unroll
    for (int i = 0; i < FM; ++i) ta[i] = get(a[i]);
    multiply(ta, tb);
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[wave][i][j][e][lane] = acc[i][j][e];
  __syncthreads();
  if (wave >= FM) return;
  float x[FN][4];
#pragma unroll
  for (int j = 0; j < FN; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[j][e] = part[0][wave][j][e][lane] + part[1][wave][j][e][lane] + part[2][wave][j][e][lane] + part[3][wave][j][e][lane];
  const int row = m0 + 16 * wave + i16, col = n0 + 4 * g4;
  const int64_t at = row < M ? lp.labels[row] - lp.label0 : -1;   // the label's column
  if constexpr (!GRAD) {
    float mx = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + 16 * j + e < N) mx = fmaxf(mx, x[j][e]);
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float off = finite_or_zero(mx);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (col + 16 * j + e < N) sum += exp_of(x[j][e] - off);
        if (at == col + 16 * j + e && at < N) lp.target[row] = x[j][e];
      }
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (g4 == 0 && row < M) {
      float* o = lp.stats + ((int64_t)cb * M + row) * 2;
      o[0] = mx;
      o[1] = sum;
    }
  } else {
    const f32x4_t rv = *reinterpret_cast<const f32x4_t*>(lp.rows + 4 * (int64_t)min(row, M - 1));
    const float f = (DT == kDtypeFp16 ? 16384.0f : 1.0f) / rv[3];
    const float wa = rv[1] * f, wb = rv[2] * f;
    const float power = DT == kDtypeFp16 ? rv[3] / lp.scale_all[0] : 1.0f;   // d^T's scale is one for all rows
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = col + 16 * j + e;
        v[e] = wa * exp_of(x[j][e] - rv[0]);
        if (at == c) v[e] -= wb;
        if (row >= M || c >= N) v[e] = 0.0f;
      }
      const u32x2_t w = {pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
      if (lp.d && row < M && col + 16 * j < lp.ldd)
        *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(lp.d) + (int64_t)row * lp.ldd + col + 16 * j) = w;
      if (lp.dt && row < lp.ldt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + 16 * j + e < N)
            static_cast<uint16_t*>(lp.dt)[(int64_t)(col + 16 * j + e) * lp.ldt + row] =
                DT == kDtypeFp16 ? cvt1<DT>(v[e] * power) : (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
  }
}

// Merge `parts` partial (maximum, sum) pairs of each row with the running
// ones of earlier pieces (first: none); the last piece also writes the outputs.
// ROWS rows x 256 / ROWS partials at a time; the lanes of a row in a wave merge
// by shuffles, the four waves through LDS, always in the same order.
template <int ROWS>
__global__ __launch_bounds__(256) void loss_combine_kernel(LossCombine c) {
  constexpr int LANES = 256 / ROWS;
  __shared__ float sm[4][ROWS], ss[4][ROWS];
  const int r = threadIdx.x % ROWS, l = threadIdx.x / ROWS, wave = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * ROWS + r;
  float m = -__builtin_inff(), s = 0.0f;
  const auto merge = [&](float pm, float ps) {
    const float top = fmaxf(m, pm), off = finite_or_zero(top);
    // a maximum that is not larger keeps its terms' weights exp(0) = 1
    s = s * exp_of(m - off) + ps * exp_of(pm - off);
    m = top;
  };
  // eight partials are on their way at a time
  if (row < c.m)
    for (int q0 = l; q0 < c.parts; q0 += 8 * LANES) {
      f32x2_t v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int q = q0 + e * LANES;
        v[e] = q < c.parts ? *reinterpret_cast<const f32x2_t*>(c.stats + ((int64_t)q * c.m + row) * 2)
                           : f32x2_t{-__builtin_inff(), 0.0f};
      }
      float top = v[0][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, v[e][0]);
      const float off = finite_or_zero(top);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += v[e][1] * exp_of(v[e][0] - off);
      merge(top, sum);
    }
#pragma unroll
  for (int d = ROWS; d < 64; d *= 2) merge(__shfl_xor(m, d), __shfl_xor(s, d));
  if ((threadIdx.x & 63) < ROWS) {
    sm[wave][r] = m;
    ss[wave][r] = s;
  }
  __syncthreads();
  if (l != 0 || row >= c.m) return;
#pragma unroll
  for (int q = 1; q < 4; ++q) merge(sm[q][r], ss[q][r]);
  if (!c.first) merge(c.running[2 * row], c.running[2 * row + 1]);
  if (!c.last) {
    c.running[2 * row] = m;
    c.running[2 * row + 1] = s;
    return;
  }
  const float lse = finite_or_zero(m) + __builtin_amdgcn_logf(s) * kLn2;
  const int64_t label = c.labels[row];
  const bool here = label >= c.start && label < c.start + c.n;
  const float target = here ? c.target[row] : 0.0f;
  if (!here) c.target[row] = 0.0f;
  c.lse[row] = lse;
  c.loss[row] = label == c.ignore ? 0.0f : label < 0 || label >= c.total ? __builtin_nanf("") : lse - target;
}

// a and b of a row: a = grad_loss + grad_lse (grad_lse alone for ignored rows),
// b = grad_loss.  A label outside the vocabulary makes both NaN.
__device__ __forceinline__ void row_weights(const LossRows& c, int64_t row, float& a, float& b) {
  const int64_t label = c.labels[row];
  b = label == c.ignore ? 0.0f : c.grad_loss[row];
  a = b + (c.grad_lse ? c.grad_lse[row] : 0.0f);
  if (label != c.ignore && (label < 0 || label >= c.total)) a = b = __builtin_nanf("");
}

__device__ __forceinline__ float finite_size(float x) {
  x = __builtin_fabsf(x);
  return x < __builtin_inff() ? x : 0.0f;
}

// 2^exponent of a positive normal number.
__device__ __forceinline__ float power_below(float x) {
  return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & 0x7F800000u);
}

// rows[m] = {lse, a, b, s} and scale_all = S, the scales of d: s_i d_i are the
// gradients' rows.  S is the largest |b| times the power of two that keeps
// |a| <= 2 S: where all rows weigh the same (a mean over tokens) the label's
// entry of d is exactly -1 plus its probability, instead of every row being
// off by the rounding of one and the same weight.  bf16: s_i = S.  fp16: S
// times the power of two, at most 1, that brings |a_i| + |b_i|, which bounds
// |d|, near 1: (|a_i| + |b_i|) / s_i is below 2, or, where s_i = S, at most 3,
// so that 2^14 d / s_i stays below 49152 (the type ends at 65504) whatever the
// signs of a and b.  One workgroup: the maxima are over all rows.
template <int DT>
__device__ __forceinline__ void loss_rows(const LossRows& c) {
  __shared__ float top[2][16];
  float most[2] = {0.0f, 0.0f};
  for (int64_t row = threadIdx.x; row < c.m; row += 1024) {
    float a, b;
    row_weights(c, row, a, b);
    most[0] = fmaxf(most[0], finite_size(a));
    most[1] = fmaxf(most[1], finite_size(b));
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
#pragma unroll
    for (int o = 1; o < 64; o *= 2) most[q] = fmaxf(most[q], __shfl_xor(most[q], o));
    if ((threadIdx.x & 63) == 0) top[q][threadIdx.x >> 6] = most[q];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q)
    for (int w = 0; w < 16; ++w) most[q] = fmaxf(most[q], top[q][w]);
  // 2^-100 (fp16, whose s_i may be 2^-24 S: 2^-60) and 2^100: 2^14 over any s_i is normal
  constexpr float kLow = DT == kDtypeFp16 ? 8.673617379884035e-19f : 7.888609052210118e-31f, kHigh = 1.2676506002282294e30f;
  float all = most[1] > 0.0f ? most[1] : most[0] > 0.0f ? most[0] : 1.0f;
  all = fminf(fmaxf(all, kLow), kHigh);
  const float over = most[0] / all;
  if (over > 2.0f) all = fminf(all * power_below(over), kHigh);
  if (threadIdx.x == 0) c.scale_all[0] = all;
  for (int64_t row = threadIdx.x; row < c.m; row += 1024) {
    float a, b;
    row_weights(c, row, a, b);
    float s = all;
    if constexpr (DT == kDtypeFp16) {
      const float part = finite_size(a) / all + finite_size(b) / all;
      if (part > 0.0f) s = all * fminf(fmaxf(power_below(part), 5.9604644775390625e-08f), 1.0f);   // 2^-24: a power of two in fp16
    }
    *reinterpret_cast<f32x4_t*>(c.rows + 4 * row) = f32x4_t{c.lse[row], a, b, s};
  }
}

// Rows of 16-bit elements, `cols` of each, as rows of whole 16-byte vectors:
// out[(g * rows + t) * chunks * 8 + c] = group[g][t * ld + c], zeros past cols.
// A source row may start at any element (16-byte accesses to global memory
// need no alignment); its last chunk is read element by element.
__device__ __forceinline__ void pad_chunk(const PadRows& c, int64_t u) {
  const int64_t row = u / (uint32_t)c.chunks;
  const int ch = (int)(u - row * c.chunks);
  const int64_t g = row / (uint32_t)c.rows;
  if (g >= c.num_groups) return;
  const uint16_t* src = static_cast<const uint16_t*>(c.group[g]) + (row - g * c.rows) * c.ld + ch * 8;
  const int count = (int)c.cols - ch * 8;
  u32x4_t v = {0u, 0u, 0u, 0u};
  if (count >= 8) {
    v = *reinterpret_cast<const u32x4_any_t*>(src);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < count) v[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
  }
  *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(c.out) + row * c.chunks * 8 + ch * 8) = v;
}

// The rows' weights (workgroup 0, where asked for) and the copy of A (the
// others) in one launch.  LONG: more chunks than a launch has threads, so each
// takes several (the loop alone costs a small copy 0.3 us).
template <int DT, bool ROWS, bool LONG>
__global__ __launch_bounds__(1024) void loss_prepare_kernel(LossRows r, PadRows c) {
  if (ROWS && blockIdx.x == 0) {
    loss_rows<DT>(r);
    return;
  }
  int64_t u = ((int64_t)blockIdx.x - (ROWS ? 1 : 0)) * 1024 + threadIdx.x;
  if constexpr (LONG) {
    const int64_t chunks = c.num_groups * c.rows * c.chunks, step = ((int64_t)gridDim.x - (ROWS ? 1 : 0)) * 1024;
    for (; u < chunks; u += step) pad_chunk(c, u);
  } else {
    pad_chunk(c, u);
  }
}

template <int DT>
hipError_t launch_body(const LossProblem& p, bool grad, hipStream_t s) {
  const unsigned grid = (unsigned)(p.gemm.order.num_rb * p.gemm.order.num_cb);
  if (p.tile == 256) {
    if (grad) hipLaunchKernelGGL((loss_grad_kernel<256, 256, DT, 1>), dim3(grid), dim3(256), 0, s, p);
    else hipLaunchKernelGGL((loss_stats_kernel<256, 256, DT, 1>), dim3(grid), dim3(256), 0, s, p);
  } else {
    if (grad) hipLaunchKernelGGL((loss_grad_kernel<128, 128, DT, 2>), dim3(grid), dim3(256), 0, s, p);
    else hipLaunchKernelGGL((loss_stats_kernel<128, 128, DT, 2>), dim3(grid), dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

template <int DT, int FM, int FN, int UN>
void launch_few_tile(const LossProblem& p, bool grad, unsigned grid, hipStream_t s) {
  const bool odd = p.gemm.ldb % 2 != 0 || p.gemm.rows.a_ld % 2 != 0;
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, s, p); };
  if (odd) grad ? go(loss_few_kernel<DT, FM, FN, UN, true, true>) : go(loss_few_kernel<DT, FM, FN, UN, true, false>);
  else grad ? go(loss_few_kernel<DT, FM, FN, UN, false, true>) : go(loss_few_kernel<DT, FM, FN, UN, false, false>);
}

template <int DT>
hipError_t launch_few(const LossProblem& p, int fm, int fn, bool grad, unsigned grid, hipStream_t s) {
  if (fm == 1 && fn == 1) launch_few_tile<DT, 1, 1, 4>(p, grad, grid, s);
  else if (fm == 1) launch_few_tile<DT, 1, 4, 2>(p, grad, grid, s);
  else if (fn == 1) launch_few_tile<DT, 4, 1, 2>(p, grad, grid, s);
  else launch_few_tile<DT, 4, 4, 1>(p, grad, grid, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_loss_logits(const LossProblem& p, int dtype, bool grad, hipStream_t stream) {
  const int t = p.tile;
  if ((t != 256 && t != 128) || p.gemm.order.num_rb != (p.gemm.m + t - 1) / t ||
      p.gemm.order.num_cb != (p.gemm.n + t - 1) / t ||
      (int64_t)p.gemm.order.num_rb * p.gemm.order.num_cb >= kLossGrid || p.gemm.k % 8 != 0)
    return hipErrorInvalidValue;
  return dtype == kDtypeBf16 ? launch_body<kDtypeBf16>(p, grad, stream)
       : dtype == kDtypeFp16 ? launch_body<kDtypeFp16>(p, grad, stream) : hipErrorInvalidValue;
}

hipError_t launch_loss_few(const LossProblem& p, int fm, int fn, int dtype, bool grad, hipStream_t stream) {
  const int64_t grid = (int64_t)p.gemm.order.num_rb * p.gemm.order.num_cb;
  if ((fm != 1 && fm != 4) || (fn != 1 && fn != 4) || p.gemm.order.num_rb != (p.gemm.m + 16 * fm - 1) / (16 * fm) ||
      p.gemm.order.num_cb != (p.gemm.n + 16 * fn - 1) / (16 * fn) || grid < 1 || grid >= kLossGrid ||
      (dtype != kDtypeBf16 && dtype != kDtypeFp16) || (int64_t)p.gemm.rows.num_groups * p.gemm.rows.rows_per_group != p.gemm.m ||
      (grad && (p.ldd % 8 != 0 || p.ldt % 8 != 0)))
    return hipErrorInvalidValue;
  return dtype == kDtypeBf16 ? launch_few<kDtypeBf16>(p, fm, fn, grad, (unsigned)grid, stream)
                             : launch_few<kDtypeFp16>(p, fm, fn, grad, (unsigned)grid, stream);
}

hipError_t launch_loss_combine(const LossCombine& c, hipStream_t stream) {
  // few rows: more lanes share a row's partials
  if (c.m <= 256) hipLaunchKernelGGL((loss_combine_kernel<1>), dim3((unsigned)c.m), dim3(256), 0, stream, c);
  else hipLaunchKernelGGL((loss_combine_kernel<16>), dim3((unsigned)((c.m + 15) / 16)), dim3(256), 0, stream, c);
  return hipGetLastError();
}

constexpr int64_t kCopyGroups = 1 << 14;

hipError_t launch_loss_prepare(const LossRows* r, const PadRows* c, int dtype, hipStream_t stream) {
  int64_t copies = 0;
  if (c) {
    if (c->rows < 1 || c->rows > INT32_MAX || c->chunks < 1 || c->chunks > INT32_MAX || c->cols <= (c->chunks - 1) * 8 ||
        c->cols > c->chunks * 8 || c->num_groups < 1 || c->num_groups > kMaxGroups)
      return hipErrorInvalidValue;
    // beyond 2^14 workgroups (256 MiB) each copies several pieces: any size fits a launch
    copies = (c->num_groups * c->rows * c->chunks + 1023) / 1024;
    copies = copies < kCopyGroups ? copies : kCopyGroups;
  }
  const int64_t grid = copies + (r ? 1 : 0);
  if (grid < 1) return hipErrorInvalidValue;
  const PadRows none{};
  const LossRows no_rows{};
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(1024), 0, stream, r ? *r : no_rows, c ? *c : none);
  };
  const bool half = dtype == kDtypeFp16, more = copies == kCopyGroups;
  if (!r) more ? go(loss_prepare_kernel<kDtypeBf16, false, true>) : go(loss_prepare_kernel<kDtypeBf16, false, false>);
  else if (half) more ? go(loss_prepare_kernel<kDtypeFp16, true, true>) : go(loss_prepare_kernel<kDtypeFp16, true, false>);
  else more ? go(loss_prepare_kernel<kDtypeBf16, true, true>) : go(loss_prepare_kernel<kDtypeBf16, true, false>);
  return hipGetLastError();
}

}  // namespace agmm
