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
//    dA = d W and transposed [v][i] for dW = d^T A.  a_i and b_i are scaled by
//    powers of two (exact): by rows to [1, 2), undone on dA's fp32 sums;
//    transposed to the largest row's, undone on dW's.  fp16 also carries 2^14,
//    so that a probability of 2^-28 is still a normal number.  Rounding d
//    to 16 bits (the operands' own precision) is what lets the matrix cores
//    compute both gradients; the sums are fp32.
//
// Bound: MFMA.  The exponentials cost 256 (256 x 256 tile) per lane once per
// tile, 3-5% beside the k loop of a 4096-deep product.
//
// The maximum uses v_max, which passes over NaN, but a NaN logit makes its
// sum NaN, so a row with one has a NaN loss.  Infinite maxima are replaced
// by 0 inside exp: a row of -inf only gives lse = -inf, one with +inf gives +inf.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "agmm_kernels.h"
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
    const float top = DT == kDtypeFp16 ? 16384.0f : 1.0f;
    const float inv_all = top / lp.scale_all[0];
    // the rows' values, all on their way at once
    f32x4_t rv[FM];
    int at[FM];       // the label's column within the wave's, or anything outside
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int row = m0 + wm * T::TM + 16 * i + i16;
      rv[i] = row < M ? *reinterpret_cast<const f32x4_t*>(lp.rows + 4 * (int64_t)row) : f32x4_t{0.f, 0.f, 0.f, 1.f};
      const int64_t rel = row < M ? lp.labels[row] - lp.label0 - wcol : -1;
      at[i] = rel >= 0 && rel < T::TN ? (int)rel : -1;
    }
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = exp_of(acc[i][j][e] - rv[i][0]);
    __syncthreads();   // the LDS now holds the output tiles
    // Row by row: chunk c (16 bytes) of tile row r at c ^ (r mod 8), as 4
    // columns of a row are 8 bytes; transposed: columns are rows of BM elements.
    constexpr int RB = BN * 2, TB = BM * 2;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      if (!(pass ? lp.dt : lp.d)) continue;
      if (pass) __syncthreads();   // the row-major tile has been read
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int r = wm * T::TM + 16 * i + i16;
        const int row = m0 + r;
        const bool in = row < M;
        const float f = pass ? inv_all : top / rv[i][3];
        const float af = rv[i][1] * f, bf = rv[i][2] * f;
        const bool hit = __any(at[i] >= 0);
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          float d[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] = af * acc[i][j][e];
          if (hit)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (at[i] == 16 * j + 4 * g4 + e) d[e] -= bf;
          if (!whole)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!in || wcol + 16 * j + 4 * g4 + e >= N) d[e] = 0.0f;
          const int c = wn * T::TN + 16 * j + 4 * g4;
          if (pass == 0) {
            *reinterpret_cast<u32x2_t*>(smem + r * RB + (((c >> 3) ^ (r & 7)) << 4) + (c & 4) * 2) =
                u32x2_t{pack2<DT>(d[0], d[1]), pack2<DT>(d[2], d[3])};
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint16_t*>(smem + (c + e) * TB + (((r >> 3) ^ (((c >> 2) & 3) * 2)) << 4) + (r & 7) * 2) =
                  cvt1<DT>(d[e]);
          }
        }
      }
      __syncthreads();
      if (pass == 0) {
        constexpr int CH = RB / 16;
        for (int u = tid; u < BM * CH; u += T::THREADS) {
          const int r = u / CH, c = u % CH;
          if (m0 + r < M && n0 + c * 8 < lp.ldd)
            *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(lp.d) + (int64_t)(m0 + r) * lp.ldd + n0 + c * 8) =
                *reinterpret_cast<const u32x4_t*>(smem + r * RB + ((c ^ (r & 7)) << 4));
        }
      } else {
        constexpr int CH = TB / 16;
        for (int u = tid; u < BN * CH; u += T::THREADS) {
          const int v = u / CH, c = u % CH;
          if (n0 + v < N && m0 + c * 8 < lp.ldt)
            *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(lp.dt) + (int64_t)(n0 + v) * lp.ldt + m0 + c * 8) =
                *reinterpret_cast<const u32x4_t*>(smem + v * TB + ((c ^ (((v >> 2) & 3) * 2)) << 4));
        }
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

// Merge `parts` partial (maximum, sum) pairs of each row with the running
// ones of earlier pieces (first: none); the last piece also writes the outputs.
// ROWS rows x 256 / ROWS partials at a time.
template <int ROWS>
__global__ __launch_bounds__(256) void loss_combine_kernel(LossCombine c) {
  constexpr int LANES = 256 / ROWS;
  __shared__ float sm[LANES][ROWS], ss[LANES][ROWS];
  const int r = threadIdx.x % ROWS, l = threadIdx.x / ROWS;
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
  sm[l][r] = m;
  ss[l][r] = s;
  __syncthreads();
  if (l != 0 || row >= c.m) return;
  for (int q = 1; q < LANES; ++q) merge(sm[q][r], ss[q][r]);
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

// Per row {lse, a, b, s}: a = grad_loss + grad_lse (0 and grad_lse for ignored
// rows), b = grad_loss, s the power of two that brings the larger of them to
// [1, 2); scale_all = max s.  A label outside the vocabulary makes a and b NaN.
// One workgroup: the maximum is over all rows.
__global__ __launch_bounds__(1024) void loss_rows_kernel(LossRows c) {
  __shared__ float top[16];
  float most = 0.0f;
  for (int64_t row = threadIdx.x; row < c.m; row += 1024) {
    const int64_t label = c.labels[row];
    float b = label == c.ignore ? 0.0f : c.grad_loss[row];
    float a = b + (c.grad_lse ? c.grad_lse[row] : 0.0f);
    if (label != c.ignore && (label < 0 || label >= c.total)) a = b = __builtin_nanf("");
    const float big = fmaxf(__builtin_fabsf(a), __builtin_fabsf(b));
    // 2^exponent, kept within [2^-100, 2^100] so that it and its inverse are normal
    uint32_t e = __builtin_bit_cast(uint32_t, big) & 0x7F800000u;
    float s = 1.0f;
    if (big > 0.0f && e < 0x7F800000u) {
      e = min(max(e, 27u << 23), 227u << 23);
      s = __builtin_bit_cast(float, e);
      most = fmaxf(most, s);
    }
    float* d = c.rows + 4 * row;
    d[0] = c.lse[row];
    d[1] = a;
    d[2] = b;
    d[3] = s;
  }
#pragma unroll
  for (int o = 1; o < 64; o *= 2) most = fmaxf(most, __shfl_xor(most, o));
  if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 16; ++w) most = fmaxf(most, top[w]);
    c.scale_all[0] = most > 0.0f ? most : 1.0f;
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

}  // namespace

hipError_t launch_loss_logits(const LossProblem& p, int dtype, bool grad, hipStream_t stream) {
  const int t = p.tile;
  if ((t != 256 && t != 128) || p.gemm.order.num_rb != (p.gemm.m + t - 1) / t ||
      p.gemm.order.num_cb != (p.gemm.n + t - 1) / t ||
      (int64_t)p.gemm.order.num_rb * p.gemm.order.num_cb >= (int64_t(1) << 24) || p.gemm.k % 8 != 0)
    return hipErrorInvalidValue;
  return dtype == kDtypeBf16 ? launch_body<kDtypeBf16>(p, grad, stream)
       : dtype == kDtypeFp16 ? launch_body<kDtypeFp16>(p, grad, stream) : hipErrorInvalidValue;
}

hipError_t launch_loss_combine(const LossCombine& c, hipStream_t stream) {
  // few rows: more lanes share a row's partials
  if (c.m <= 64) hipLaunchKernelGGL((loss_combine_kernel<4>), dim3((unsigned)((c.m + 3) / 4)), dim3(256), 0, stream, c);
  else hipLaunchKernelGGL((loss_combine_kernel<16>), dim3((unsigned)((c.m + 15) / 16)), dim3(256), 0, stream, c);
  return hipGetLastError();
}

hipError_t launch_loss_rows(const LossRows& c, hipStream_t stream) {
  hipLaunchKernelGGL(loss_rows_kernel, dim3(1), dim3(1024), 0, stream, c);
  return hipGetLastError();
}

}  // namespace agmm
