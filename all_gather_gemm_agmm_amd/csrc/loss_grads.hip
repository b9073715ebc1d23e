// Vocabulary loss, the two gradient products (gfx950), on the 16-bit
// d[i, v] that loss_grad_kernel leaves:
//
//     dA[i, :] = s_i * sum_v d[i, v] * W[v, :]         (rows of d, W k x n as stored)
//     dW[v, :] = S   * sum_i dt[v, i] * A[i, :]        (d transposed, all over S; A k x n as gathered)
//
// Both are the part-ring GEMM (gemm_m16_loop.inc) with B stored k x n, and
// share a launch: with few rows neither fills the CUs alone.  dA is summed
// over the pieces of the vocabulary (and over ranges of a piece where few
// output tiles would leave CUs idle) in fp32 sums [range][m][k] that each
// piece adds to in place, in order; one last pass adds the ranges, scales and
// casts.  dW of a piece is complete at once.
//
// Bound: MFMA; with few rows the stores of dW.  Measured: 8192 x 4096 bf16 over
// 16384 columns, both products 1.48-1.57 ms, 1400-1490 TFLOP/s; 16 x 4096 over 65536
// 286 us, 1.07 GB of W read and dW written: 3.8 TB/s; 30 x 500 over 50000 38 us
// (80 with 256 x 256 tiles and dW, whose rows are then not whole 16-byte
// vectors, stored by elements).  The last pass: 8192 x 4096 37-40 us, 5.0-5.4 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_kernels.h"
#include "gemm_device.h"

namespace agmm {

namespace {

// Vectors of 16-bit results in global memory: element alignment only.
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
typedef u32x2_t u32x2_any_t __attribute__((aligned(2)));

struct GradPair {
  GemmProblem a, w;        // dA and dW
  int32_t a_tiles;         // workgroups of dA: the first ones
  int32_t add;             // dA: add to the sums that are there
  const float* scale;      // dW: its factor
};

template <int BM, int BN, int DT, int OCC>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
void loss_grads_kernel(GradPair gp) {
  constexpr bool BT = false, SPLIT = true;
  constexpr int BK = 64, WAVES = 4;
  using T = GemmTile<BM, BN, BK, DT, BT, 5, WAVES, kLoopParts>;
  constexpr int kBK = BK;
  constexpr int FM = T::TM / 16, FN = T::TN / 16;
  constexpr int STEPS = BK / 32;
  __shared__ __attribute__((aligned(1024))) char smem[T::LDS_BYTES];
  const bool is_a = (int)blockIdx.x < gp.a_tiles;
  const GemmProblem& p = is_a ? gp.a : gp.w;

#define AGMM_TILE_ID (is_a ? (int)blockIdx.x : (int)blockIdx.x - gp.a_tiles)
#include "gemm_m16_loop.inc"

  if (is_a) {
    // rows of the sums are whole 16-byte vectors; what lies past k in the last
    // one is never used
    const int row0 = m0 + wm * T::TM + i16, col0 = n0 + wn * T::TN + 4 * g4;
    const int64_t ld = (N + 3) & ~3;
    float* base = p.partials + ((int64_t)split * M + row0) * ld + col0;
#pragma unroll
    for (int i = 0; i < FM; ++i, base += 16 * ld) {
      if (row0 + 16 * i < M) {
        if (gp.add) {
          f32x4_t was[FN];
#pragma unroll
          for (int j = 0; j < FN; ++j)
            if (col0 + 16 * j < N) was[j] = *reinterpret_cast<const f32x4_t*>(base + 16 * j);
#pragma unroll
          for (int j = 0; j < FN; ++j)
            if (col0 + 16 * j < N) *reinterpret_cast<f32x4_t*>(base + 16 * j) = was[j] + acc[i][j];
        } else {
#pragma unroll
          for (int j = 0; j < FN; ++j)
            if (col0 + 16 * j < N) *reinterpret_cast<f32x4_t*>(base + 16 * j) = acc[i][j];
        }
      }
      __builtin_amdgcn_sched_barrier(0);   // one block row's values at a time
    }
  } else {
    const float f = gp.scale[0] * (DT == kDtypeFp16 ? 1.0f / 16384.0f : 1.0f);
    // whole rows through LDS
    constexpr int RB = BN * 2, CH = RB / 16;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = wm * T::TM + i * 16 + i16;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int c = wn * T::TN + j * 16 + 4 * g4;
        const f32x4_t v = acc[i][j] * f;
        *reinterpret_cast<u32x2_t*>(smem + r * RB + (((c >> 3) ^ (r & (CH - 1))) << 4) + (c & 4) * 2) =
            u32x2_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
      }
    }
    __syncthreads();
    constexpr int ROWS = T::THREADS / CH;
    const int c = tid % CH, left = N - (n0 + c * 8);   // columns from this lane's chunk on
    uint16_t* out = static_cast<uint16_t*>(p.c) + (int64_t)m0 * p.ldc + n0 + c * 8;
#pragma unroll 8
    for (int r = tid / CH; r < BM; r += ROWS) {
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(smem + r * RB + ((c ^ (r & (CH - 1))) << 4));
      uint16_t* d = out + (int64_t)r * p.ldc;
      if (m0 + r >= M) continue;
      if (left >= 8) {
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any_t*>(d));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < left) d[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

// dA = s_i * (sum of the ranges in order), cast.  Four columns per thread.
template <int DT>
__global__ __launch_bounds__(256) void loss_da_finish_kernel(LossFinish c) {
  const int n4 = (c.k + 3) / 4;
  const int64_t plane = c.m * (int64_t)n4 * 4;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < c.m * n4; u += (int64_t)gridDim.x * 256) {
    const int64_t row = u / n4;
    const int col = (int)(u - row * n4) * 4;
    const float* src = c.sums + u * 4;
    const float f = c.rows[4 * row + 3] * (DT == kDtypeFp16 ? 1.0f / 16384.0f : 1.0f);
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    // eight ranges are on their way at a time, added in order
    for (int q0 = 0; q0 < c.ranges; q0 += 8) {
      f32x4_t w[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q0 + q < c.ranges) w[q] = *reinterpret_cast<const f32x4_t*>(src + (q0 + q) * plane);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q0 + q < c.ranges) v += w[q];
    }
    v *= f;
    uint16_t* d = static_cast<uint16_t*>(c.da) + row * c.ldda + col;
    if (col + 4 <= c.k) {
      *reinterpret_cast<u32x2_any_t*>(d) = u32x2_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < c.k) d[e] = cvt1<DT>(v[e]);
    }
  }
}

bool fits(const GemmProblem& p, int tile) {
  return (tile == 256 || tile == 128) && p.order.num_rb == (p.m + tile - 1) / tile &&
         p.order.num_cb == (p.n + tile - 1) / tile && p.splits >= 1 && p.k_per_split % 64 == 0 &&
         (int64_t)p.splits * p.k_per_split >= p.k && (int64_t)(p.splits - 1) * p.k_per_split < p.k &&
         (int64_t)p.order.num_rb * p.order.num_cb * p.splits < kLossGrid;
}

}  // namespace

hipError_t launch_loss_grads(const GemmProblem* a, bool add, const GemmProblem* w, const float* scale, int tile, int dtype,
                             hipStream_t s) {
  if ((!a && !w) || (a && (!fits(*a, tile) || !a->partials)) || (w && (!fits(*w, tile) || w->splits != 1 || !scale)))
    return hipErrorInvalidValue;
  GradPair gp{};
  int64_t grid = 0;
  if (a) {
    gp.a = *a;
    grid += (int64_t)a->order.num_rb * a->order.num_cb * a->splits;
  }
  gp.a_tiles = (int32_t)grid;
  gp.add = add;
  if (w) {
    gp.w = *w;
    grid += (int64_t)w->order.num_rb * w->order.num_cb;
  }
  gp.scale = scale;
  if (grid >= kLossGrid) return hipErrorInvalidValue;
  if (tile == 256) {
    if (dtype == kDtypeBf16) hipLaunchKernelGGL((loss_grads_kernel<256, 256, kDtypeBf16, 1>), dim3((unsigned)grid), dim3(256), 0, s, gp);
    else hipLaunchKernelGGL((loss_grads_kernel<256, 256, kDtypeFp16, 1>), dim3((unsigned)grid), dim3(256), 0, s, gp);
  } else {
    if (dtype == kDtypeBf16) hipLaunchKernelGGL((loss_grads_kernel<128, 128, kDtypeBf16, 2>), dim3((unsigned)grid), dim3(256), 0, s, gp);
    else hipLaunchKernelGGL((loss_grads_kernel<128, 128, kDtypeFp16, 2>), dim3((unsigned)grid), dim3(256), 0, s, gp);
  }
  return hipGetLastError();
}

hipError_t launch_loss_da_finish(const LossFinish& c, int dtype, hipStream_t s) {
  const int64_t blocks = (c.m * ((c.k + 3) / 4) + 255) / 256;
  const dim3 grid((unsigned)(blocks < (1 << 16) ? blocks : (1 << 16)));
  if (dtype == kDtypeBf16) hipLaunchKernelGGL((loss_da_finish_kernel<kDtypeBf16>), grid, dim3(256), 0, s, c);
  else hipLaunchKernelGGL((loss_da_finish_kernel<kDtypeFp16>), grid, dim3(256), 0, s, c);
  return hipGetLastError();
}

}  // namespace agmm
