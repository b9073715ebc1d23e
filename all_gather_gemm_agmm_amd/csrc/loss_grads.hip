// Vocabulary loss, the two gradient products (gfx950), on the 16-bit
// d[i, v] that loss_grad_kernel leaves:
//
//     dA[i, :] = s_i * sum_v d[i, v] * W[v, :]         (rows of d, W k x n as stored)
//     dW[v, :] = S   * sum_i dt[v, i] * A[i, :]        (d transposed, A k x n as gathered)
//
// Both are the part-ring GEMM (gemm_m16_loop.inc) with B stored k x n.  dA is
// summed over the pieces of the vocabulary (and over ranges of a piece where
// few output tiles would leave CUs idle) in fp32 sums [range][m][k] that
// each piece adds to in place, in order; one last pass adds the ranges, scales
// and casts.  dW of a piece is complete at once.  Bound: MFMA.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "agmm_kernels.h"
#include "gemm_device.h"

namespace agmm {

namespace {

// SPLIT: fp32 sums of range `split` into p.partials, added to what is there
// when `add`; else C = scale * sums.
template <int BM, int BN, int BK, int DT, bool SPLIT, int WAVES, int OCC>
__device__ __forceinline__ void grad_body(const GemmProblem& p, bool add, const float* scale, char* smem) {
  constexpr bool BT = false;
  using T = GemmTile<BM, BN, BK, DT, BT, 5, WAVES, kLoopParts>;
  constexpr int kBK = BK;
  constexpr int FM = T::TM / 16, FN = T::TN / 16;
  constexpr int STEPS = BK / 32;

#include "gemm_m16_loop.inc"

  if constexpr (SPLIT) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int row = m0 + wm * T::TM + 16 * i + i16;
      if (row >= M) continue;
      float* d = p.partials + ((int64_t)split * M + row) * N;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int col = n0 + wn * T::TN + 16 * j + 4 * g4;
        if (col + 3 < N && N % 4 == 0) {
          f32x4_t* q = reinterpret_cast<f32x4_t*>(d + col);
          *q = add ? *q + acc[i][j] : acc[i][j];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col + e < N) d[col + e] = add ? d[col + e] + acc[i][j][e] : acc[i][j][e];
        }
      }
    }
  } else {
    const float f = scale[0] * (DT == kDtypeFp16 ? 1.0f / 16384.0f : 1.0f);
    // whole rows through LDS, as in gemm_m16_kernel
    constexpr int kRowB = BN * 2, kChunks = kRowB / 16;
    const bool staged = m0 + BM <= M && n0 + BN <= N && p.ldc % 8 == 0 && (reinterpret_cast<uintptr_t>(p.c) & 15) == 0;
    if (staged) __syncthreads();
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = wm * T::TM + 16 * i + i16;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int c = wn * T::TN + 16 * j + 4 * g4;
        const f32x4_t v = acc[i][j] * f;
        if (staged) {
          *reinterpret_cast<u32x2_t*>(smem + r * kRowB + (((c >> 3) ^ (r & (kChunks - 1))) << 4) + (c & 4) * 2) =
              u32x2_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
        } else if (m0 + r < M) {
          uint16_t* d = static_cast<uint16_t*>(p.c) + (int64_t)(m0 + r) * p.ldc + n0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n0 + c + e < N) d[c + e] = cvt1<DT>(v[e]);
        }
      }
    }
    if (staged) {
      __syncthreads();
      for (int u = tid; u < BM * kChunks; u += T::THREADS) {
        const int r = u / kChunks, c = u % kChunks;
        __builtin_nontemporal_store(
            *reinterpret_cast<const u32x4_t*>(smem + r * kRowB + ((c ^ (r & (kChunks - 1))) << 4)),
            reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p.c) + (int64_t)(m0 + r) * p.ldc + n0 + c * 8));
      }
    }
  }
}

template <int BM, int BN, int DT, int OCC>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
void loss_da_kernel(GemmProblem p, int add) {
  __shared__ __attribute__((aligned(1024))) char smem[GemmTile<BM, BN, 64, DT, false, 5, 4, kLoopParts>::LDS_BYTES];
  grad_body<BM, BN, 64, DT, true, 4, OCC>(p, add != 0, nullptr, smem);
}

template <int BM, int BN, int DT, int OCC>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
void loss_dw_kernel(GemmProblem p, const float* scale) {
  __shared__ __attribute__((aligned(1024))) char smem[GemmTile<BM, BN, 64, DT, false, 5, 4, kLoopParts>::LDS_BYTES];
  grad_body<BM, BN, 64, DT, false, 4, OCC>(p, false, scale, smem);
}

// dA = s_i * (sum of the ranges in order), cast.  Four columns per thread.
template <int DT>
__global__ __launch_bounds__(256) void loss_da_finish_kernel(LossFinish c) {
  const int n4 = (c.k + 3) / 4;
  const int64_t plane = c.m * (int64_t)c.k;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < c.m * n4; u += (int64_t)gridDim.x * 256) {
    const int64_t row = u / n4;
    const int col = (int)(u % n4) * 4;
    const float* src = c.sums + row * c.k + col;
    const float f = c.rows[4 * row + 3] * (DT == kDtypeFp16 ? 1.0f / 16384.0f : 1.0f);
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    if (c.k % 4 == 0) {
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
    } else {
      for (int q = 0; q < c.ranges; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < c.k) v[e] += src[q * plane + e];
    }
    v *= f;
    uint16_t* d = static_cast<uint16_t*>(c.da) + row * c.ldda + col;
    if (c.k % 4 == 0 && c.ldda % 4 == 0) {
      *reinterpret_cast<u32x2_t*>(d) = u32x2_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
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
         (int64_t)p.order.num_rb * p.order.num_cb * p.splits < (int64_t(1) << 24);
}

}  // namespace

hipError_t launch_loss_da(const GemmProblem& p, int tile, int dtype, bool add, hipStream_t s) {
  if (!fits(p, tile) || !p.partials) return hipErrorInvalidValue;
  const dim3 grid((unsigned)(p.order.num_rb * p.order.num_cb * p.splits));
  if (tile == 256) {
    if (dtype == kDtypeBf16) hipLaunchKernelGGL((loss_da_kernel<256, 256, kDtypeBf16, 1>), grid, dim3(256), 0, s, p, (int)add);
    else hipLaunchKernelGGL((loss_da_kernel<256, 256, kDtypeFp16, 1>), grid, dim3(256), 0, s, p, (int)add);
  } else {
    if (dtype == kDtypeBf16) hipLaunchKernelGGL((loss_da_kernel<128, 128, kDtypeBf16, 2>), grid, dim3(256), 0, s, p, (int)add);
    else hipLaunchKernelGGL((loss_da_kernel<128, 128, kDtypeFp16, 2>), grid, dim3(256), 0, s, p, (int)add);
  }
  return hipGetLastError();
}

hipError_t launch_loss_dw(const GemmProblem& p, int tile, int dtype, const float* scale, hipStream_t s) {
  if (!fits(p, tile) || p.splits != 1 || !scale) return hipErrorInvalidValue;
  const dim3 grid((unsigned)(p.order.num_rb * p.order.num_cb));
  if (tile == 256) {
    if (dtype == kDtypeBf16) hipLaunchKernelGGL((loss_dw_kernel<256, 256, kDtypeBf16, 1>), grid, dim3(256), 0, s, p, scale);
    else hipLaunchKernelGGL((loss_dw_kernel<256, 256, kDtypeFp16, 1>), grid, dim3(256), 0, s, p, scale);
  } else {
    if (dtype == kDtypeBf16) hipLaunchKernelGGL((loss_dw_kernel<128, 128, kDtypeBf16, 2>), grid, dim3(256), 0, s, p, scale);
    else hipLaunchKernelGGL((loss_dw_kernel<128, 128, kDtypeFp16, 2>), grid, dim3(256), 0, s, p, scale);
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
