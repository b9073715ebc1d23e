// The way back through the product with an epilogue and the gated product, the
// two products (gfx950), on the 16-bit d that feed_d_kernel leaves:
//
//     dA = d W        (rows of d [m][parts * n], W k x n as stored)
//     dW = d^T A      (d transposed [parts * n][m], A k x n: gathered, or, where the
//                      shards' rows are whole k-tiles, in the shards)
//     db = sums of the column sums that feed_d_kernel leaves
//
// The products are the part-ring GEMM (gemm_m16_loop.inc) with B stored k x n
// and share a launch: with few rows neither fills the CUs alone.  Where few output
// tiles would leave CUs idle, a product's sum is cut into ranges, whose fp32
// sums a last pass adds in order and rounds; otherwise the tile is rounded and
// stored here, whole rows through LDS.  The product with the longer sum begins
// first, so that the last round's tiles are the short ones.
//
// Bound: MFMA (power).  Measured, rows x k -> columns: 8192 x 8192 -> 2 x 3584
// bf16 1376-1428 us, 1350-1400 TFLOP/s, 1920 tiles of 256 x 256, seven and a half
// rounds; 2048 x 4096 -> 1024 bf16 38, 256 tiles of 128 x 128 of dW
// and then 512 of dA, whose sums are half as long; 111 x 1000 -> 2 x 2051 fp16 12 and 3-4 for the ranges.
#include "feed_device.h"

namespace agmm {

namespace {

// out[c] = sum over groups, in a fixed order, of sums[group][c], rounded.
template <int DT>
__device__ __forceinline__ void bias_sums(const FeedBias& b, int64_t block, float (&part)[4][64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = block * 64 + lane;
  float t = 0.0f;
  if (col < b.cols) {
    int64_t g = wave;
    for (; g + 28 < b.groups; g += 32) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = b.sums[(g + 4 * q) * b.cols + col];
#pragma unroll
      for (int q = 0; q < 8; ++q) t += v[q];
    }
    for (; g < b.groups; g += 4) t += b.sums[g * b.cols + col];
  }
  part[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && col < b.cols)
    static_cast<uint16_t*>(b.out)[col] = cvt1<DT>((part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]));
}

template <int BM, int BN, int DT, int OCC>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
void feed_grads_kernel(FeedGrads gp) {
  constexpr bool BT = false, SPLIT = true;
  constexpr int BK = 64, WAVES = 4;
  using T = GemmTile<BM, BN, BK, DT, BT, 5, WAVES, kLoopParts>;
  constexpr int kBK = BK;
  constexpr int FM = T::TM / 16, FN = T::TN / 16;
  constexpr int STEPS = BK / 32;
  __shared__ __attribute__((aligned(1024))) char smem[T::LDS_BYTES];
  if ((int)blockIdx.x >= gp.tiles) {
    bias_sums<DT>(gp.bias, (int)blockIdx.x - gp.tiles, *reinterpret_cast<float(*)[4][64]>(smem));
    return;
  }
  const bool is_a = (int)blockIdx.x >= gp.a_first && (int)blockIdx.x < gp.a_first + gp.a_tiles;
  const GemmProblem& p = is_a ? gp.a : gp.w;

#define AGMM_CLAMP
#define AGMM_B_GROUPS gp.w_group
#define AGMM_B_GROUP_ROWS (is_a ? 0 : gp.w_rows)
#define AGMM_TILE_ID ((int)blockIdx.x - (is_a ? gp.a_first : gp.a_first ? 0 : gp.a_tiles))
#include "gemm_m16_loop.inc"

  if (p.splits > 1) {
    // rows of the sums are whole 16-byte vectors; what lies past n in the last
    // one is never used
    const int out_row = m0 + wm * T::TM + i16, out_col = n0 + wn * T::TN + 4 * g4;
    const int64_t ld = (N + 3) & ~3;
    float* base = p.partials + ((int64_t)split * M + out_row) * ld + out_col;
#pragma unroll
    for (int i = 0; i < FM; ++i, base += 16 * ld) {
      if (out_row + 16 * i < M)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          if (out_col + 16 * j < N) *reinterpret_cast<f32x4_t*>(base + 16 * j) = acc[i][j];
      __builtin_amdgcn_sched_barrier(0);   // one block row's values at a time
    }
  } else {
    constexpr int RB = BN * 2, CH = RB / 16;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = wm * T::TM + i * 16 + i16;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int c = wn * T::TN + j * 16 + 4 * g4;
        const f32x4_t v = acc[i][j];
        *reinterpret_cast<u32x2_t*>(smem + r * RB + (((c >> 3) ^ (r & (CH - 1))) << 4) + (c & 4) * 2) =
            u32x2_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
      }
    }
    __syncthreads();
    constexpr int ROWS = T::THREADS / CH;
    const int c = tid % CH, left = N - (n0 + c * 8);   // columns from this lane's piece on
    uint16_t* out = static_cast<uint16_t*>(p.c) + (int64_t)m0 * p.ldc + n0 + c * 8;
#pragma unroll 8
    for (int r = tid / CH; r < BM; r += ROWS) {
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(smem + r * RB + ((c ^ (r & (CH - 1))) << 4));
      uint16_t* d = out + (int64_t)r * p.ldc;
      if (m0 + r >= M) continue;
      if (left >= 8) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any_t*>(d));
      else store8(d, v, left);
    }
  }
}

bool fits(const GemmProblem& p, int tile) {
  return (tile == 256 || tile == 128) && p.order.num_rb == (p.m + tile - 1) / tile &&
         p.order.num_cb == (p.n + tile - 1) / tile && p.splits >= 1 && p.k_per_split % 64 == 0 &&
         (int64_t)p.splits * p.k_per_split >= p.k && (int64_t)(p.splits - 1) * p.k_per_split < p.k &&
         (p.splits == 1 || p.partials) && (int64_t)p.order.num_rb * p.order.num_cb * p.splits < kFeedGrid;
}

}  // namespace

hipError_t launch_feed_grads(FeedGrads gp, int tile, int dtype, hipStream_t s) {
  const bool a = gp.a.m > 0, w = gp.w.m > 0, bias = gp.bias.out != nullptr;
  if ((!a && !w && !bias) || (a && !fits(gp.a, tile)) || (w && !fits(gp.w, tile)) ||
      (w && gp.w_rows && (gp.w_rows % 64 != 0 || gp.w.k % gp.w_rows != 0 || gp.w.k / gp.w_rows > kMaxGroups)))
    return hipErrorInvalidValue;
  const int64_t a_tiles = a ? (int64_t)gp.a.order.num_rb * gp.a.order.num_cb * gp.a.splits : 0;
  const int64_t w_tiles = w ? (int64_t)gp.w.order.num_rb * gp.w.order.num_cb * gp.w.splits : 0;
  int64_t grid = a_tiles + w_tiles;
  gp.a_tiles = (int32_t)a_tiles;
  // the longer sums begin first, the others fill what they leave
  gp.a_first = a && w && gp.w.k_per_split > gp.a.k_per_split ? (int32_t)w_tiles : 0;
  gp.tiles = (int32_t)grid;
  if (bias) grid += (gp.bias.cols + 63) / 64;
  if (grid >= kFeedGrid) return hipErrorInvalidValue;
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(256), 0, s, gp); };
  if (dtype == kDtypeBf16) tile == 256 ? go(feed_grads_kernel<256, 256, kDtypeBf16, 1>) : go(feed_grads_kernel<128, 128, kDtypeBf16, 2>);
  else if (dtype == kDtypeFp16) tile == 256 ? go(feed_grads_kernel<256, 256, kDtypeFp16, 1>) : go(feed_grads_kernel<128, 128, kDtypeFp16, 2>);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace agmm
