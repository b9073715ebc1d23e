// Product with an epilogue, and the gated product: large tiles (gfx950).
//
//     p = A B^T + bias,  y = act(p) + residual      or, gated,  y = act(p_0) * p_1
//
// A tile is one of the part-ring GEMM (gemm_m16_loop.inc), 256 x 256 or 128 x
// 128 tile columns.  Gated, the tile's columns are blocks of 16 rows of the
// first n rows of B and 16 of the second n in turn, so that both parts of a
// column of y are in the tile: one launch instead of two products and an
// elementwise kernel that reads and writes both.
//
// The finished sums go through LDS in fp32 (the 256 x 256 tile in two halves of
// 128 KiB) to a thread per eight columns of a row, in loops that are not
// unrolled over the tile: bias, activation, product and residual are fp32 in
// that thread, y is rounded once, and every access to memory is one 16-byte
// piece of a row.  An epilogue on the accumulators where they lie, 256 of a
// lane, took the compiler 30 s a kernel and spilled.  The way through LDS costs
// 4 thousand cycles of a 256 x 256 tile, 2% of an 8192-deep product.
//
// Pre-activations kept for the way back leave the same registers, rounded to
// the operands' type or to 8 bits: a power of two for 32 columns of a row, four
// neighbouring threads', so their largest takes two exchanges, and multiplying
// by its inverse is exact: e4m3's rounding is the only one.
#include "feed_device.h"

namespace agmm {

namespace {

template <int BM, int BN, int DT, int OCC, bool GATED>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
void feed_tile_kernel(FeedProblem fp) {
  constexpr bool BT = true, SPLIT = false;
  constexpr int BK = 64, WAVES = 4;
  using T = GemmTile<BM, BN, BK, DT, BT, 5, WAVES, kLoopParts>;
  constexpr int kBK = BK;
  constexpr int FM = T::TM / 16, FN = T::TN / 16;
  constexpr int STEPS = BK / 32;
  __shared__ __attribute__((aligned(1024))) char smem[T::LDS_BYTES];
  const GemmProblem& p = fp.gemm;
  const int NC = fp.n;                         // columns of y

// Tile column r of a gated tile: block r / 32 of y's columns, part (r / 16) % 2.
#define AGMM_CLAMP
#define AGMM_B_ROW(r) \
  (GATED ? min((n0 >> 1) + (((r) >> 5) << 4) + ((r) & 15), NC - 1) + (((r) >> 4) & 1) * NC : min(n0 + (r), N - 1))
#define AGMM_B_IN(r) true
#define AGMM_B_FIRST (GATED ? n0 >> 1 : n0)
#define AGMM_B_LAST (GATED ? (n0 >> 1) + BN / 2 - 1 + NC : n0 + BN - 1)
#define AGMM_B_WHOLE (GATED ? (n0 + BN) >> 1 <= NC : n0 + BN <= N)
#include "gemm_m16_loop.inc"

  constexpr int PARTS = GATED ? 2 : 1;
  constexpr int ROW = BN * 4;                  // bytes of a row of sums; 16-byte piece c of row r at c ^ (r % 16)
  constexpr int HALVES = BM * ROW > T::LDS_BYTES ? 2 : 1, HR = BM / HALVES;
  static_assert(HALVES == 1 || HR == T::TM, "a half is the rows of one wave row");
  constexpr int PIECES = BN / PARTS / 8;       // of eight columns of y, a thread each
  constexpr int STEP = T::THREADS / PIECES;    // rows at a time
  const int c = tid % PIECES;
  const int col = n0 / PARTS + 8 * c, left = NC - col;
  // 16-byte pieces of the thread's columns: pieces at, at + 1 of the first part
  // and, gated, at + 4, at + 5 of the second
  const int at = GATED ? 8 * (c >> 1) + 2 * (c & 1) : 2 * c;
  float bias[PARTS][8];
#pragma unroll
  for (int h = 0; h < PARTS; ++h) {
    u32x4_t b = {0u, 0u, 0u, 0u};
    if (fp.bias && left > 0) b = load8(static_cast<const uint16_t*>(fp.bias) + (int64_t)h * NC + col, left);
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[h][e] = e & 1 ? high16<DT>(b[e >> 1]) : low16<DT>(b[e >> 1]);
  }
  const int64_t wide = fp.kept.wide;
  const bool keep = fp.kept.values && col < wide;
  const float c1 = fp.act.c1, c3 = fp.act.c3;

#pragma unroll 1
  for (int half = 0; half < HALVES; ++half) {
    __syncthreads();                           // every wave is done with what the LDS held
    if (HALVES == 1 || wm == half) {
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int r = (HALVES == 1 ? wm * T::TM : 0) + 16 * i + i16;
#pragma unroll
        for (int j = 0; j < FN; ++j)
          *reinterpret_cast<f32x4_t*>(smem + r * ROW + ((((wn * T::TN + 16 * j) >> 2) + g4) ^ (r & 15)) * 16) = acc[i][j];
      }
    }
    __syncthreads();
    with_kind(fp.act.kind, [&](auto kind) {
      constexpr int KIND = decltype(kind)::value;
#pragma unroll 2
      for (int it = 0; it < HR / STEP; ++it) {
        const int r = it * STEP + tid / PIECES;
        const int64_t row = m0 + half * HR + r;
        float v[PARTS][8];
#pragma unroll
        for (int h = 0; h < PARTS; ++h)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const f32x4_t x = *reinterpret_cast<const f32x4_t*>(smem + r * ROW + ((at + 4 * h + s) ^ (r & 15)) * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[h][4 * s + e] = x[e] + bias[h][4 * s + e];
          }
        if (keep) {
#pragma unroll
          for (int h = 0; h < PARTS; ++h) {
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = e < left ? v[h][e] : 0.0f;
            const int64_t out = (row * PARTS + h) * wide + col;
            if (!fp.kept.scales) {
              if (row < M)
                *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(fp.kept.values) + out) =
                    u32x4_t{pack2<DT>(w[0], w[1]), pack2<DT>(w[2], w[3]), pack2<DT>(w[4], w[5]), pack2<DT>(w[6], w[7])};
            } else {
              float size = 0.0f;
#pragma unroll
              for (int e = 0; e < 8; ++e) size = larger_finite(size, w[e]);
              size = fmaxf(size, __shfl_xor(size, 1));
              size = fmaxf(size, __shfl_xor(size, 2));
              const uint32_t code = scale_code(size);
              const float inv = scale_inverse(code);
              if (row < M) {
                *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(fp.kept.values) + out) =
                    u32x2_t{pack4_e4m3(w[0], w[1], w[2], w[3], inv), pack4_e4m3(w[4], w[5], w[6], w[7], inv)};
                if ((c & 3) == 0) fp.kept.scales[out / kKeptBlock] = (uint8_t)code;
              }
            }
          }
        }
        if (row < M && left > 0) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] = act_value<KIND>(v[0][e], c1, c3);
            if constexpr (GATED) y[e] *= v[1][e];
          }
          if (!GATED && fp.residual) {
            const u32x4_t b = load8(static_cast<const uint16_t*>(fp.residual) + row * fp.ldr + col, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] += e & 1 ? high16<DT>(b[e >> 1]) : low16<DT>(b[e >> 1]);
          }
          store8(static_cast<uint16_t*>(fp.y) + row * fp.ldy + col,
                 u32x4_t{pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3]), pack2<DT>(y[4], y[5]), pack2<DT>(y[6], y[7])}, left);
        }
      }
    });
  }
}

template <int DT>
hipError_t launch_type(const FeedProblem& p, int tile, hipStream_t s) {
  const unsigned grid = (unsigned)(p.gemm.order.num_rb * p.gemm.order.num_cb);
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, s, p); };
  if (tile == 256) p.gated ? go(feed_tile_kernel<256, 256, DT, 1, true>) : go(feed_tile_kernel<256, 256, DT, 1, false>);
  else p.gated ? go(feed_tile_kernel<128, 128, DT, 2, true>) : go(feed_tile_kernel<128, 128, DT, 2, false>);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_feed_tiles(const FeedProblem& p, int tile, int dtype, hipStream_t s) {
  const int64_t cols = p.gated ? 2 * (((int64_t)p.n + 15) / 16 * 16) : p.n;
  if ((tile != 256 && tile != 128) || p.gemm.n != cols || p.gemm.order.num_rb != (p.gemm.m + tile - 1) / tile ||
      p.gemm.order.num_cb != (p.gemm.n + tile - 1) / tile ||
      (int64_t)p.gemm.order.num_rb * p.gemm.order.num_cb >= kFeedGrid || p.gemm.k % 8 != 0 ||
      (p.gated && p.residual) || (p.kept.values && p.kept.wide != ((int64_t)p.n + kKeptBlock - 1) / kKeptBlock * kKeptBlock))
    return hipErrorInvalidValue;
  return dtype == kDtypeBf16 ? launch_type<kDtypeBf16>(p, tile, s)
       : dtype == kDtypeFp16 ? launch_type<kDtypeFp16>(p, tile, s) : hipErrorInvalidValue;
}

}  // namespace agmm
