// Product with an epilogue, and the gated product: large tiles (gfx950).
//
//     p = A B^T + bias,  y = act(p) + residual      or, gated,  y = act(p_0) * p_1
//
// A tile is one of the part-ring GEMM (gemm_m16_loop.inc), 256 x 256, 256 x 224
// or 128 x 128 tile columns.  Gated, the tile's columns are blocks of 16 rows of the
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
//
// Bound: MFMA, in practice power.  Measured, rows x k -> columns: 8192 x 8192 ->
// 2 x 7168 bf16, silu, 8 bits kept, 1360-1450 us, 1330-1410 TFLOP/s (a library
// product of that size alone reaches 1480); 8192 x 8192 -> 3584 fp16, gelu, 372-
// 416 us by 256 x 224 (two even rounds of the CUs, where 448 tiles of 256 x 256
// are one and three quarters: 380), 10 of them gelu's exponentials, which no
// MFMA of the same wave runs beside.  1011 x 4040 -> 2 x 2051 fp16: 57 us on 264
// tiles, more than the CUs at one each, and 16 for the copies.
#include "feed_device.h"

namespace agmm {

namespace {

// The main loop's B for both kernels here, GATED, BN and NC, the columns of y,
// being the kernel's own.  Tile column r of a gated tile: block r / 32 of y's
// columns, part (r / 16) % 2.
#define AGMM_CLAMP
#define AGMM_B_ROW(r) \
  (GATED ? min((n0 >> 1) + (((r) >> 5) << 4) + ((r) & 15), NC - 1) + (((r) >> 4) & 1) * NC : min(n0 + (r), N - 1))
#define AGMM_B_IN(r) true
#define AGMM_B_FIRST (GATED ? n0 >> 1 : n0)
#define AGMM_B_LAST (GATED ? (n0 >> 1) + BN / 2 - 1 + NC : n0 + BN - 1)
#define AGMM_B_WHOLE (GATED ? (n0 + BN) >> 1 <= NC : n0 + BN <= N)

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

#include "gemm_m16_loop.inc"

  constexpr int PARTS = GATED ? 2 : 1;
  constexpr int ROW = BN == 224 ? 1024 : BN * 4;   // bytes of a row of sums; 16-byte piece c of row r at c ^ (r % 16)
  constexpr int HALVES = BM * ROW > T::LDS_BYTES ? 2 : 1, HR = BM / HALVES;
  static_assert(HALVES == 1 || HR == T::TM, "a half is the rows of one wave row");
  constexpr int PIECES = BN / PARTS / 8;       // of eight columns of y, a thread each
  constexpr int STEP = T::THREADS / PIECES;    // rows at a time; 224: four threads are left over
  constexpr bool EVEN = STEP * PIECES == T::THREADS && HR % STEP == 0;
  const int c = tid % PIECES;
  const int col = n0 / PARTS + 8 * c;
  // 16-byte pieces of the thread's columns: pieces at, at + 1 of the first part
  // and, gated, at + 4, at + 5 of the second
  const int at = GATED ? 8 * (c >> 1) + 2 * (c & 1) : 2 * c;
  // A gated tile of 224 ends in the middle of a block of 32 kept columns (112 of y):
  // where it is the last one, the block's other 16, all past n, are zeros from
  // the two threads whose own columns are 16 before them.
  const bool tail = GATED && BN == 224 && fp.kept.values && n0 + BN >= N && c >= PIECES - 2 && col + 16 < fp.kept.wide;
  float bias[PARTS][8];
  bias8<DT, GATED>(fp, col, bias);

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
      const auto one = [&](int r) {
        const int64_t row = m0 + half * HR + r;
        float v[PARTS][8];
#pragma unroll
        for (int h = 0; h < PARTS; ++h)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const f32x4_t x = *reinterpret_cast<const f32x4_t*>(smem + r * ROW + ((at + 4 * h + s) ^ (r & 15)) * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[h][4 * s + e] = x[e];
          }
        if (fp.bias)
#pragma unroll
          for (int h = 0; h < PARTS; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[h][e] += bias[h][e];
        finish8<DT, GATED, KIND>(fp, v, row, row < M, col);
        if (GATED && BN == 224 && tail && row < M)
#pragma unroll
          for (int h = 0; h < PARTS; ++h)
            *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(fp.kept.values) + (row * PARTS + h) * fp.kept.wide + col + 16) =
                u32x4_t{0u, 0u, 0u, 0u};
      };
      if constexpr (EVEN) {
#pragma unroll 2
        for (int it = 0; it < HR / STEP; ++it) one(it * STEP + tid / PIECES);
      } else if (tid < STEP * PIECES) {
#pragma unroll 1
        for (int r = tid / PIECES; r < HR; r += STEP) one(r);
      }
    });
  }
}

// Few tiles: ranges of k, 128 x 128 tile columns each, to fp32 sums [range][m]
// [tile columns rounded up to 16] ...
template <int DT, bool GATED>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2)))
void feed_part_kernel(FeedProblem fp) {
  constexpr bool BT = true, SPLIT = true;
  constexpr int BM = 128, BN = 128, BK = 64, WAVES = 4, OCC = 2;
  using T = GemmTile<BM, BN, BK, DT, BT, 5, WAVES, kLoopParts>;
  constexpr int kBK = BK;
  constexpr int FM = T::TM / 16, FN = T::TN / 16;
  constexpr int STEPS = BK / 32;
  __shared__ __attribute__((aligned(1024))) char smem[T::LDS_BYTES];
  const GemmProblem& p = fp.gemm;
  const int NC = fp.n;
#include "gemm_m16_loop.inc"

  const int out_row = m0 + wm * T::TM + i16, out_col = n0 + wn * T::TN + 4 * g4;
  const int64_t ld = (N + 15) & ~15;
  float* base = p.partials + ((int64_t)split * M + out_row) * ld + out_col;
#pragma unroll
  for (int i = 0; i < FM; ++i, base += 16 * ld)
    if (out_row + 16 * i < M)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        if (out_col + 16 * j < ld) *reinterpret_cast<f32x4_t*>(base + 16 * j) = acc[i][j];
}

// ... which are added in order, and finished, by a thread per eight columns of y.
template <int DT, bool GATED>
__global__ __launch_bounds__(256) void feed_join_kernel(FeedProblem fp) {
  constexpr int PARTS = GATED ? 2 : 1;
  const GemmProblem& p = fp.gemm;
  const uint32_t pieces = (uint32_t)((fp.n + kKeptBlock - 1) / kKeptBlock * (kKeptBlock / 8));   // of four lanes each
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x, row = u / pieces;
  const int c = (int)(u - row * pieces), col = 8 * c;
  const bool in = row < p.m;
  const int64_t ld = (p.n + 15) & ~15, plane = p.m * ld;
  const int at = GATED ? 32 * (c >> 1) + 8 * (c & 1) : col;
  float v[PARTS][8];
  bias8<DT, GATED>(fp, col, v);
  if (in && col < fp.n) {
    const float* src = p.partials + row * ld + at;
    f32x4_t t[PARTS][2] = {};
    for (int s0 = 0; s0 < p.splits; s0 += 4) {
      f32x4_t x[4][PARTS][2];
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (s0 + s < p.splits)
#pragma unroll
          for (int h = 0; h < PARTS; ++h)
#pragma unroll
            for (int q = 0; q < 2; ++q) x[s][h][q] = *reinterpret_cast<const f32x4_t*>(src + (s0 + s) * plane + 16 * h + 4 * q);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (s0 + s < p.splits)
#pragma unroll
          for (int h = 0; h < PARTS; ++h)
#pragma unroll
            for (int q = 0; q < 2; ++q) t[h][q] += x[s][h][q];
    }
#pragma unroll
    for (int h = 0; h < PARTS; ++h)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[h][e] += t[h][e >> 2][e & 3];
  }
  with_kind(fp.act.kind, [&](auto kind) { finish8<DT, GATED, decltype(kind)::value>(fp, v, row, in, col); });
}

template <int DT>
hipError_t launch_type(const FeedProblem& p, int tile, hipStream_t s) {
  const unsigned grid = (unsigned)((int64_t)p.gemm.order.num_rb * p.gemm.order.num_cb * p.gemm.splits);
  const auto go = [&](auto kernel, unsigned wgs) { hipLaunchKernelGGL(kernel, dim3(wgs), dim3(256), 0, s, p); };
  if (p.gemm.splits > 1) {
    p.gated ? go(feed_part_kernel<DT, true>, grid) : go(feed_part_kernel<DT, false>, grid);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    return launch_feed_join(p, DT, s);
  } else if (tile == 224) {
    p.gated ? go(feed_tile_kernel<256, 224, DT, 1, true>, grid) : go(feed_tile_kernel<256, 224, DT, 1, false>, grid);
  } else if (tile == 256) {
    p.gated ? go(feed_tile_kernel<256, 256, DT, 1, true>, grid) : go(feed_tile_kernel<256, 256, DT, 1, false>, grid);
  } else {
    p.gated ? go(feed_tile_kernel<128, 128, DT, 2, true>, grid) : go(feed_tile_kernel<128, 128, DT, 2, false>, grid);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_feed_join(const FeedProblem& p, int dtype, hipStream_t s) {
  const int64_t pieces = ((int64_t)p.n + kKeptBlock - 1) / kKeptBlock * (kKeptBlock / 8), all = p.gemm.m * pieces;
  if (all >= kFeedGrid * 256 || !p.gemm.partials || (dtype != kDtypeBf16 && dtype != kDtypeFp16)) return hipErrorInvalidValue;
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)((all + 255) / 256)), dim3(256), 0, s, p); };
  if (dtype == kDtypeBf16) p.gated ? go(feed_join_kernel<kDtypeBf16, true>) : go(feed_join_kernel<kDtypeBf16, false>);
  else p.gated ? go(feed_join_kernel<kDtypeFp16, true>) : go(feed_join_kernel<kDtypeFp16, false>);
  return hipGetLastError();
}

hipError_t launch_feed_tiles(const FeedProblem& p, int tile, int dtype, hipStream_t s) {
  const int64_t cols = p.gated ? 2 * (((int64_t)p.n + 15) / 16 * 16) : p.n;
  const int bm = tile == 224 ? 256 : tile;
  if ((tile != 256 && tile != 224 && tile != 128) || p.gemm.n != cols || p.gemm.order.num_rb != (p.gemm.m + bm - 1) / bm ||
      p.gemm.order.num_cb != (p.gemm.n + tile - 1) / tile ||
      p.gemm.splits < 1 || (int64_t)p.gemm.order.num_rb * p.gemm.order.num_cb * p.gemm.splits >= kFeedGrid || p.gemm.k % 8 != 0 ||
      (p.gemm.splits > 1 && (tile != 128 || !p.gemm.partials || p.gemm.k_per_split % 64 != 0 ||
                             (int64_t)p.gemm.splits * p.gemm.k_per_split < p.gemm.k ||
                             (int64_t)(p.gemm.splits - 1) * p.gemm.k_per_split >= p.gemm.k)) ||
      (p.gated && p.residual) || (tile == 224 && p.gated && p.kept.scales) || (p.kept.values && p.kept.wide != ((int64_t)p.n + kKeptBlock - 1) / kKeptBlock * kKeptBlock))
    return hipErrorInvalidValue;
  return dtype == kDtypeBf16 ? launch_type<kDtypeBf16>(p, tile, s)
       : dtype == kDtypeFp16 ? launch_type<kDtypeFp16>(p, tile, s) : hipErrorInvalidValue;
}

}  // namespace agmm
