// Launch interfaces of the feed-forward block's kernels and of layer norm.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_kernels.h"

namespace agmm {

// Activations y = x * share(x) by the form of their share.
enum ActKind : int {
  kActLinear = 0,      // 1
  kActRelu = 1,        // 1 for x > 0, else 0
  kActLogistic = 2,    // 1 / (1 + exp(-x (c1 + c3 x^2))): gelu's tanh form
  kActNormal = 3,      // the normal distribution function: gelu
  kActSilu = 4,        // 1 / (1 + exp(-x))
};
struct Activation {
  int32_t kind;
  float c1, c3;
};

// Columns of a row that share one scale of the 8-bit pre-activations, and what
// a part's columns are padded to (with zeros) in either form.
constexpr int kKeptBlock = 32;

// Pre-activations kept for the way back, [m][parts][wide]: in the operands'
// type (scales null) or e4m3 with a power of two per kKeptBlock columns, as its
// biased exponent, in scales [m][parts][wide / kKeptBlock].
struct KeptRows {
  void* values;            // null: none
  uint8_t* scales;
  int64_t wide;            // n rounded up to kKeptBlock
};

// y = act(p) [* p of the second part] [+ residual], p = A B^T + bias.  gemm
// describes the product in tile columns: plain, the n rows of B; gated,
// interleaved blocks of 16 rows of the first and the second n rows
// (gemm.n = 2 * (n rounded up to 16)).
struct FeedProblem {
  GemmProblem gemm;
  int32_t n;               // columns of y
  int32_t gated;
  Activation act;
  const void* bias;        // [parts * n] or null
  const void* residual;    // or null
  int64_t ldr;
  void* y;
  int64_t ldy;
  KeptRows kept;
};
constexpr int64_t kFeedGrid = int64_t(1) << 24;
// Tiles of 256 x 256 (tile 256), 256 x 224 (224; not for 8-bit pre-activations of
// a gated product, whose blocks of 32 columns its 112 columns of y would cut; 16-bit
// ones need no block in one tile, and the last tile column writes the zeros of the
// block that it ends in) or 128 x 128 tile columns (128); rows of whole 16-byte
// vectors.
// gemm.splits > 1 (tile 128): ranges of k to gemm.partials [splits][m][tile
// columns rounded up to 16], and a second launch that finishes.
hipError_t launch_feed_tiles(const FeedProblem& p, int tile, int dtype, hipStream_t stream);
// The sums of gemm.splits ranges in gemm.partials, added in order and finished.
hipError_t launch_feed_join(const FeedProblem& p, int dtype, hipStream_t stream);
// Few rows: blocks of 16 fm rows x yc columns of y (fm 1 or 4; yc 8 with fm 1,
// 16, or 64, gated 32: that where pre-activations are kept, whose blocks of 32
// columns of a part lie in one workgroup); any k and strides, operands in place.
// order.num_cb counts blocks of yc columns.  gemm.splits > 1 (not yc 8): ranges of
// k, as above, and launch_feed_join; kept pre-activations then at any yc.
hipError_t launch_feed_few(const FeedProblem& p, int fm, int yc, int dtype, hipStream_t stream);

// Copies of A and of W as rows of whole 128-byte lines (PadRows, ops_kernels.h;
// num_groups 0: none).
struct FeedCopies {
  PadRows a, w;
};
hipError_t launch_feed_copies(const FeedCopies& c, hipStream_t stream);

// The elementwise part of the way back: d = dy * (derivative of y by p), by
// rows [m][ldd] (zeros past parts * n up to a multiple of 8) and transposed
// [parts * n][ldt] (the same past m), each where asked for, and the sums of d
// over blocks of `block` rows, 32 or 128.
constexpr int kDCols = 64;
struct FeedDProblem {
  int64_t m;
  int32_t n, gated;
  int32_t block;
  Activation act;
  KeptRows kept;           // values may be null for a linear product without a gate
  const void* dy;
  int64_t lddy;
  void* d;
  int64_t ldd;
  void* dt;
  int64_t ldt;
  float* sums;             // [blocks of rows][parts * n] or null
};
// ... and, in the same launch, copies of A and W.
hipError_t launch_feed_d(const FeedDProblem& p, const FeedCopies& c, int dtype, hipStream_t stream);

// y = act(p) [* p of the second part] from the kept pre-activations.
struct FeedAgainProblem {
  int64_t m;
  int32_t n, gated;
  Activation act;
  KeptRows kept;
  void* y;
  int64_t ldy;
};
hipError_t launch_feed_again(const FeedAgainProblem& p, int dtype, hipStream_t stream);

// The products dA = d W and dW = dt A, B k x n, in one launch (m 0: none): with
// splits > 1 fp32 sums per k range into partials [splits][m][n rounded up to 4],
// else the result itself, rounded; and the bias's gradient (out null: none) from
// the sums over blocks of rows.
struct FeedBias {
  const float* sums;       // [groups][cols]
  int64_t groups, cols;
  void* out;
};
struct FeedGrads {
  GemmProblem a, w;
  // dW's B, A's rows: in one piece at w.b (w_rows 0), or w_rows rows, a multiple
  // of 64, at each of w_group
  const void* w_group[kMaxGroups];
  int32_t w_rows;
  int32_t a_tiles, a_first, tiles;   // set by launch_feed_grads: workgroups of dA, the first of them, of both
  FeedBias bias;
};
hipError_t launch_feed_grads(FeedGrads g, int tile, int dtype, hipStream_t stream);

// out[row][col] = sum over ranges, in order, of sums[range][row][cols rounded
// up to 4], rounded to `dtype` (a 16-bit type).
struct SumRanges {
  const float* sums;
  int32_t ranges;
  int64_t rows, cols;
  void* out;
  int64_t ldo;
};
// One or two of them (null: none) in one launch.
hipError_t launch_sum_ranges(const SumRanges* a, const SumRanges* b, int dtype, hipStream_t stream);

// out[c] = sum over groups, in a fixed order, of sums[group][c], for c < cols,
// rounded to `dtype`; columns from `first` on go to out2 (first = cols: none).
// Either of out and out2 may be null.
struct SumColumns {
  const float* sums;
  int64_t groups, cols, first;
  void *out, *out2;
  int32_t dtype;
};
hipError_t launch_sum_columns(const SumColumns& p, hipStream_t stream);

// Layer norm over rows of any alignment.  weight and bias may be null (1, 0);
// mean and rstd may be null on the way forward.
struct NormProblem {
  int64_t rows, cols;
  int32_t dtype, wtype;
  int32_t cus;             // of the GPU
  const void* x;
  int64_t ldx;
  const void* weight;
  const void* bias;
  float eps;
  void* y;                 // forward
  int64_t ldy;
  float* mean;
  float* rstd;
  const void* dy;          // backward
  int64_t lddy;
  void* dx;                // or null
  int64_t lddx;
  float* sums;             // [groups][2][cols]: sums of dy * xhat and of dy; or null
  int32_t groups;
  void *dweight, *dbias;   // one group: the sums themselves, rounded to wtype (sums null); or null
};
hipError_t launch_norm_forward(const NormProblem& p, hipStream_t stream);
hipError_t launch_norm_backward(const NormProblem& p, hipStream_t stream);
// Whether the backward pass writes dweight and dbias itself.
bool norm_direct(int64_t cols, int dtype, int groups);
// Workgroups (and groups of sums) of the backward pass.
int norm_groups(int64_t rows, int64_t cols, int dtype, int cus);

}  // namespace agmm
