// Launch interfaces of the operators beside the all-gather matmul: the
// block-scaled 8-bit quantiser and product, and the vocabulary loss.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "agmm_kernels.h"

namespace agmm {

// 8-bit formats (OCP: e4m3 without infinities, e5m2 with them).
constexpr int kFmtE4M3 = 0;
constexpr int kFmtE5M2 = 1;

// Elements of k that share one scale of the block-scaled 8-bit operands.
constexpr int kScaleBlock = 128;

// Block-scaled 8-bit copies of x [rows][cols]: q [rows][ldq] with
// scale[block of columns][row block] and, of x transposed, qt [cols][ldqt]
// with scale_t[block of rows][column block].  Either pair may be null.
// Columns cols .. cols16 of q (rows .. rows16 of qt) are written as zeros.
struct QuantProblem {
  const void* x;
  int64_t rows, cols, ldx;
  int32_t dtype, format;
  int32_t block_rows;      // 1: a scale per row and 128 columns; 128: per 128 x 128 tile
  void* q;
  int64_t ldq;
  float* scale;
  void* qt;
  int64_t ldqt;
  float* scale_t;
  int64_t cols16, rows16;  // cols and rows rounded up to 16
};
hipError_t launch_quantize(const QuantProblem& p, hipStream_t stream);

// Division of 0 <= n < 2^31 by a divisor known on the host: the high half of
// n * floor(2^32 / d) is the quotient or one less.
struct FastDiv {
  uint32_t d, m;
  FastDiv() = default;
  explicit FastDiv(uint32_t by) : d(by), m(by == 1 ? 0xFFFFFFFFu : (uint32_t)((uint64_t(1) << 32) / by)) {}
  __device__ __forceinline__ int quotient(int n) const {
    const uint32_t q = (uint32_t)(((uint64_t)(uint32_t)n * m) >> 32);
    return (int)((uint32_t)n - q * d >= d ? q + 1 : q);
  }
};

// Block-scaled 8-bit product: logical row i is row i % rows_per_group of
// group i / rows_per_group, and row i of C.  Scales are [k block][row] for A
// (per group) and [k block][nb] for B.
struct ScaledProblem {
  const void* a_group[kMaxGroups];
  const float* a_scale[kMaxGroups];
  int64_t a_ld;            // bytes between rows of a group
  int32_t rows_per_group, num_groups;
  int32_t m, n, k16;       // k16: row length rounded up to 16 (zeros past k)
  int32_t kb;              // blocks of 128 of k
  const void* b;
  int64_t ldb;
  const float* b_scale;
  int32_t nb;              // row blocks of B (n for b_block_rows 1)
  int32_t b_block_rows;
  int32_t a_format;        // B is e4m3
  void* c;
  int64_t ldc;             // elements
  int32_t c_dtype;
  int32_t deep;            // kScaled128: four k-tiles in LDS, one workgroup per CU
  int32_t wide;            // kScaled128: sums of 128 by bf16 MFMAs on the widened values
  TileOrder order;         // tiles kScaled256 and kScaled128
  int32_t splits;          // k ranges of kb_per_split blocks, into partials [splits][m][part_ld]
  int32_t kb_per_split;
  float* partials;
  int64_t part_ld;         // a multiple of 4
  FastDiv by_rows, by_tiles, by_group, by_full, by_last;   // set by launch_scaled
};
enum ScaledTile : int {
  kScaled256 = 0,          // 256 x 256, 8 waves, 8-bit MFMAs
  kScaled128 = 1,          // 128 x 128, 4 waves, two workgroups per CU; 8-bit or bf16 MFMAs (wide)
  kScaledSkinny16 = 2,     // 16 x 32, k-tiles shared out over 4 waves, bf16 MFMAs
  kScaledSkinny32 = 3,     // 32 x 32
  kScaledSkinny16n = 4,    // 16 x 16, 8 waves
  kScaledSkinny64 = 5,     // 64 x 64
};
constexpr int scaled_tile_rows(int t) {
  return t == kScaled256 ? 256 : t == kScaled128 ? 128 : t == kScaledSkinny16 || t == kScaledSkinny16n ? 16
       : t == kScaledSkinny32 ? 32 : t == kScaledSkinny64 ? 64 : 0;
}
constexpr int scaled_tile_cols(int t) {
  return t == kScaledSkinny16n ? 16 : t == kScaledSkinny16 || t == kScaledSkinny32 ? 32 : scaled_tile_rows(t);
}
hipError_t launch_scaled(const ScaledProblem& p, int tile, hipStream_t stream);

// Workgroups of one launch of the loss's products.
constexpr int64_t kLossGrid = int64_t(1) << 24;

// Vocabulary loss over one piece of the vocabulary: gemm describes the logits
// of the piece (A rows through the row map, B the piece's rows of W, n x k;
// rows of whole 16-byte vectors), label0 is the label of its column 0.
struct LossProblem {
  GemmProblem gemm;
  int32_t tile;            // 256 or 128 (launch_loss_logits)
  const int64_t* labels;   // [m]
  int64_t label0;
  // statistics: (maximum, sum of exp) pairs [2 * column block + half][m]
  float* stats;
  float* target;           // [m], written where the piece holds the label
  // gradient: rows {lse, a, b, s} [m] and scale_all (see LossRows); d [m][ldd],
  // row i over s_i, and dt [n][ldt], all over scale_all (either may be null),
  // the columns past n (m) up to ldd (ldt) as zeros; both strides are
  // multiples of 8
  const float* rows;
  const float* scale_all;
  void* d;
  int64_t ldd;
  void* dt;
  int64_t ldt;
};
hipError_t launch_loss_logits(const LossProblem& p, int dtype, bool grad, hipStream_t stream);
// The same for few rows, in blocks of 16 fm rows x 16 fn columns (1 or 4 each;
// order.num_rb and num_cb count those): any k and any strides, operands in
// place; stats [column block][m][2].
hipError_t launch_loss_few(const LossProblem& p, int fm, int fn, int dtype, bool grad, hipStream_t stream);

struct LossCombine {
  const float* stats;
  int32_t parts;
  int64_t m;
  float* running;          // (maximum, sum) [m] between pieces
  int32_t first, last;
  const int64_t* labels;
  int64_t start, n, total, ignore;
  float *loss, *lse, *target;
};
hipError_t launch_loss_combine(const LossCombine& c, hipStream_t stream);

struct LossRows {
  int64_t m;
  const int64_t* labels;
  int64_t total, ignore;
  const float *lse, *grad_loss, *grad_lse;   // grad_lse may be null
  float* rows;
  float* scale_all;
};

// Copy of 16-bit rows as rows of whole 16-byte vectors (zeros past cols):
// out [num_groups][rows][8 * chunks], chunks = ceil(cols / 8).  Sources need
// element alignment only.
struct PadRows {
  const void* group[kMaxGroups];
  int64_t num_groups, rows, cols, ld, chunks;
  void* out;
};
// One launch: the rows' weights (r, or null) and a copy (c, or null).
hipError_t launch_loss_prepare(const LossRows* r, const PadRows* c, int dtype, hipStream_t stream);

// The two gradient products, B k x n, in one launch: fp32 sums of d W (A = d
// [m][ldd]) into a->partials [splits][m][n rounded up to 4], added to what is there
// when `add`, and C = scale[0] * dt A.  Either may be null.
hipError_t launch_loss_grads(const GemmProblem* a, bool add, const GemmProblem* w, const float* scale, int tile, int dtype,
                             hipStream_t stream);
struct LossFinish {
  const float* sums;       // [ranges][m][k rounded up to 4]
  int32_t ranges;
  int64_t m;
  int32_t k;
  const float* rows;
  void* da;
  int64_t ldda;
};
hipError_t launch_loss_da_finish(const LossFinish& c, int dtype, hipStream_t stream);

}  // namespace agmm
