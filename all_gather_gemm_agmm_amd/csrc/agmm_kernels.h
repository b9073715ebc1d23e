// Internal interface between the plan/scheduler (agmm_api.cpp) and the HIP
// kernels.  Not installed; the public interface is include/agmm.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace agmm {

// Largest number of shard buffers one call can name.  The pointer table
// travels in the kernel arguments (8 bytes per entry).
constexpr int kMaxGroups = 64;

constexpr int kDtypeBf16 = 0;
constexpr int kDtypeFp16 = 1;
constexpr int kDtypeFp32 = 2;

// Row mapping shared by every kernel that reads the gathered operand.
//
// A launch covers m = num_groups * rows_per_group logical rows.  Logical row
// i belongs to group g = i / rows_per_group at position t = i % rows_per_group:
//   its A row starts at  a_group[g] + t * a_ld            (elements)
//   its C row is         g * c_group_rows + c_row_off + t
// The fused path passes the shard pointers themselves (one group per shard);
// a ring slot or the fully gathered buffer is described the same way.
struct RowMap {
  const void* a_group[kMaxGroups];
  int64_t a_ld;            // elements between consecutive rows of one group
  int32_t rows_per_group;  // rows of each group covered by this launch
  int32_t num_groups;
  int64_t c_group_rows;    // C rows between the starts of consecutive groups
  int64_t c_row_off;       // C row of position t = 0 inside each group
};

// Order in which workgroups visit output tiles.
struct TileOrder {
  const int32_t* rb_order;  // device table: visit order of row blocks (nullptr = natural)
  int32_t num_rb;           // row blocks  (ceil(m / BM))
  int32_t num_cb;           // column blocks (ceil(n / BN))
  int32_t group_m;          // row blocks walked together for L2 reuse
  int32_t xcd_remap;        // 1: keep consecutive tiles on one XCD
};

struct GemmProblem {
  RowMap rows;
  TileOrder order;
  int32_t m, n, k;
  const void* b;
  int64_t ldb;             // elements between rows of B as stored
  void* c;
  int64_t ldc;             // elements between rows of C
  // split-K (used when splits > 1): partial sums, then a reduction kernel
  int32_t splits;
  int32_t k_per_split;     // multiple of kTileBK
  float* partials;         // [splits][m][n] fp32 scratch
};

// Tile shapes compiled for the MFMA kernels.  Each one is reached by the
// plan's automatic choice or by the autotuner's candidate list.
enum TileCfg : int {
  kTile256x256 = 0,      // 4 waves, 128x128 per wave, 32-deep k-tiles in a 4-stage ring (k < 256)
  kTile128x128 = 1,      // 64x64 per wave, two workgroups per CU
  kTile256x128 = 2,      // 128x64 per wave, two workgroups per CU
  kTile128x64 = 3,       // 4 waves, 64x32 per wave; B stored n x k only
  kTile128x64s8 = 4,     // 8-stage LDS ring (whole short k ranges in flight); B stored n x k only
  kTile256x256r5 = 5,    // 64-deep k-tiles in a ring of 5 operand slots (whole L2 lines per load)
  kTile128x128r5 = 6,    // same ring, 128x128, two workgroups per CU
  kTile128x64r5 = 7,     // same ring, 128x64; B stored n x k only
  kTile256x256m16 = 8,   // part ring, 256x256, on 16x16x32 MFMAs (automatic for k >= 256)
  kTile128x128m16 = 9,   // part ring, 128x128, on 16x16x32 MFMAs
  kTileSkinny = 10,      // narrow tiles over all of k or k ranges, wave-private LDS rings (launch_skinny_fullk); B n x k only
  kTile256x224m16 = 11,  // part ring, 256x224 on 16x16x32 MFMAs (7 column blocks per wave); B n x k only
  kTileCount = 12,
};
// Tiles that read B only as stored n x k (rhs_transpose).
constexpr bool tile_needs_bt(int cfg) {
  return cfg == kTile128x64 || cfg == kTile128x64s8 || cfg == kTile128x64r5 || cfg == kTileSkinny ||
         cfg == kTile256x224m16;
}
int tile_bm(int cfg);
int tile_bn(int cfg);
int tile_bk(int cfg);
int tile_occ(int cfg);   // workgroups of this tile that fit on one CU
// k granularity of split-K ranges (a multiple of every configuration's depth)
constexpr int kTileBK = 64;

// bf16/fp16 MFMA GEMM (16-bit inputs, fp32 accumulate, output in the input dtype).
// With p.splits > 1 this is two launches on `stream`: fp32 partial sums per
// k range, then their fixed-order sum and cast.
hipError_t launch_gemm_mfma(const GemmProblem& p, int tile_cfg, int dtype, bool rhs_transpose,
                            hipStream_t stream);

// Skinny-m kernel (tile kTileSkinny, B stored n x k): small output tiles
// (32 x 32 by default), each over the whole of k in one workgroup (one
// launch), or with p.splits > 1 over one of p.splits k ranges of
// p.k_per_split elements (a multiple of 64) into p.partials [splits][m][n]
// fp32, then launch_splitk_reduce.  C rows through the row map.
// `shape` selects the tile: 0: 64 x 16, 1: 32 x 32, 2: 32 x 16, 3: 16 x 32,
// 4: 64 x 32, 7: 64 x 64 (rows x columns) with 4 waves; 5: 32 x 32 and 6:
// 64 x 16 with 8 waves (the LDS shared out over twice as many, half as
// deep, rings).
hipError_t launch_skinny_fullk(const GemmProblem& p, int dtype, int shape, hipStream_t stream);

// Fixed-order sum of p.partials [p.splits][p.m][p.n] fp32 (split 0 first),
// cast to the output dtype and stored to C through the row map.
hipError_t launch_splitk_reduce(const GemmProblem& p, int dtype, hipStream_t stream);

// fp32 inputs, fp64 accumulate, fp32 output (any shape).
hipError_t launch_gemm_f32(const GemmProblem& p, bool rhs_transpose, hipStream_t stream);

// Bit copy of rows into a dense destination:
//   dst[(g * dst_group_rows + t) * row_bytes ...] = src_group[g][(src_row0 + t) * src_ld_bytes ...]
// for g < num_groups, t < rows.  row_bytes % 16 == 0 and src_ld_bytes % 16 == 0
// (src_ld_bytes == 0: row_bytes), all pointers 16-byte aligned.
struct GatherProblem {
  const void* src_group[kMaxGroups];
  int32_t num_groups;
  int64_t src_row0;
  int64_t rows;
  int64_t row_bytes;
  int64_t src_ld_bytes;    // bytes between source rows (0: row_bytes)
  void* dst;
  int64_t dst_group_rows;
};
hipError_t launch_gather(const GatherProblem& p, int max_workgroups, hipStream_t stream);

// Element-granular copy of rows for rows that are not whole 16-byte vectors
// (any row length and strides), with zero fill:
//   dst[(g * dst_group_rows + t) * dst_ld + c] =
//       (t < src_rows && c < cols) ? src_group[g][(src_row0 + t) * src_ld + c] : 0
// for g < num_groups, t < rows, c < dst_cols.  Strides and lengths in
// elements of elem_bytes (2 or 4) bytes; pointers aligned to an element.
struct PadCopyProblem {
  const void* src_group[kMaxGroups];
  int32_t num_groups;
  int32_t elem_bytes;
  int64_t src_row0;
  int64_t src_rows;        // rows of each group that exist in the source (the rest are zeros)
  int64_t src_ld;
  int64_t cols;            // elements of a source row that are copied
  int64_t rows;            // rows written per group
  void* dst;
  int64_t dst_group_rows;
  int64_t dst_ld;
  int64_t dst_cols;        // elements written per row (zeros past cols)
};
hipError_t launch_pad_copy(const PadCopyProblem& p, hipStream_t stream);

// Transpose of a 16-bit matrix: out[c * rows + r] = in[r * ld_in + c] for
// r < rows, c < cols.  rows, cols and ld_in multiples of 8, both pointers
// 16-byte aligned (else hipErrorInvalidValue, nothing launched).
hipError_t launch_transpose16(const void* in, int64_t ld_in, int64_t rows, int64_t cols, void* out,
                              hipStream_t stream);

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
  kScaledTiles = 6,
};
constexpr int scaled_tile_rows(int t) {
  return t == kScaled256 ? 256 : t == kScaled128 ? 128 : t == kScaledSkinny16 || t == kScaledSkinny16n ? 16
       : t == kScaledSkinny32 ? 32 : t == kScaledSkinny64 ? 64 : 0;
}
constexpr int scaled_tile_cols(int t) {
  return t == kScaledSkinny16n ? 16 : t == kScaledSkinny16 || t == kScaledSkinny32 ? 32 : scaled_tile_rows(t);
}
hipError_t launch_scaled(const ScaledProblem& p, int tile, hipStream_t stream);

// Vocabulary loss over one piece of the vocabulary: gemm describes the logits
// of the piece (A rows through the row map, B the piece's rows of W, n x k;
// rows of whole 16-byte vectors), label0 is the label of its column 0.
struct LossProblem {
  GemmProblem gemm;
  int32_t tile;            // 256 or 128
  const int64_t* labels;   // [m]
  int64_t label0;
  // statistics: (maximum, sum of exp) pairs [2 * column block + half][m]
  float* stats;
  float* target;           // [m], written where the piece holds the label
  // gradient: rows {lse, a, b, s} [m]; d [m][ldd] and dt [n][ldt] (either
  // may be null), the columns past n (m) up to ldd (ldt) as zeros; both
  // strides are multiples of 8
  const float* rows;
  void* d;
  int64_t ldd;
  void* dt;
  int64_t ldt;
};
hipError_t launch_loss_logits(const LossProblem& p, int dtype, bool grad, hipStream_t stream);

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

// out [m][8 * chunks] = fp16 rows of A times rows[i][3] / scale_all[0], powers of two of at most 1.
struct LossScaleRows {
  const void* group[kMaxGroups];
  int64_t rows_per_group, ld, m, chunks;
  const float* rows;
  const float* scale_all;
  void* out;
};
hipError_t launch_loss_scale_rows(const LossScaleRows& c, hipStream_t stream);

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

// Size of the device scratch of the no-allocation entry point (one per GPU,
// held for the life of the process; equal to AGMM_NOALLOC_SCRATCH_BYTES).
constexpr size_t kNoallocScratchBytes = size_t(32) << 20;
// Device address of the current GPU's scratch (looked up on the first call
// on each device, then cached).
hipError_t noalloc_scratch(void** ptr);

}  // namespace agmm
