// Block-scaled 8-bit all-gather matmul (gfx950):
//
//     C[i, j] = sum_b sa[b, i] * sb[b, j / br] * ( sum_{k in block b} qa[i, k] * qb[j, k] )
//
// over blocks b of 128 elements of k; the rows i are the concatenation of the
// shards' rows, B is stored n x k, br is 1 or 128.  The inner sums come from
// the matrix cores (one v_mfma_f32_16x16x128, or four bf16 ones), started from
// zero: their four results per lane are scaled in fp32 and added to the fp32
// accumulators by ordinary FMAs.  (The MFMA's own block scales are powers of
// two; these scales are any fp32.)
//
// Both operands of an MFMA see the same order of k, whatever it is: lane
// group g of a fragment holds the 16-byte chunks g and 4 + g of a 128-byte
// row, the chunks the bf16 kernel's 64-deep rows are read in, so the same XOR
// swizzle keeps the reads free of LDS bank conflicts.
//
//  * scaled_gemm_kernel: two 128-deep k-tiles in LDS (four where a CU has one
//    workgroup of the small tile to itself), refilled by global -> LDS loads;
//    the row and column scales of a k-tile ride along as one 4-byte-per-lane
//    load per wave.  B fragments of a k-tile stay in
//    registers, A fragments pass through; the FMAs of row block i run beside
//    the MFMAs of row block i + 1.  The workgroup synchronises before the last
//    row block of a k-tile, once every fragment of it has been read, so that
//    the next k-tile's first reads and the refill run beside its MFMAs.
//    VALU and MFMA share the accumulators, which therefore live in ordinary
//    registers: two waves per SIMD with 128 accumulators each.  Bound: MFMA
//    (8-bit form: power, at 1.74 GHz; the pipe is busy 63% of the cycles).
//    Measured: 32768 x 8192 -> 7168 to bf16 1.52-1.62 ms, 2380-2530 TFLOP/s
//    (a library's 8-bit product with one scale: 2660 at 8192^3); 1011 x 4040 ->
//    2051 to fp16 28.8 us: 136 tiles of 128 x 128, each its CU's operand stream.
//    In bf16 MFMAs (below) the conversions and the scaling cost about as many
//    cycles as the MFMAs: 3584 x 8192 -> 4096 to fp32 228-245 us, 980-1055
//    TFLOP/s.
//  * scaled_skinny_kernel: few rows.  Every wave streams its own k-tiles
//    through a private LDS ring (no barrier in the loop); the waves' sums are
//    added in LDS in a fixed order.  Bound: what one workgroup with all of a
//    CU's LDS streams, 26 bytes per cycle (two with half of it each reach 38, so
//    this is the form's limit, not the CU's; the 64 x 64 tile's rings hold two
//    k-tiles per wave); a tile of 64 columns and rows needs half as many bytes
//    as two of 32.  Measured: 8 x 4096 -> 1792 5.6 us; 128 x 8192 -> 3584 in two
//    k ranges 17-20 us and 3.5-3.9 for their sum.
//  * scaled_reduce_kernel: fixed-order sum of k ranges.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_kernels.h"
#include "gemm_device.h"

namespace agmm {

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// One 16 x 16 block of sums over 128 of k, of a B fragment (first operand,
// e4m3) and an A fragment: lane (g, i) of the result holds row i, columns
// 4g .. 4g + 3.
//  * 8-bit MFMA: one instruction, but its adder cuts the products: measured, of
//    each 8 neighbours along k every product is cut to a multiple of 2^(E - 13),
//    E the largest sum of the two operands' exponents among the 8 (a subnormal
//    number counts with the smallest normal one's); the 16 sums of 8 are then
//    added like fp32 numbers.  A block may so lose 16 * 7 * 2^(E - 13): up to
//    7 * 2^-13 (14336 u, u = 2^-24) of its terms' sizes, and more where the
//    largest operand of 8 is subnormal.  On random bytes it is 400 u (rms), on
//    normally distributed values of one scale 30 u, and 850 u with one value in
//    128 at the format's end.
//  * bf16 MFMAs on the widened values (both formats are exact in bf16): 0.6 u
//    and 4.4 u at most on random bytes, at half the rate.
template <int FMTA>
__device__ __forceinline__ f32x4_t mfma128(const u32x4_t (&b)[2], const u32x4_t (&a)[2]) {
  i32x8_t bv, av;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    bv[e] = (int)b[0][e];
    bv[4 + e] = (int)b[1][e];
    av[e] = (int)a[0][e];
    av[4 + e] = (int)a[1][e];
  }
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv, av, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, FMTA, 0, 0, 0, 0);
}

// The 32 8-bit values of a fragment as four bf16 fragments of 8.
template <int FMT>
__device__ __forceinline__ void widen(const u32x4_t (&f)[2], bf16x8_t (&w)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const uint32_t v = f[q >> 1][2 * (q & 1) + d];
      bf16x2_t lo, hi;
      if constexpr (FMT == kFmtE4M3) {
        lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false);
        hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true);
      } else {
        lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(v, 1.0f, false);
        hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(v, 1.0f, true);
      }
      w[q][4 * d] = lo[0];
      w[q][4 * d + 1] = lo[1];
      w[q][4 * d + 2] = hi[0];
      w[q][4 * d + 3] = hi[1];
    }
}

__device__ __forceinline__ f32x4_t mfma128_wide(const bf16x8_t (&b)[4], const bf16x8_t (&a)[4]) {
  f32x4_t c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int q = 0; q < 4; ++q) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[q], a[q], c, 0, 0, 0);
  return c;
}

// One 4-byte-per-lane global -> LDS load: lane i writes bytes [4i, 4i + 4) at
// `lds_addr` (wave-uniform).
__device__ __forceinline__ void load_lds4_at(const void* gsrc, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
               :
               : "v"(gsrc), "s"(__builtin_amdgcn_readfirstlane(lds_addr))
               : "m0");
}

// The same through a buffer descriptor.
__device__ __forceinline__ void load_lds4_buf(const u32x4_t& rsrc, uint32_t voff, uint32_t soff, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %3 offen lds"
               :
               : "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(lds_addr)),
                 "s"(__builtin_amdgcn_readfirstlane(soff))
               : "m0");
}

// One element, and four consecutive ones, of an output type.  Vectors in
// global memory need element alignment only.
typedef f32x4_t f32x4_any_t __attribute__((aligned(4)));
typedef u32x2_t u32x2_any_t __attribute__((aligned(2)));
template <int CT>
struct OutOf {
  typedef uint16_t type;
};
template <>
struct OutOf<kDtypeFp32> {
  typedef float type;
};
template <int CT, class P>
__device__ __forceinline__ void put1(P* c, float v) {
  if constexpr (CT == kDtypeFp32) *c = v;
  else *c = cvt1<CT>(v);
}
template <int CT, class P>
__device__ __forceinline__ void put4(P* c, const f32x4_t& v) {
  if constexpr (CT == kDtypeFp32) *reinterpret_cast<f32x4_any_t*>(c) = v;
  else *reinterpret_cast<u32x2_any_t*>(c) = u32x2_t{pack2<CT>(v[0], v[1]), pack2<CT>(v[2], v[3])};
}

// Four consecutive columns (col % 4 == 0) of one row to C in its own type.
__device__ __forceinline__ void store4(const ScaledProblem& p, int row, int col, const f32x4_t& v) {
  const int64_t at = (int64_t)row * p.ldc + col;
  const bool whole = col + 3 < p.n;
  const auto put = [&](auto type) {
    constexpr int CT = decltype(type)::value;
    typename OutOf<CT>::type* c = static_cast<typename OutOf<CT>::type*>(p.c) + at;
    if (whole) {
      put4<CT>(c, v);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < p.n) put1<CT>(c + e, v[e]);
    }
  };
  if (p.c_dtype == kDtypeFp32) put(IntTag<kDtypeFp32>{});
  else if (p.c_dtype == kDtypeBf16) put(IntTag<kDtypeBf16>{});
  else put(IntTag<kDtypeFp16>{});
}

// One element to C.
__device__ __forceinline__ void store1(const ScaledProblem& p, int row, int col, float v) {
  const int64_t at = (int64_t)row * p.ldc + col;
  if (p.c_dtype == kDtypeFp32) static_cast<float*>(p.c)[at] = v;
  else static_cast<uint16_t*>(p.c)[at] = p.c_dtype == kDtypeBf16 ? cvt1<kDtypeBf16>(v) : cvt1<kDtypeFp16>(v);
}

// ---- products of two scales beyond fp32 ---------------------------------------
// The kernels form sa * sb in fp32 (one operation less per element than scaling
// the sums twice).  Where that overflows, a block's contribution becomes
// infinite, or NaN if its sum is 0, although sa * sb * sum may be a finite number
// or 0.  No such result is finite, so a lane whose results all are has nothing
// to do; one that holds another looks whether scales were the cause, and
// computes those elements anew from the operands, in 64 bits.

// `t` if v is four finite numbers, else NaN.
__device__ __forceinline__ float finite_or_nan(f32x4_t v, float t) {
#pragma unroll
  for (int e = 0; e < 4; ++e) t = __builtin_fmaf(v[e], 0.0f, t);
  return t;
}

__device__ __forceinline__ bool overflows(float a, float b) {
  const float inf = __builtin_inff();
  return __builtin_fabsf(a) < inf && __builtin_fabsf(b) < inf && !(__builtin_fabsf(a * b) < inf);
}

// The scales of row `row` (column `col`), one every `step` k blocks.
__device__ __forceinline__ const float* row_scales(const ScaledProblem& p, int row, int64_t& step) {
  const int g = p.by_rows.quotient(row);
  step = p.rows_per_group;
  return p.a_scale[g] + (row - g * p.rows_per_group);
}
__device__ __forceinline__ const float* col_scales(const ScaledProblem& p, int col, int64_t& step) {
  step = p.nb;
  return p.b_scale + (p.b_block_rows == 1 ? col : col >> 7);
}

// The largest finite |scale| of k blocks [b0, b1).
__device__ __forceinline__ float largest(const float* s, int64_t step, int b0, int b1) {
  float top = 0.0f;
#pragma unroll 8
  for (int b = b0; b < b1; ++b) {
    const float v = __builtin_fabsf(s[b * step]);
    top = v < __builtin_inff() ? fmaxf(top, v) : top;
  }
  return top;
}

template <int FMT>
__device__ __forceinline__ void four_values(uint32_t w, float (&v)[4]) {
  if constexpr (FMT == kFmtE4M3) {
    v[0] = __builtin_amdgcn_cvt_f32_fp8(w, 0);
    v[1] = __builtin_amdgcn_cvt_f32_fp8(w, 1);
    v[2] = __builtin_amdgcn_cvt_f32_fp8(w, 2);
    v[3] = __builtin_amdgcn_cvt_f32_fp8(w, 3);
  } else {
    v[0] = __builtin_amdgcn_cvt_f32_bf8(w, 0);
    v[1] = __builtin_amdgcn_cvt_f32_bf8(w, 1);
    v[2] = __builtin_amdgcn_cvt_f32_bf8(w, 2);
    v[3] = __builtin_amdgcn_cvt_f32_bf8(w, 3);
  }
}

// Element (row, col) over k blocks [b0, b1) in 64 bits, into `value`, if a
// product of its scales overflows; else false.
template <int FMTA>
__device__ __forceinline__ bool recompute(const ScaledProblem& p, int row, int col, int b0, int b1, float& value) {
  int64_t sa_step, sb_step;
  const float* sa = row_scales(p, row, sa_step);
  const float* sb = col_scales(p, col, sb_step);
  bool over = false;
#pragma unroll 8
  for (int b = b0; b < b1; ++b) over |= overflows(sa[b * sa_step], sb[b * sb_step]);
  if (!over) return false;
  const int g = p.by_rows.quotient(row);
  const char* qa = static_cast<const char*>(p.a_group[g]) + (int64_t)(row - g * p.rows_per_group) * p.a_ld;
  const char* qb = static_cast<const char*>(p.b) + (int64_t)col * p.ldb;
  double sum = 0.0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    double part = 0.0;
    const int end = min(p.k16, b * 128 + 128);
#pragma unroll 1
    for (int k = b * 128; k < end; k += 4) {
      float x[4], y[4];
      four_values<FMTA>(*reinterpret_cast<const uint32_t*>(qa + k), x);
      four_values<kFmtE4M3>(*reinterpret_cast<const uint32_t*>(qb + k), y);
#pragma unroll
      for (int e = 0; e < 4; ++e) part += (double)x[e] * (double)y[e];
    }
    sum += (double)sa[b * sa_step] * (double)sb[b * sb_step] * part;
  }
  value = (float)sum;
  return true;
}

// Tile and k range of a workgroup: k ranges outermost; of a range, XCD x
// (workgroup id mod 8) takes consecutive tiles, in groups of group_m row
// blocks walked column by column.
__device__ __forceinline__ void tile_of(const ScaledProblem& p, int wg, int& rb, int& cb, int& split) {
  const int ntiles = p.order.num_rb * p.order.num_cb;
  split = p.by_tiles.quotient(wg);
  wg -= split * ntiles;
  const int xcd = wg & 7, per = ntiles >> 3, rem = ntiles & 7;
  wg = xcd * per + min(xcd, rem) + (wg >> 3);
  const int grp = p.by_group.quotient(wg);
  const int first = grp * p.order.group_m, rows = min(p.order.num_rb - first, p.order.group_m);
  const int in = wg - grp * p.order.group_m * p.order.num_cb;
  cb = (rows == p.order.group_m ? p.by_full : p.by_last).quotient(in);
  rb = first + in - cb * rows;
}

// BM x BN output tile, WM x WN waves, NST k-tiles in LDS.  WIDE: bf16 MFMAs.
template <int FMTA, bool BROW, bool WIDE, int BM, int BN, int WM, int WN, int NST, int OCC>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
void scaled_gemm_kernel(ScaledProblem p) {
  constexpr int WAVES = WM * WN;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
  constexpr int AL = A_BYTES / 1024 / WAVES, BL = B_BYTES / 1024 / WAVES;   // 1 KiB loads per wave and k-tile
  static_assert(BM + BN == 64 * WAVES, "one scale per lane of the workgroup");
  static_assert(AL >= 1 && BL >= 1 && BM % 64 == 0, "tile too small for the load split");
  static_assert(NST * (AL + BL + 1) < 64, "vmcnt range");
  // [stage][A tile, B tile], then [stage][row scales, column scales]
  __shared__ __attribute__((aligned(1024))) char smem[NST * (STAGE + (BM + BN) * 4)];
  char* const sc = smem + NST * STAGE;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int g4 = lane >> 4, i16 = lane & 15;
  int rb, cb, split;
  tile_of(p, blockIdx.x, rb, cb, split);
  const int m0 = rb * BM, n0 = cb * BN;
  const int t0 = split * p.kb_per_split;
  const int nk = min(p.kb, t0 + p.kb_per_split) - t0;
  const int rpg = p.rows_per_group;
  const char* zero = reinterpret_cast<const char*>(g_zero_chunk);

  // ---- this lane's loads -----------------------------------------------------
  // Instruction j of this wave fills rows 8 (wave * AL + j) + lane / 8 of its
  // tile; position lane % 8 holds chunk (lane % 8) ^ swz_k16(row).  The scales
  // of a k-tile are LDS words [BM + BN], one per thread; row scales sit in the
  // order a lane reads them: word wm*TM + i16*FM + i is row wm*TM + 16i + i16.
  const int pos = lane & 7;
  auto a_row = [&](int j) { return (wave * AL + j) * 8 + (lane >> 3); };
  auto b_row = [&](int j) { return (wave * BL + j) * 8 + (lane >> 3); };
  auto chunk = [&](int r) { return (pos ^ swz_k16(r)) * 16; };
  const int s_row = (tid / TM) * TM + 16 * ((tid % TM) % FM) + (tid % TM) / FM;   // waves of row scales

  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char_t*)smem;
  const uint32_t lds_a = lds0 + wave * (AL * 1024), lds_b = lds0 + A_BYTES + wave * (BL * 1024);
  const uint32_t lds_s = lds0 + NST * STAGE + wave * 256;
  const int kend = p.k16 - t0 * 128;               // bytes of a row from k-tile t0 on

  // Tiles wholly inside one shard, n and k load through buffer descriptors
  // over the tile's rows (scalar base and k offset, 32-bit lane offsets).
  const int g0 = p.by_rows.quotient(m0), in0 = m0 - g0 * rpg;
  const int64_t a_span = (int64_t)(BM - 1) * p.a_ld + nk * 128, b_span = (int64_t)(BN - 1) * p.ldb + nk * 128;
  const int s_ld = wave * 64 < BM ? rpg : p.nb;    // this wave's scales: rows or columns
  const int64_t s_span = ((int64_t)(nk - 1) * s_ld + 256) * 4;
  const bool fast = m0 + BM <= p.m && n0 + BN <= p.n && in0 + BM <= rpg && nk * 128 <= kend && p.a_ld >= 128 &&
                    p.ldb >= 128 && a_span < (1ll << 32) && b_span < (1ll << 32) && s_span < (1ll << 32);

  // ---- LDS fragment offsets ----------------------------------------------------
  // rows of consecutive 16-row blocks have the same swizzle (it depends on
  // row bits 1-3), so one lane offset serves every block
  const int fx = swz_k16(i16);
  const int f_lo = i16 * 128 + ((g4 ^ fx) << 4), f_hi = i16 * 128 + (((4 + g4) ^ fx) << 4);
  const int a_base = wm * TM * 128, b_base = A_BYTES + wn * TN * 128;

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto body = [&](auto tag) {
    constexpr bool FAST = decltype(tag)::value;
    constexpr int LOADS = AL + BL + 1;
    u32x4_t rsrc_a{}, rsrc_b{}, rsrc_s{};
    uint32_t a_voff[AL], b_voff[BL], s_voff = 0;
    const char *a_src[AL], *b_src[BL], *s_src = zero;
    uint32_t ok_bits = 0;
    int64_t s_step = 0;
    if constexpr (FAST) {
      // offsets shifted for load_lds16_buf_j
      rsrc_a = buffer_rsrc(static_cast<const char*>(p.a_group[g0]) + (int64_t)in0 * p.a_ld + (int64_t)t0 * 128, a_span);
      rsrc_b = buffer_rsrc(static_cast<const char*>(p.b) + (int64_t)n0 * p.ldb + (int64_t)t0 * 128, b_span);
      if (wave * 64 < BM) {
        rsrc_s = buffer_rsrc(p.a_scale[g0] + (int64_t)t0 * rpg + in0, s_span);
        s_voff = s_row * 4;
      } else {
        rsrc_s = buffer_rsrc(p.b_scale + (int64_t)t0 * p.nb + (BROW ? n0 : n0 >> 7), s_span);
        s_voff = (BROW ? tid - BM : (tid - BM) >> 7) * 4;
      }
#pragma unroll
      for (int j = 0; j < AL; ++j)
        a_voff[j] = (uint32_t)((int64_t)a_row(j) * p.a_ld + chunk(a_row(j)) - (j & 3) * 1024);
#pragma unroll
      for (int j = 0; j < BL; ++j)
        b_voff[j] = (uint32_t)((int64_t)b_row(j) * p.ldb + chunk(b_row(j)) - (j & 3) * 1024);
    } else {
      // rows past the end keep the last row's address and are never read; all
      // pointer loads of a lane are on their way at once
#pragma unroll
      for (int j = 0; j < AL; ++j) {
        const int gi = m0 + a_row(j), gc = min(gi, p.m - 1), g = p.by_rows.quotient(gc);
        a_src[j] = static_cast<const char*>(p.a_group[g]) + (int64_t)(gc - g * rpg) * p.a_ld + (int64_t)t0 * 128 +
                   chunk(a_row(j));
        ok_bits |= (uint32_t)(gi < p.m) << j;
      }
#pragma unroll
      for (int j = 0; j < BL; ++j) {
        const int gn = n0 + b_row(j);
        b_src[j] = static_cast<const char*>(p.b) + (int64_t)min(gn, p.n - 1) * p.ldb + (int64_t)t0 * 128 +
                   chunk(b_row(j));
        ok_bits |= (uint32_t)(gn < p.n) << (AL + j);
      }
      if (wave * 64 < BM) {
        const int gi = m0 + s_row, gc = min(gi, p.m - 1), g = p.by_rows.quotient(gc);
        const float* src = p.a_scale[g] + (int64_t)t0 * rpg + (gc - g * rpg);
        s_src = gi < p.m ? reinterpret_cast<const char*>(src) : zero;
        s_step = gi < p.m ? (int64_t)rpg * 4 : 0;
      } else {
        const int gn = n0 + tid - BM;
        const float* src = p.b_scale + (int64_t)t0 * p.nb + (BROW ? min(gn, p.n - 1) : min(gn, p.n - 1) >> 7);
        s_src = gn < p.n ? reinterpret_cast<const char*>(src) : zero;
        s_step = gn < p.n ? (int64_t)p.nb * 4 : 0;
      }
    }
    // load number d of k-tile t (relative) into stage st: A, B, then scales;
    // k-tiles past the end read the last one again into a stage nobody reads
    auto issue = [&](int d, int st, int t) {
      const int tc = t < nk ? t : nk - 1;
      if (d < AL) {
        if constexpr (FAST) {
          load_lds16_buf_j(d, rsrc_a, a_voff[d < AL ? d : 0], tc * 128, lds_a + st * STAGE);
        } else {
          const int j = d < AL ? d : 0;
          const bool ok = (((ok_bits >> j) & 1) != 0) & (tc * 128 + chunk(a_row(j)) < kend);
          load_lds16_at(ok ? a_src[j] + (int64_t)tc * 128 : zero, lds_a + st * STAGE + j * 1024);
        }
      } else if (d < AL + BL) {
        const int j = d >= AL && d < AL + BL ? d - AL : 0;
        if constexpr (FAST) {
          load_lds16_buf_j(j, rsrc_b, b_voff[j], tc * 128, lds_b + st * STAGE);
        } else {
          const bool ok = (((ok_bits >> (AL + j)) & 1) != 0) & (tc * 128 + chunk(b_row(j)) < kend);
          load_lds16_at(ok ? b_src[j] + (int64_t)tc * 128 : zero, lds_b + st * STAGE + j * 1024);
        }
      } else {
        if constexpr (FAST)
          load_lds4_buf(rsrc_s, s_voff, (uint32_t)((int64_t)tc * s_ld * 4), lds_s + st * (BM + BN) * 4);
        else
          load_lds4_at(s_src + tc * s_step, lds_s + st * (BM + BN) * 4);
      }
    };
    auto read_frag = [&](const char* base, u32x4_t (&f)[2]) {
      f[0] = *reinterpret_cast<const u32x4_t*>(base + f_lo);
      f[1] = *reinterpret_cast<const u32x4_t*>(base + f_hi);
    };
    u32x4_t bf[FN][2], af[2][2];
    bf16x8_t bw[WIDE ? FN : 1][4], aw[4];
    f32x4_t part[FN];
    float sa[FM], sa_last = 0.0f;
    f32x4_t sb[BROW ? FN : 1];
    // block (i, j)'s accumulators += its scaled product
    auto add = [&](int i, int j, float f) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[i][j][e] += (BROW ? f * sb[BROW ? j : 0][e] : f) * part[j][e];
    };
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      part[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (BROW) sb[BROW ? j : 0] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }

    // Schedule.  One slot per product: the FMAs of the product FN slots ago,
    // the product, then the slot's memory operation, fenced so that it stays
    // there.  Slots of block row i < FM - 1 read A fragment i + 1 (first slot);
    // before the last block row the workgroup synchronises (all reads of
    // k-tile t are done, the loads of t + 1 have landed), and its slots read
    // the first fragments of k-tile t + 1 and begin to refill t's stage; the
    // other loads of that refill ride on the first slots of t + 1, where the
    // scales are read too.
    constexpr int EARLY = FN - 1;   // refill loads in the last block row
    static_assert(EARLY + (FM - 1) * FN >= LOADS, "every refill is issued before the next synchronisation");
    for (int t = 0; t < NST - 1; ++t)
#pragma unroll
      for (int d = 0; d < LOADS; ++d) issue(d, t, t);
#pragma unroll
    for (int d = 0; d < EARLY; ++d) issue(d, NST - 1, NST - 1);
    wait_vmcnt<(NST - 2) * LOADS + EARLY>();
    block_barrier();
    read_frag(smem + a_base, af[0]);
#pragma unroll
    for (int j = 0; j < FN; ++j) read_frag(smem + b_base + j * 2048, bf[j]);
    int st = 0, prev = NST - 1;                    // stages of k-tiles t and t - 1
    for (int t = 0; t < nk; ++t) {
      const int sn = st + 1 == NST ? 0 : st + 1;
      const char* cur = smem + st * STAGE;
      const char* nxt = smem + sn * STAGE;
      const float* s = reinterpret_cast<const float*>(sc + st * (BM + BN) * 4);
      float b128 = 0.0f;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if (i == FM - 1) {
          wait_vmcnt<(NST - 2) * LOADS>();
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          block_barrier();
        }
        if constexpr (WIDE) {
          // the four MFMAs of a block depend on each other: block by block in
          // turn, scheduled by the compiler within the block row
          widen<FMTA>(af[i & 1], aw);
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            if (i == 0) widen<kFmtE4M3>(bf[j], bw[j]);
            add(i > 0 ? i - 1 : FM - 1, j, i > 0 ? sa[i > 0 ? i - 1 : 0] : sa_last);
            part[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < FN; ++j)
              part[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bw[j][q], aw[q], part[j], 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if constexpr (!WIDE) {
            if (i > 0) add(i - 1, j, sa[i - 1]);
            else add(FM - 1, j, sa_last);          // of the previous k-tile
            part[j] = mfma128<FMTA>(bf[j], af[i & 1]);
          }
          if (i < FM - 1) {
            if (j == 0) read_frag(cur + a_base + (i + 1) * 2048, af[(i + 1) & 1]);
            const int d = EARLY + i * FN + j;
            if (d < LOADS) issue(d < LOADS ? d : 0, prev, t - 1 + NST);
            if (i == 0) {
              if (j == 1) {
#pragma unroll
                for (int q = 0; q < FM; q += 4) {
                  const f32x4_t v = *reinterpret_cast<const f32x4_t*>(s + wm * TM + i16 * FM + q);
#pragma unroll
                  for (int e = 0; e < 4; ++e) sa[q + e] = v[e];
                }
                if constexpr (!BROW) b128 = s[BM + wn * TN];   // one scale per 128 columns
              }
              if constexpr (BROW) sb[j] = *reinterpret_cast<const f32x4_t*>(s + BM + wn * TN + 16 * j + 4 * g4);
              if constexpr (!BROW)
                if (j == FN - 1)
#pragma unroll
                  for (int q = 0; q < FM; ++q) sa[q] *= b128;
            }
          } else {
            if (j == 0) read_frag(nxt + a_base, af[FM & 1]);
            read_frag(nxt + b_base + j * 2048, bf[j]);
            if (j > 0) issue(j > 0 ? j - 1 : 0, st, t + NST);
          }
          if (!WIDE || j == FN - 1) __builtin_amdgcn_sched_barrier(0);
        }
      }
      sa_last = sa[FM - 1];
      prev = st;
      st = sn;
      static_assert(FM % 4 == 0, "two sets of A fragments alternate by row block; scales are read by fours");
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) add(FM - 1, j, sa_last);
    wait_vmcnt<0>();
  };
  if (fast) body(BoolTag<true>{});
  else body(BoolTag<false>{});

  // ---- epilogue: acc[i][j][e] = C[m0 + wm*TM + 16i + i16][n0 + wn*TN + 16j + 4*g4 + e]
  const int row0 = m0 + wm * TM + i16, col0 = n0 + wn * TN + 4 * g4;
  const bool split_k = p.splits > 1;
  const int64_t ld = split_k ? p.part_ld : p.ldc;
  const int ncols = split_k ? (int)p.part_ld : p.n;   // padding columns of the sums are never read as results
  const bool inside = m0 + BM <= p.m && n0 + BN <= ncols;
  const auto store = [&](auto type) {
    constexpr int CT = decltype(type)::value;
    typedef typename OutOf<CT>::type out_t;
    out_t* base = static_cast<out_t*>(split_k ? p.partials + (int64_t)split * p.m * ld : p.c) + (int64_t)row0 * ld + col0;
#pragma unroll
    for (int i = 0; i < FM; ++i, base += 16 * ld)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if (inside) {
          put4<CT>(base + 16 * j, acc[i][j]);
        } else if (row0 + 16 * i < p.m && col0 + 16 * j + 4 <= ncols) {
          put4<CT>(base + 16 * j, acc[i][j]);
        } else if (row0 + 16 * i < p.m) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col0 + 16 * j + e < p.n) put1<CT>(base + 16 * j + e, acc[i][j][e]);
        }
      }
  };
  if (split_k || p.c_dtype == kDtypeFp32) store(IntTag<kDtypeFp32>{});
  else if (p.c_dtype == kDtypeBf16) store(IntTag<kDtypeBf16>{});
  else store(IntTag<kDtypeFp16>{});

  float all = 0.0f;
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) all = finite_or_nan(acc[i][j], all);
  if (all == 0.0f) return;
  float top_a = 0.0f, top_b = 0.0f;
  int64_t step;
#pragma unroll 1
  for (int i = 0; i < FM; ++i)
    if (row0 + 16 * i < p.m) top_a = fmaxf(top_a, largest(row_scales(p, row0 + 16 * i, step), step, t0, t0 + nk));
#pragma unroll 1
  for (int c = 0; c < FN * 4; ++c) {
    const int col = col0 + 16 * (c >> 2) + (c & 3);
    if (col < p.n) top_b = fmaxf(top_b, largest(col_scales(p, col, step), step, t0, t0 + nk));
  }
  if (!overflows(top_a, top_b)) return;
#pragma unroll 1
  for (int u = 0; u < FM * FN * 4; ++u) {
    const int row = row0 + 16 * (u / (FN * 4)), col = col0 + 16 * (u / 4 % FN) + u % 4;
    float v;
    if (row >= p.m || col >= p.n || !recompute<FMTA>(p, row, col, t0, t0 + nk, v)) continue;
    if (split_k) p.partials[((int64_t)split * p.m + row) * p.part_ld + col] = v;
    else store1(p, row, col, v);
  }
}

// Few rows: ROWS x COLS outputs per workgroup, over all of k or one of
// p.splits ranges of it.  The waves take the k-tiles round robin, each through
// its own LDS ring; a slot holds ROWS + COLS rows of 128 bytes and their
// scales (word l: row l, then column l - ROWS).
template <int FMTA, int ROWS, int COLS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(WAVES / 4, WAVES / 4)))
void scaled_skinny_kernel(ScaledProblem p) {
  constexpr int SL = (ROWS + COLS + 63) / 64;                 // loads of scales
  constexpr int AL = ROWS / 8, BL = COLS / 8, LOADS = AL + BL + SL;
  constexpr int SLOT = (ROWS + COLS) * 128 + SL * 256;
  constexpr int FIT = 160 * 1024 / WAVES / SLOT, SLOTS = FIT < 6 ? FIT : 6;
  constexpr int WAVE_LDS = SLOTS * SLOT;
  constexpr int FM = ROWS / 16, FN = COLS / 16;
  static_assert(SLOTS >= 2 && SLOTS * LOADS < 64, "ring");
  __shared__ __attribute__((aligned(1024))) char smem[WAVES * WAVE_LDS];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int tile, split;
  {
    // XCD x (workgroup id mod 8) takes a contiguous range, row blocks
    // fastest: the row blocks of one column block share its L2
    const int ntiles = p.order.num_rb * p.order.num_cb;
    const int T = ntiles * p.splits, wg = blockIdx.x;
    const int xcd = wg & 7, local = wg >> 3, per = T >> 3, rem = T & 7;
    const int u = xcd * per + min(xcd, rem) + local;
    split = p.by_tiles.quotient(u);
    tile = u - split * ntiles;
  }
  const int cb = p.by_group.quotient(tile);
  const int row0 = (tile - cb * p.order.num_rb) * ROWS, n0 = cb * COLS;
  const int t0 = split * p.kb_per_split, t1 = min(p.kb, t0 + p.kb_per_split);
  const int rpg = p.rows_per_group;
  const char* zero = reinterpret_cast<const char*>(g_zero_chunk);

  // rows and columns past the end keep the last one's address and are never
  // read; all pointer loads of a lane are on their way at once
  const char* a_src[AL];
  const char* b_src[BL];
  uint32_t ok_bits = 0;
#pragma unroll
  for (int q = 0; q < AL; ++q) {
    const int r = 8 * q + (lane >> 3), gr = row0 + r, gc = min(gr, p.m - 1), g = p.by_rows.quotient(gc);
    a_src[q] = static_cast<const char*>(p.a_group[g]) + (int64_t)(gc - g * rpg) * p.a_ld + ((lane & 7) ^ swz_k16(r)) * 16;
    ok_bits |= (uint32_t)(gr < p.m) << q;
  }
#pragma unroll
  for (int q = 0; q < BL; ++q) {
    const int r = 8 * q + (lane >> 3), gn = n0 + r;
    b_src[q] = static_cast<const char*>(p.b) + (int64_t)min(gn, p.n - 1) * p.ldb + ((lane & 7) ^ swz_k16(r)) * 16;
    ok_bits |= (uint32_t)(gn < p.n) << (AL + q);
  }
  const char* s_src[SL];
  int64_t s_step[SL];
#pragma unroll
  for (int q = 0; q < SL; ++q) {
    const int l = 64 * q + lane;
    const int gr = row0 + l, gn = n0 + l - ROWS;
    const int gc = min(gr, p.m - 1), g = p.by_rows.quotient(gc);
    const int cn = min(max(gn, 0), p.n - 1);
    const float* as = p.a_scale[g] + (gc - g * rpg);
    const float* bs = p.b_scale + (p.b_block_rows == 1 ? cn : cn >> 7);
    const bool is_a = l < ROWS, ok = is_a ? gr < p.m : l < ROWS + COLS && gn < p.n;
    s_src[q] = ok ? reinterpret_cast<const char*>(is_a ? as : bs) : zero;
    s_step[q] = ok ? (int64_t)(is_a ? rpg : p.nb) * 4 : 0;
  }

  char* const ring = smem + wave * WAVE_LDS;
  const uint32_t ring_lds = (uint32_t)(uintptr_t)(lds_char_t*)ring;
  const int nt = t1 - t0 > wave ? (t1 - t0 - wave + WAVES - 1) / WAVES : 0;
  auto issue = [&](int j) {   // this wave's k-tile number j
    const int t = t0 + wave + WAVES * j;
    const uint32_t dst = ring_lds + (j % SLOTS) * SLOT;
    const int64_t off = (int64_t)t * 128;
#pragma unroll
    for (int q = 0; q < AL + BL; ++q) {
      const int r = 8 * (q < AL ? q : q - AL) + (lane >> 3);
      const bool ok = (((ok_bits >> q) & 1) != 0) & (t * 128 + ((lane & 7) ^ swz_k16(r)) * 16 < p.k16);
      load_lds16_at(ok ? (q < AL ? a_src[q < AL ? q : 0] : b_src[q < AL ? 0 : q - AL]) + off : zero, dst + q * 1024);
    }
#pragma unroll
    for (int q = 0; q < SL; ++q) load_lds4_at(s_src[q] + (int64_t)t * s_step[q], dst + (ROWS + COLS) * 128 + q * 256);
  };

  const int g4 = lane >> 4, i16 = lane & 15;
  const int fx = swz_k16(i16);
  const int f_lo = i16 * 128 + ((g4 ^ fx) << 4), f_hi = i16 * 128 + (((4 + g4) ^ fx) << 4);
  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  __builtin_amdgcn_sched_barrier(0);
  const int pre = nt < SLOTS ? nt : SLOTS;
  for (int j = 0; j < pre; ++j) issue(j);
  for (int j = 0; j < nt; ++j) {
    // k-tiles after j still allowed in flight
    const int after = min(SLOTS - 1, nt - 1 - j);
    switch (after) {
      case 0: wait_vmcnt<0>(); break;
      case 1: wait_vmcnt<LOADS>(); break;
      case 2: wait_vmcnt<(SLOTS > 2 ? 2 : 1) * LOADS>(); break;
      case 3: wait_vmcnt<(SLOTS > 3 ? 3 : 1) * LOADS>(); break;
      case 4: wait_vmcnt<(SLOTS > 4 ? 4 : 1) * LOADS>(); break;
      default: wait_vmcnt<(SLOTS > 5 ? 5 : 1) * LOADS>(); break;
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    const char* slot = ring + (j % SLOTS) * SLOT;
    u32x4_t af[FM][2], bf[FN][2];
    float sa[FM];
    f32x4_t sb[FN];
    const float* s = reinterpret_cast<const float*>(slot + (ROWS + COLS) * 128);
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      bf[f][0] = *reinterpret_cast<const u32x4_t*>(slot + (ROWS + 16 * f) * 128 + f_lo);
      bf[f][1] = *reinterpret_cast<const u32x4_t*>(slot + (ROWS + 16 * f) * 128 + f_hi);
      sb[f] = *reinterpret_cast<const f32x4_t*>(s + ROWS + 16 * f + 4 * g4);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      af[i][0] = *reinterpret_cast<const u32x4_t*>(slot + 16 * i * 128 + f_lo);
      af[i][1] = *reinterpret_cast<const u32x4_t*>(slot + 16 * i * 128 + f_hi);
      sa[i] = s[16 * i + i16];
    }
    // the slot's refill goes out as soon as its k-tile is in registers
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    if (j + SLOTS < nt) issue(j + SLOTS);
    bf16x8_t bw[FN][4];
#pragma unroll
    for (int f = 0; f < FN; ++f) widen<kFmtE4M3>(bf[f], bw[f]);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      bf16x8_t aw[4];
      widen<FMTA>(af[i], aw);
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        const f32x4_t d = mfma128_wide(bw[f], aw);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][f][e] += (sa[i] * sb[f][e]) * d[e];
      }
    }
  }
  wait_vmcnt<0>();
  asm volatile("" ::: "memory");

  // the waves' sums, added in wave order
  constexpr int RLD = COLS + 4;
  static_assert(ROWS * RLD * 4 <= WAVE_LDS, "partial tile fits the wave's ring");
  float* red = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int f = 0; f < FN; ++f)
      *reinterpret_cast<f32x4_t*>(red + (16 * i + i16) * RLD + 16 * f + 4 * g4) = acc[i][f];
  __syncthreads();
  float all = 0.0f;
  for (int e4 = tid; e4 < ROWS * COLS / 4; e4 += 64 * WAVES) {
    const int r = e4 / (COLS / 4), c = (e4 % (COLS / 4)) * 4;
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(smem) + r * RLD + c);
#pragma unroll
    for (int w = 1; w < WAVES; ++w)
      v += *reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(smem + w * WAVE_LDS) + r * RLD + c);
    const int row = row0 + r, col = n0 + c;
    if (row >= p.m || col >= p.n) continue;
    all = finite_or_nan(v, all);
    if (p.splits > 1) {
      *reinterpret_cast<f32x4_t*>(p.partials + ((int64_t)split * p.m + row) * p.part_ld + col) = v;
    } else {
      store4(p, row, col, v);
    }
  }
  if (all == 0.0f) return;
#pragma unroll 1
  for (int e = 4 * tid; e < ROWS * COLS; e += e % 4 == 3 ? 256 * WAVES - 3 : 1) {
    const int row = row0 + e / COLS, col = n0 + e % COLS;
    float v;
    if (row >= p.m || col >= p.n || !recompute<FMTA>(p, row, col, t0, t1, v)) continue;
    if (p.splits > 1) p.partials[((int64_t)split * p.m + row) * p.part_ld + col] = v;
    else store1(p, row, col, v);
  }
}

// Sum of the k ranges in order, four columns per thread.
__global__ __launch_bounds__(256) void scaled_reduce_kernel(ScaledProblem p) {
  const int n4 = (int)(p.part_ld / 4);
  const int64_t plane = (int64_t)p.m * p.part_ld;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < (int64_t)p.m * n4; u += (int64_t)gridDim.x * 256) {
    const int row = (int)(u / n4), col = (int)(u % n4) * 4;
    const float* src = p.partials + (int64_t)row * p.part_ld + col;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    // eight ranges are on their way at a time, added in order
    for (int s0 = 0; s0 < p.splits; s0 += 8) {
      f32x4_t w[8];
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s0 + s < p.splits) w[s] = *reinterpret_cast<const f32x4_t*>(src + (s0 + s) * plane);
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s0 + s < p.splits) v += w[s];
    }
    store4(p, row, col, v);
  }
}

template <int FMTA, bool BROW>
hipError_t launch_tile(const ScaledProblem& p, int tile, hipStream_t stream) {
  const int64_t grid = (int64_t)p.order.num_rb * p.order.num_cb * p.splits;
#define AGMM_SCALED(WIDE, BM, BN, WM, WN, NST, OCC)                                                             \
  hipLaunchKernelGGL((scaled_gemm_kernel<FMTA, BROW, WIDE, BM, BN, WM, WN, NST, OCC>), dim3((unsigned)grid),   \
                     dim3(64 * WM * WN), 0, stream, p)
  if (tile == kScaled256) AGMM_SCALED(false, 256, 256, 2, 4, 2, 2);
  else if (p.wide && p.deep) AGMM_SCALED(true, 128, 128, 2, 2, 4, 2);
  else if (p.wide) AGMM_SCALED(true, 128, 128, 2, 2, 2, 2);
  else if (p.deep) AGMM_SCALED(false, 128, 128, 2, 2, 4, 2);
  else AGMM_SCALED(false, 128, 128, 2, 2, 2, 2);
#undef AGMM_SCALED
  return hipGetLastError();
}

template <int FMTA>
hipError_t launch_skinny(const ScaledProblem& p, int tile, hipStream_t stream) {
  const int rows = scaled_tile_rows(tile), cols = scaled_tile_cols(tile);
  const int64_t grid = (int64_t)((p.m + rows - 1) / rows) * ((p.n + cols - 1) / cols) * p.splits;
  if (tile == kScaledSkinny16n)
    hipLaunchKernelGGL((scaled_skinny_kernel<FMTA, 16, 16, 8>), dim3((unsigned)grid), dim3(512), 0, stream, p);
  else if (tile == kScaledSkinny16)
    hipLaunchKernelGGL((scaled_skinny_kernel<FMTA, 16, 32, 4>), dim3((unsigned)grid), dim3(256), 0, stream, p);
  else if (tile == kScaledSkinny32)
    hipLaunchKernelGGL((scaled_skinny_kernel<FMTA, 32, 32, 4>), dim3((unsigned)grid), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((scaled_skinny_kernel<FMTA, 64, 64, 4>), dim3((unsigned)grid), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_scaled(const ScaledProblem& problem, int tile, hipStream_t stream) {
  ScaledProblem p = problem;
  const int rows = scaled_tile_rows(tile), cols = scaled_tile_cols(tile);
  const int64_t grid = (int64_t)((p.m + rows - 1) / rows) * ((p.n + cols - 1) / cols) * p.splits;
  if (rows == 0 || grid < 1 || grid >= (int64_t(1) << 23) || p.splits < 1 ||
      (p.splits > 1 && (!p.partials || p.part_ld % 4 != 0 || p.part_ld < p.n)) || (int64_t)p.splits * p.kb_per_split < p.kb ||
      (int64_t)(p.splits - 1) * p.kb_per_split >= p.kb || p.k16 % 16 != 0 || p.kb != (p.k16 + 127) / 128 ||
      p.num_groups < 1 || p.num_groups > kMaxGroups || p.order.num_rb != (p.m + rows - 1) / rows ||
      p.order.num_cb != (p.n + cols - 1) / cols || (int64_t)p.num_groups * p.rows_per_group != p.m)
    return hipErrorInvalidValue;
  const int group_m = p.order.group_m;
  if (tile < kScaledSkinny16 && group_m < 1) return hipErrorInvalidValue;
  p.by_rows = FastDiv(p.rows_per_group);
  p.by_tiles = FastDiv(p.order.num_rb * p.order.num_cb);
  if (tile >= kScaledSkinny16) {
    p.by_group = FastDiv(p.order.num_rb);
  } else {
    const int last = p.order.num_rb % group_m;
    p.by_group = FastDiv(group_m * p.order.num_cb);
    p.by_full = FastDiv(group_m);
    p.by_last = FastDiv(last ? last : group_m);
  }
  hipError_t err;
  const bool e5m2 = p.a_format == kFmtE5M2;
  if (tile >= kScaledSkinny16)
    err = e5m2 ? launch_skinny<kFmtE5M2>(p, tile, stream) : launch_skinny<kFmtE4M3>(p, tile, stream);
  else if (p.b_block_rows == 1)
    err = e5m2 ? launch_tile<kFmtE5M2, true>(p, tile, stream) : launch_tile<kFmtE4M3, true>(p, tile, stream);
  else
    err = e5m2 ? launch_tile<kFmtE5M2, false>(p, tile, stream) : launch_tile<kFmtE4M3, false>(p, tile, stream);
  if (err != hipSuccess || p.splits == 1) return err;
  const int64_t blocks = ((int64_t)p.m * ((p.n + 3) / 4) + 255) / 256;
  hipLaunchKernelGGL(scaled_reduce_kernel, dim3((unsigned)(blocks < (1 << 16) ? blocks : (1 << 16))), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace agmm
