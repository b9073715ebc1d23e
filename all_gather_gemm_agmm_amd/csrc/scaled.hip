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
//  * scaled_gemm_kernel: two 128-deep k-tiles in LDS, refilled by global ->
//    LDS loads; the row and column scales of a k-tile ride along as one
//    4-byte-per-lane load per wave.  B fragments of a k-tile stay in
//    registers, A fragments pass through; the FMAs of row block i run beside
//    the MFMAs of row block i + 1.  The workgroup synchronises before the last
//    row block of a k-tile, once every fragment of it has been read, so that
//    the next k-tile's first reads and the refill run beside its MFMAs.
//    VALU and MFMA share the accumulators, which therefore live in ordinary
//    registers: two waves per SIMD with 128 accumulators each.
//  * scaled_skinny_kernel: few rows.  Every wave streams its own k-tiles
//    through a private LDS ring (no barrier in the loop); the waves' sums are
//    added in LDS in a fixed order.
//  * scaled_reduce_kernel: fixed-order sum of k ranges.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "agmm_kernels.h"
#include "gemm_device.h"

namespace agmm {

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// One 16 x 16 block of sums over 128 of k, of a B fragment (first operand,
// e4m3) and an A fragment: lane (g, i) of the result holds row i, columns
// 4g .. 4g + 3.
//  * 8-bit MFMA: one instruction, but its adder aligns the products to the
//    largest of them with few bits to spare: measured on random bytes, the
//    error against the exact sum is 400 u (rms) and up to 3700 u of the sum of
//    the terms' sizes, u = 2^-24, for the 16x16x32 form as for 16x16x128.
//  * bf16 MFMAs on the widened values (both formats are exact in bf16): 0.6 u
//    and 4.4 u, at half the rate.
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

// Four consecutive columns of one row to C in its own type.
__device__ __forceinline__ void store4(const ScaledProblem& p, int row, int col, const f32x4_t& v) {
  const int64_t at = (int64_t)row * p.ldc + col;
  const bool whole = col + 3 < p.n && (p.ldc % 4) == 0;
  if (p.c_dtype == kDtypeFp32) {
    float* c = static_cast<float*>(p.c) + at;
    if (whole) {
      *reinterpret_cast<f32x4_t*>(c) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < p.n) c[e] = v[e];
    }
  } else {
    uint16_t* c = static_cast<uint16_t*>(p.c) + at;
    uint32_t lo, hi;
    if (p.c_dtype == kDtypeBf16) {
      lo = pack2<kDtypeBf16>(v[0], v[1]);
      hi = pack2<kDtypeBf16>(v[2], v[3]);
    } else {
      lo = pack2<kDtypeFp16>(v[0], v[1]);
      hi = pack2<kDtypeFp16>(v[2], v[3]);
    }
    if (whole) {
      *reinterpret_cast<u32x2_t*>(c) = u32x2_t{lo, hi};
    } else {
      if (col + 0 < p.n) c[0] = (uint16_t)lo;
      if (col + 1 < p.n) c[1] = (uint16_t)(lo >> 16);
      if (col + 2 < p.n) c[2] = (uint16_t)hi;
      if (col + 3 < p.n) c[3] = (uint16_t)(hi >> 16);
    }
  }
}

// BM x BN output tile, WM x WN waves.  WIDE: bf16 MFMAs.
template <int FMTA, bool BROW, bool WIDE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2)))
void scaled_gemm_kernel(ScaledProblem p) {
  constexpr int WAVES = WM * WN;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
  constexpr int AL = A_BYTES / 1024 / WAVES, BL = B_BYTES / 1024 / WAVES;   // 1 KiB loads per wave and k-tile
  static_assert(BM + BN == 64 * WAVES, "one scale per lane of the workgroup");
  static_assert(AL >= 1 && BL >= 1 && BM % 64 == 0, "tile too small for the load split");
  // [stage][A tile, B tile], then [stage][row scales, column scales]
  __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE + 2 * (BM + BN) * 4];
  char* const sc = smem + 2 * STAGE;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int g4 = lane >> 4, i16 = lane & 15;
  const int ntiles = p.order.num_rb * p.order.num_cb;
  int wg = blockIdx.x, split = 0;
  if (p.splits > 1) {
    split = wg / ntiles;
    wg -= split * ntiles;
  }
  int rb, cb;
  tile_coords(p.order, wg, ntiles, rb, cb);
  const int m0 = rb * BM, n0 = cb * BN;
  const int t0 = split * p.kb_per_split;
  const int nk = min(p.kb, t0 + p.kb_per_split) - t0;
  const int rpg = p.rows_per_group;
  const char* zero = reinterpret_cast<const char*>(g_zero_chunk);

  // ---- sources of this lane's loads ------------------------------------------
  // Instruction j of this wave fills rows 8 (wave * AL + j) + lane / 8 of its
  // tile; position lane % 8 holds chunk (lane % 8) ^ swz_k16(row).
  const char* a_src[AL];
  const char* b_src[BL];
  uint32_t ok_bits = 0;
  const int pos = lane & 7;
  // chunk of the row: the same for every instruction up to row bits 0-3
  int a_kc[AL], b_kc[BL];
#pragma unroll
  for (int j = 0; j < AL; ++j) {
    const int r = (wave * AL + j) * 8 + (lane >> 3);
    const int c = pos ^ swz_k16(r);
    a_kc[j] = c * 16;
    a_src[j] = zero;
    const int gi = m0 + r;
    if (gi < p.m) {
      const int g = gi / rpg, t = gi - g * rpg;
      a_src[j] = static_cast<const char*>(p.a_group[g]) + (int64_t)t * p.a_ld + (int64_t)t0 * 128 + c * 16;
      ok_bits |= 1u << j;
    }
  }
#pragma unroll
  for (int j = 0; j < BL; ++j) {
    const int r = (wave * BL + j) * 8 + (lane >> 3);
    const int c = pos ^ swz_k16(r);
    b_kc[j] = c * 16;
    b_src[j] = zero;
    const int gn = n0 + r;
    if (gn < p.n) {
      b_src[j] = static_cast<const char*>(p.b) + (int64_t)gn * p.ldb + (int64_t)t0 * 128 + c * 16;
      ok_bits |= 1u << (AL + j);
    }
  }
  // Scale of this thread: LDS word tid of a k-tile's [BM + BN].  Row scales
  // sit in the order a lane reads them: word wm*TM + i16*FM + i is row
  // wm*TM + 16i + i16.
  const char* s_src = zero;
  int64_t s_step = 0;
  if (tid < BM) {
    const int in = tid % TM;
    const int gi = m0 + (tid / TM) * TM + 16 * (in % FM) + in / FM;
    if (gi < p.m) {
      const int g = gi / rpg;
      s_src = reinterpret_cast<const char*>(p.a_scale[g] + (int64_t)t0 * rpg + (gi - g * rpg));
      s_step = (int64_t)rpg * 4;
    }
  } else {
    const int gn = n0 + tid - BM;
    if (gn < p.n) {
      s_src = reinterpret_cast<const char*>(p.b_scale + (int64_t)t0 * p.nb + (BROW ? gn : gn >> 7));
      s_step = (int64_t)p.nb * 4;
    }
  }

  // Tiles wholly inside one shard, n and k: buffer descriptors over the tile's
  // rows (scalar base and k offset, 32-bit lane offsets), offsets shifted for
  // load_lds16_buf_j.  `s_` is the wave's scale array: its rows or columns.
  const int g0 = m0 / rpg, in0 = m0 - g0 * rpg;
  const int kend = p.k16 - t0 * 128;               // bytes of a row from k-tile t0 on
  const int64_t a_span = (int64_t)(BM - 1) * p.a_ld + nk * 128, b_span = (int64_t)(BN - 1) * p.ldb + nk * 128;
  const int s_ld = wave * 64 < BM ? rpg : p.nb;
  const int64_t s_span = ((int64_t)(nk - 1) * s_ld + 256) * 4;
  const bool fast = m0 + BM <= p.m && n0 + BN <= p.n && in0 + BM <= rpg && nk * 128 <= kend && p.a_ld >= 128 &&
                    p.ldb >= 128 && a_span < (1ll << 32) && b_span < (1ll << 32) && s_span < (1ll << 32);
  u32x4_t rsrc_a{}, rsrc_b{}, rsrc_s{};
  uint32_t a_voff[AL], b_voff[BL], s_voff = 0;
  if (fast) {
    rsrc_a = buffer_rsrc(static_cast<const char*>(p.a_group[g0]) + (int64_t)in0 * p.a_ld + (int64_t)t0 * 128, a_span);
    rsrc_b = buffer_rsrc(static_cast<const char*>(p.b) + (int64_t)n0 * p.ldb + (int64_t)t0 * 128, b_span);
    if (wave * 64 < BM) {
      const int in = tid % TM;
      rsrc_s = buffer_rsrc(p.a_scale[g0] + (int64_t)t0 * rpg + in0, s_span);
      s_voff = ((tid / TM) * TM + 16 * (in % FM) + in / FM) * 4;
    } else {
      rsrc_s = buffer_rsrc(p.b_scale + (int64_t)t0 * p.nb + (BROW ? n0 : n0 >> 7), s_span);
      s_voff = (BROW ? tid - BM : (tid - BM) >> 7) * 4;
    }
  }
#pragma unroll
  for (int j = 0; j < AL; ++j) {
    const int r = (wave * AL + j) * 8 + (lane >> 3);
    a_voff[j] = (uint32_t)((int64_t)r * p.a_ld + a_kc[j] - (j & 3) * 1024);
  }
#pragma unroll
  for (int j = 0; j < BL; ++j) {
    const int r = (wave * BL + j) * 8 + (lane >> 3);
    b_voff[j] = (uint32_t)((int64_t)r * p.ldb + b_kc[j] - (j & 3) * 1024);
  }

  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char_t*)smem;
  const uint32_t lds_a = lds0 + wave * (AL * 1024), lds_b = lds0 + A_BYTES + wave * (BL * 1024);
  const uint32_t lds_s = lds0 + 2 * STAGE + wave * 256;

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
    // loads of k-tile t (relative) into stage st; k-tiles past the end read
    // the last one again into a stage nobody reads
    auto issue = [&](int st, int t) {
      const int tc = t < nk ? t : nk - 1;
      if constexpr (FAST) {
#pragma unroll
        for (int j = 0; j < AL; ++j) load_lds16_buf_j(j, rsrc_a, a_voff[j], tc * 128, lds_a + st * STAGE);
#pragma unroll
        for (int j = 0; j < BL; ++j) load_lds16_buf_j(j, rsrc_b, b_voff[j], tc * 128, lds_b + st * STAGE);
        load_lds4_buf(rsrc_s, s_voff, (uint32_t)((int64_t)tc * s_ld * 4), lds_s + st * (BM + BN) * 4);
      } else {
        const int64_t off = (int64_t)tc * 128;
#pragma unroll
        for (int j = 0; j < AL; ++j) {
          const bool ok = ((ok_bits >> j) & 1) && tc * 128 + a_kc[j] < kend;
          load_lds16_at(ok ? a_src[j] + off : zero, lds_a + st * STAGE + j * 1024);
        }
#pragma unroll
        for (int j = 0; j < BL; ++j) {
          const bool ok = ((ok_bits >> (AL + j)) & 1) && tc * 128 + b_kc[j] < kend;
          load_lds16_at(ok ? b_src[j] + off : zero, lds_b + st * STAGE + j * 1024);
        }
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
    float sa[FM];
    f32x4_t sb[BROW ? FN : 1];
    auto read_scales = [&](int st) {
      const float* s = reinterpret_cast<const float*>(sc + st * (BM + BN) * 4);
#pragma unroll
      for (int i = 0; i < FM; i += 4) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(s + wm * TM + i16 * FM + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) sa[i + e] = v[e];
      }
      if constexpr (BROW) {
#pragma unroll
        for (int j = 0; j < FN; ++j) sb[j] = *reinterpret_cast<const f32x4_t*>(s + BM + wn * TN + 16 * j + 4 * g4);
      } else {
        const float b = s[BM + wn * TN];           // one scale per 128 columns
#pragma unroll
        for (int i = 0; i < FM; ++i) sa[i] *= b;
      }
    };
    auto product = [&](int i, int j) {
      if constexpr (WIDE) part[j] = mfma128_wide(bw[j], aw);
      else part[j] = mfma128<FMTA>(bf[j], af[i & 1]);
    };
    // acc of block (i, j) += its scaled product
    auto add = [&](int i, int j) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[i][j][e] += sa[i] * (BROW ? part[j][e] * sb[BROW ? j : 0][e] : part[j][e]);
    };

    issue(0, 0);
    issue(1, 1);
    wait_vmcnt<AL + BL + 1>();
    block_barrier();
    read_scales(0);
#pragma unroll
    for (int j = 0; j < FN; ++j) read_frag(smem + b_base + j * 2048, bf[j]);
    read_frag(smem + a_base, af[0]);
    for (int t = 0; t < nk; ++t) {
      const char* cur = smem + (t & 1) * STAGE;
      const char* nxt = smem + ((t + 1) & 1) * STAGE;
      if constexpr (WIDE)
#pragma unroll
        for (int j = 0; j < FN; ++j) widen<kFmtE4M3>(bf[j], bw[j]);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if constexpr (WIDE) widen<FMTA>(af[i & 1], aw);
        if (i + 1 < FM) {
          read_frag(cur + a_base + (i + 1) * 2048, af[(i + 1) & 1]);
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            if (i > 0) add(i - 1, j);
            product(i, j);
          }
        } else {
          // every fragment of k-tile t is in registers: refill its stage, and
          // read the first fragments of k-tile t + 1 beside the last MFMAs
          wait_vmcnt<0>();
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          block_barrier();
          issue(t & 1, t + 2);
          read_frag(nxt + a_base, af[(i + 1) & 1]);
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            add(i - 1, j);
            product(i, j);
            read_frag(nxt + b_base + j * 2048, bf[j]);
          }
#pragma unroll
          for (int j = 0; j < FN; ++j) add(i, j);
          read_scales((t + 1) & 1);
        }
      }
      static_assert(FM % 2 == 0, "two sets of A fragments alternate by row block");
    }
    wait_vmcnt<0>();
  };
  if (fast) body(BoolTag<true>{});
  else body(BoolTag<false>{});

  // ---- epilogue: acc[i][j][e] = C[m0 + wm*TM + 16i + i16][n0 + wn*TN + 16j + 4*g4 + e]
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int row = m0 + wm * TM + 16 * i + i16;
    if (row >= p.m) continue;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int col = n0 + wn * TN + 16 * j + 4 * g4;
      if (col >= p.n) continue;
      if (p.splits > 1) {
        float* d = p.partials + ((int64_t)split * p.m + row) * p.n + col;
        if (col + 3 < p.n && (p.n % 4) == 0) {
          *reinterpret_cast<f32x4_t*>(d) = acc[i][j];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col + e < p.n) d[e] = acc[i][j][e];
        }
      } else {
        store4(p, row, col, acc[i][j]);
      }
    }
  }
}

// Few rows: ROWS x COLS outputs per workgroup, over all of k or one of
// p.splits ranges of it.  The waves take the k-tiles round robin, each through
// its own LDS ring; a slot holds ROWS + COLS rows of 128 bytes and their
// scales (word l: row l, then column l - ROWS).
template <int FMTA, int ROWS, int COLS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(WAVES / 4, WAVES / 4)))
void scaled_skinny_kernel(ScaledProblem p) {
  constexpr int AL = ROWS / 8, BL = COLS / 8, LOADS = AL + BL + 1;
  constexpr int SLOT = (ROWS + COLS) * 128 + 256;
  constexpr int FIT = 160 * 1024 / WAVES / SLOT, SLOTS = FIT < 6 ? FIT : 6;
  constexpr int WAVE_LDS = SLOTS * SLOT;
  constexpr int FM = ROWS / 16, FN = COLS / 16;
  static_assert(ROWS + COLS <= 64, "one scale per lane");
  static_assert(SLOTS >= 2 && SLOTS * LOADS < 64, "ring");
  __shared__ __attribute__((aligned(1024))) char smem[WAVES * WAVE_LDS];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int RB = (p.m + ROWS - 1) / ROWS, CB = (p.n + COLS - 1) / COLS;
  int tile, split;
  {
    // XCD x (workgroup id mod 8) takes a contiguous range, row blocks
    // fastest: the row blocks of one column block share its L2
    const int T = RB * CB * p.splits, wg = blockIdx.x;
    const int xcd = wg & 7, local = wg >> 3, per = T >> 3, rem = T & 7;
    const int u = xcd * per + (xcd < rem ? xcd : rem) + local;
    tile = u % (RB * CB);
    split = u / (RB * CB);
  }
  const int row0 = (tile % RB) * ROWS, n0 = (tile / RB) * COLS;
  const int t0 = split * p.kb_per_split, t1 = min(p.kb, t0 + p.kb_per_split);
  const int rpg = p.rows_per_group;
  const char* zero = reinterpret_cast<const char*>(g_zero_chunk);

  const char* a_src[AL];
  const char* b_src[BL];
  uint32_t ok_bits = 0;
#pragma unroll
  for (int q = 0; q < AL; ++q) {
    const int r = 8 * q + (lane >> 3), gr = row0 + r;
    a_src[q] = zero;
    if (gr < p.m) {
      const int g = gr / rpg, t = gr - g * rpg;
      a_src[q] = static_cast<const char*>(p.a_group[g]) + (int64_t)t * p.a_ld + ((lane & 7) ^ swz_k16(r)) * 16;
      ok_bits |= 1u << q;
    }
  }
#pragma unroll
  for (int q = 0; q < BL; ++q) {
    const int r = 8 * q + (lane >> 3), gn = n0 + r;
    b_src[q] = zero;
    if (gn < p.n) {
      b_src[q] = static_cast<const char*>(p.b) + (int64_t)gn * p.ldb + ((lane & 7) ^ swz_k16(r)) * 16;
      ok_bits |= 1u << (AL + q);
    }
  }
  const char* s_src = zero;
  int64_t s_step = 0;
  if (lane < ROWS) {
    const int gr = row0 + lane;
    if (gr < p.m) {
      const int g = gr / rpg;
      s_src = reinterpret_cast<const char*>(p.a_scale[g] + (gr - g * rpg));
      s_step = (int64_t)rpg * 4;
    }
  } else if (lane < ROWS + COLS) {
    const int gn = n0 + lane - ROWS;
    if (gn < p.n) {
      s_src = reinterpret_cast<const char*>(p.b_scale + gn / p.b_block_rows);
      s_step = (int64_t)p.nb * 4;
    }
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
      const bool ok = ((ok_bits >> q) & 1) && t * 128 + ((lane & 7) ^ swz_k16(r)) * 16 < p.k16;
      load_lds16_at(ok ? (q < AL ? a_src[q < AL ? q : 0] : b_src[q < AL ? 0 : q - AL]) + off : zero, dst + q * 1024);
    }
    load_lds4_at(s_src + (int64_t)t * s_step, dst + (ROWS + COLS) * 128);
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
  for (int e4 = tid; e4 < ROWS * COLS / 4; e4 += 64 * WAVES) {
    const int r = e4 / (COLS / 4), c = (e4 % (COLS / 4)) * 4;
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(smem) + r * RLD + c);
#pragma unroll
    for (int w = 1; w < WAVES; ++w)
      v += *reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(smem + w * WAVE_LDS) + r * RLD + c);
    const int row = row0 + r, col = n0 + c;
    if (row >= p.m || col >= p.n) continue;
    if (p.splits > 1) {
      float* d = p.partials + ((int64_t)split * p.m + row) * p.n + col;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < p.n) d[e] = v[e];
    } else {
      store4(p, row, col, v);
    }
  }
}

// Sum of the k ranges in order, four columns per thread.
__global__ __launch_bounds__(256) void scaled_reduce_kernel(ScaledProblem p) {
  const int n4 = (p.n + 3) / 4;
  const int64_t plane = (int64_t)p.m * p.n;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < (int64_t)p.m * n4; u += (int64_t)gridDim.x * 256) {
    const int row = (int)(u / n4), col = (int)(u % n4) * 4;
    const float* src = p.partials + (int64_t)row * p.n + col;
    f32x4_t v = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if ((p.n % 4) == 0) {
      v = *reinterpret_cast<const f32x4_t*>(src);
      for (int s = 1; s < p.splits; ++s) v += *reinterpret_cast<const f32x4_t*>(src + s * plane);
    } else {
      for (int s = 0; s < p.splits; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < p.n) v[e] += src[s * plane + e];
    }
    store4(p, row, col, v);
  }
}

template <int FMTA, bool BROW>
hipError_t launch_tile(const ScaledProblem& p, int tile, hipStream_t stream) {
  const int64_t grid = (int64_t)p.order.num_rb * p.order.num_cb * p.splits;
  if (tile == kScaled256)
    hipLaunchKernelGGL((scaled_gemm_kernel<FMTA, BROW, false, 256, 256, 2, 4>), dim3((unsigned)grid), dim3(512), 0, stream, p);
  else if (p.wide)
    hipLaunchKernelGGL((scaled_gemm_kernel<FMTA, BROW, true, 128, 128, 2, 2>), dim3((unsigned)grid), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((scaled_gemm_kernel<FMTA, BROW, false, 128, 128, 2, 2>), dim3((unsigned)grid), dim3(256), 0, stream, p);
  return hipGetLastError();
}

template <int FMTA>
hipError_t launch_skinny(const ScaledProblem& p, int tile, hipStream_t stream) {
  const int rows = scaled_tile_rows(tile), cols = scaled_tile_cols(tile);
  const int64_t grid = (int64_t)((p.m + rows - 1) / rows) * ((p.n + cols - 1) / cols) * p.splits;
  if (tile == kScaledSkinny16)
    hipLaunchKernelGGL((scaled_skinny_kernel<FMTA, 16, 32, 4>), dim3((unsigned)grid), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((scaled_skinny_kernel<FMTA, 32, 32, 4>), dim3((unsigned)grid), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_scaled(const ScaledProblem& p, int tile, hipStream_t stream) {
  const int rows = scaled_tile_rows(tile), cols = scaled_tile_cols(tile);
  const int64_t grid = (int64_t)((p.m + rows - 1) / rows) * ((p.n + cols - 1) / cols) * p.splits;
  if (rows == 0 || grid < 1 || grid >= (int64_t(1) << 23) || p.splits < 1 ||
      (p.splits > 1 && !p.partials) || (int64_t)p.splits * p.kb_per_split < p.kb ||
      (int64_t)(p.splits - 1) * p.kb_per_split >= p.kb || p.k16 % 16 != 0 || p.kb != (p.k16 + 127) / 128 ||
      p.num_groups < 1 || p.num_groups > kMaxGroups || (int64_t)p.num_groups * p.rows_per_group != p.m)
    return hipErrorInvalidValue;
  hipError_t err;
  const bool e5m2 = p.a_format == kFmtE5M2;
  if (tile == kScaledSkinny16 || tile == kScaledSkinny32)
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
