// bf16 / fp16 MFMA GEMM for the all-gather matmul on gfx950 (CDNA4).
//
// Computes, for the logical rows described by a RowMap (shard buffers, a ring
// slot or the fully gathered operand),
//     C[row, :] = A[row, :] @ B          (B stored k x n)
//     C[row, :] = A[row, :] @ B^T        (rhs_transpose: B stored n x k)
// with fp32 accumulation and a round-to-nearest-even cast to the input dtype
// (tpu-inference "all_gather_matmul.py", `_do_mxu`: jnp.dot / dot_general with
// preferred_element_type=float32 accumulated over bk slices, cast with
// astype(x.dtype) on the last slice; Triton-distributed-Ascend
// "AllGather-GEMM" kernel listing: fp32 accumulator over K blocks, cast on
// store).
//
// Design (MI355X-native, not a translation of either page):
//  * 4 waves of 64 lanes per workgroup, 2 x 2 over the output tile.
//  * Two main-loop forms:
//      - the part ring (gemm_m16_kernel, and gemm_mfma_kernel with
//        kLoopParts): 64-deep k-tiles, LDS split into 5 slots that each hold
//        one operand of one k-tile, so 2.5 k-tiles are resident and every
//        load fetches whole 128-byte lines; one barrier per k-tile;
//      - the stage ring (gemm_mfma_kernel, kLoopStages): 32-deep k-tiles in
//        3-8 whole stages, for short k.
//  * MFMAs: v_mfma_f32_16x16x32 (gemm_m16_kernel, the default for k >= 256;
//    it holds a higher clock than the 32x32x16 form for the same work on this
//    power-limited chip) or v_mfma_f32_32x32x16 (gemm_mfma_kernel), always
//    with the B fragment as the first operand.
//  * Every operand tile goes global -> LDS directly (lane i of a wave writes
//    bytes [16i, 16i+16) of a 1 KiB LDS block, so the LDS swizzle is chosen
//    by which global chunk each lane fetches); each wave waits only for the
//    k-tile it reads next (partial vmcnt).  gemm_m16_kernel loads interior
//    tiles whose rows lie in one shard through buffer descriptors
//    (buffer_load_dwordx4 ... lds: scalar base and k offset, fixed 32-bit
//    lane offsets); other tiles use global_load_lds_dwordx4 with 64-bit lane
//    addresses.
//  * k-contiguous tiles (A, and B when stored n x k) and n-contiguous B
//    tiles (B stored k x n, transposed on the way out by ds_read_b64_tr_b16)
//    use XOR swizzles measured free of LDS bank conflicts for each form's
//    fragment reads.
//  * Rows past m, columns past n and k past the end are fed from a zero
//    block, so ragged tails need no masking inside the main loop; interior
//    tiles take an unmasked loop.
//  * Tile order: XCD-aware remap of the workgroup id, grouped row blocks for
//    L2 reuse, then the plan's row-block visit order (ring order from the
//    local shard, or natural order).
//  * Epilogue: round-to-nearest-even cast, C staged through LDS and stored
//    as whole rows with 16-byte lanes (interior tiles), or fp32 partial sums
//    for split-K followed by a fixed-order reduction launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "agmm_kernels.h"
#include "gemm_device.h"

namespace agmm {

namespace {

template <int BM, int BN, int BK, int DT, bool BT, bool SPLIT, int NST, int WAVES, int OCC, int LOOP>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
void gemm_mfma_kernel(GemmProblem p) {
  using T = GemmTile<BM, BN, BK, DT, BT, NST, WAVES, LOOP>;
  constexpr int kBK = BK;
  constexpr int kStages = T::kStages;
  __shared__ __attribute__((aligned(1024))) char smem[T::LDS_BYTES];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // wave-uniform: LDS block addresses stay scalar
  const int wm = wave / T::WN, wn = wave % T::WN;

  const int M = p.m, N = p.n, K = p.k;
  const int ntiles = p.order.num_rb * p.order.num_cb;
  int wg = blockIdx.x;
  int split = 0;
  if constexpr (SPLIT) {
    split = wg / ntiles;
    wg -= split * ntiles;
  }
  int rb, cb;
  tile_coords(p.order, wg, ntiles, rb, cb);
  const int m0 = rb * BM, n0 = cb * BN;

  int k_begin = 0, k_end = K;
  if constexpr (SPLIT) {
    k_begin = split * p.k_per_split;
    k_end = min(K, k_begin + p.k_per_split);
  }
  const int nk = (k_end - k_begin + kBK - 1) / kBK;

  const char* zero = reinterpret_cast<const char*>(g_zero_chunk);

  // ---- per-lane global sources of the direct-to-LDS loads -------------------
  // k-contiguous tiles: instruction j of this wave fills LDS rows
  // (wave*IPW + j)*RPI + lane/CPR, position lane%CPR, which holds chunk
  // (lane%CPR) ^ swz_k(row).
  const char* a_src[T::A_IPW];
  int a_kc[T::A_IPW];
  uint32_t a_ok = 0;
#pragma unroll
  for (int j = 0; j < T::A_IPW; ++j) {
    const int r = (wave * T::A_IPW + j) * T::RPI + lane / T::CPR;
    const int c = (lane % T::CPR) ^ swz_k<BK>(r);
    a_kc[j] = c * 8;
    const int gi = m0 + r;
    a_src[j] = zero;
    if (gi < M) {
      const int g = gi / p.rows.rows_per_group;
      const int t = gi - g * p.rows.rows_per_group;
      a_src[j] = static_cast<const char*>(p.rows.a_group[g]) + ((int64_t)t * p.rows.a_ld + c * 8) * 2;
      a_ok |= 1u << j;
    }
  }
  const char* b_src[T::B_IPW];
  int b_kc[T::B_IPW];   // BT: element offset in k; !BT: k-row inside the tile
  uint32_t b_ok = 0;
#pragma unroll
  for (int j = 0; j < T::B_IPW; ++j) {
    b_src[j] = zero;
    if constexpr (BT) {
      const int r = (wave * T::B_IPW + j) * T::RPI + lane / T::CPR;
      const int c = (lane % T::CPR) ^ swz_k<BK>(r);
      b_kc[j] = c * 8;
      const int gn = n0 + r;
      if (gn < N) {
        b_src[j] = static_cast<const char*>(p.b) + ((int64_t)gn * p.ldb + c * 8) * 2;
        b_ok |= 1u << j;
      }
    } else {
      // n-contiguous k-rows of BN*2 bytes: byte (wave*IPW + j)*1024 + lane*16
      const int byte = (wave * T::B_IPW + j) * 1024 + lane * 16;
      const int kr = byte / T::B_ROW;
      const int pos = (byte % T::B_ROW) >> 4;
      const int c = pos ^ swz_n(kr);
      b_kc[j] = kr;
      const int gn = n0 + c * 8;
      if (gn < N) {
        b_src[j] = static_cast<const char*>(p.b) + ((int64_t)kr * p.ldb + gn) * 2;
        b_ok |= 1u << j;
      }
    }
  }

  // Branch-free issue of one k-tile: lanes whose row/column is out of range,
  // or whose chunk lies past k_end (ragged k, or a k-tile past the end that
  // the uniform pipeline still issues), fetch the zero block instead.
  auto issue_a = [&](char* sa, int k0) {
    const int64_t a_step = (int64_t)k0 * 2;
#pragma unroll
    for (int j = 0; j < T::A_IPW; ++j) {
      const bool ok = ((a_ok >> j) & 1) && (k0 + a_kc[j] < k_end);
      load_lds16(ok ? a_src[j] + a_step : zero, sa + (wave * T::A_IPW + j) * 1024);
    }
  };
  auto issue_b = [&](char* sb, int k0) {
    const int64_t b_step = BT ? (int64_t)k0 * 2 : (int64_t)k0 * p.ldb * 2;
#pragma unroll
    for (int j = 0; j < T::B_IPW; ++j) {
      const bool ok = ((b_ok >> j) & 1) && (k0 + b_kc[j] < k_end);
      load_lds16(ok ? b_src[j] + b_step : zero, sb + (wave * T::B_IPW + j) * 1024);
    }
  };
  auto issue = [&](int stage, int k0) {
    char* sa = smem + stage * T::STAGE_BYTES;
    issue_a(sa, k0);
    issue_b(sa + T::A_BYTES, k0);
  };

  // ---- LDS fragment read offsets -------------------------------------------
  const int hi = lane >> 5, l32 = lane & 31;
  int a_off[T::FM], a_x[T::FM];
#pragma unroll
  for (int f = 0; f < T::FM; ++f) {
    const int r = wm * T::TM + f * 32 + l32;
    a_off[f] = r * T::KROW;
    a_x[f] = hi ^ swz_k<BK>(r);
  }
  // BT: k-contiguous rows like A.  !BT: ds_read_b64_tr_b16 source lanes.
  // Lane i of 16-lane group G reads k-row 16s + 8*(G/2) + 4*half + i/4 at
  // columns nb + 16*(G%2) + 4*(i%4) .. +3; the instruction hands lane
  // 16G + j element e of the 16x4 block read by lanes 4e + j/4, i.e.
  // B[16s + 8*(G/2) + 4*half + e][nb + 16*(G%2) + j].
  int b_off[T::FN], b_x[T::FN];
  if constexpr (BT) {
#pragma unroll
    for (int f = 0; f < T::FN; ++f) {
      const int r = wn * T::TN + f * 32 + l32;
      b_off[f] = r * T::KROW;
      b_x[f] = hi ^ swz_k<BK>(r);
    }
  }
  const int tr_g = lane >> 4, tr_i = lane & 15;
  const int tr_krow = 8 * (tr_g >> 1) + (tr_i >> 2);        // + 16s + 4*half
  const int tr_swz = swz_n(tr_krow);                        // k-row % 4 is the same for every s/half
  int tr_n[T::FN];
#pragma unroll
  for (int f = 0; f < T::FN; ++f) tr_n[f] = wn * T::TN + f * 32 + 16 * (tr_g & 1) + 4 * (tr_i & 3);

  f32x16_t acc[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; ++i)
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  // Fragments of k16 substep s from the A operand at `sa` and the B operand at `sb`.
  auto read_frags2 = [&](const char* sa, const char* sb, int s, u32x4_t* af, u32x4_t* bfr) {
    // in the order mfma_block consumes them: B0, A0 .. A(FM-1), B1 .. B(FN-1)
    auto read_b = [&](int f) {
      if constexpr (BT) {
        bfr[f] = *reinterpret_cast<const u32x4_t*>(sb + b_off[f] + (((2 * s) ^ b_x[f]) << 4));
      } else {
        const int n = tr_n[f];
        const int pos = (n >> 3) ^ tr_swz;
        const int within = (n & 7) * 2;
        const char* p0 = sb + (16 * s + tr_krow) * T::B_ROW + (pos << 4) + within;
        const u32x2_t lo = read_tr(p0);
        const u32x2_t hi2 = read_tr(p0 + 4 * T::B_ROW);
        bfr[f] = u32x4_t{lo[0], lo[1], hi2[0], hi2[1]};
      }
    };
    read_b(0);
#pragma unroll
    for (int f = 0; f < T::FM; ++f)
      af[f] = *reinterpret_cast<const u32x4_t*>(sa + a_off[f] + (((2 * s) ^ a_x[f]) << 4));
#pragma unroll
    for (int f = 1; f < T::FN; ++f) read_b(f);
  };
  auto read_frags = [&](const char* stage, int s, u32x4_t* af, u32x4_t* bfr) {
    read_frags2(stage, stage + T::A_BYTES, s, af, bfr);
  };
  // B fragment outermost: the j-th group of MFMAs needs only B0..Bj and the
  // A fragments, which arrive in that order.
  auto mfma_block = [&](const u32x4_t* af, const u32x4_t* bfr) {
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int i = 0; i < T::FM; ++i) acc[i][j] = mfma32<DT>(bfr[j], af[i], acc[i][j]);
  };
  constexpr int kMfmaPerSub = T::FM * T::FN;
  constexpr int kReadsPerSub = T::FM + (BT ? T::FN : 2 * T::FN);

  // ---- main loop, part ring ----------------------------------------------------
  // Slot q % 5 receives part q: A of k-tile q/2 for even q, B for odd q.
  // Parts 0-3 are issued up front.  During k-tile t:
  //   substeps 0 .. SUB-2: the loads of part 2t+4 (A of t+2) are spread over
  //     the MFMAs, into the slot of B of t-1 (free since the previous sync);
  //   substep SUB-1: each wave waits for its own loads of parts 2t+2, 2t+3
  //     (k-tile t+1; part 2t+4 may still be in flight) and for its LDS reads
  //     of k-tile t; one barrier; then part 2t+5 (B of t+2) goes into the
  //     slot of A of t, and the fragments of k-tile t+1 are read while the
  //     last MFMAs of k-tile t run.
  // Spreading the loads keeps the L1/L2 request stream even instead of one
  // burst per k-tile from every CU at once.  Past the end the parts fetch
  // zeros into slots nobody reads again, so the vmcnt arithmetic is the same
  // in every iteration.
  if constexpr (LOOP == kLoopParts) {
    constexpr int L = T::A_IPW;                       // load instructions per A part per wave
    constexpr int LB = T::B_IPW;                      // ... per B part
    constexpr int PB = T::PART_BYTES;
    constexpr int SPREAD = T::SUB - 1;                // substeps that carry A loads
    // Interior tiles (every row and column in range, whole k-tiles) load
    // without per-lane masks: the source is the lane's row pointer plus a
    // uniform k offset, and k-tiles past the end re-read the last k-tile
    // (valid memory; those slots are never read).  Edge tiles redirect
    // out-of-range chunks to the zero block.
    const bool interior = (m0 + BM <= M) && (n0 + BN <= N) && ((k_end - k_begin) % kBK == 0) && nk > 0;
    auto ring = [&](auto tag) {
      constexpr bool FAST = decltype(tag)::value;
      auto a_addr = [&](int j, int t) -> const char* {
        if constexpr (FAST) {
          const int kk = k_begin + (t < nk ? t : nk - 1) * kBK;
          return a_src[j] + (int64_t)kk * 2;
        } else {
          const int kk = k_begin + t * kBK;
          const bool ok = ((a_ok >> j) & 1) && (kk + a_kc[j] < k_end);
          return ok ? a_src[j] + (int64_t)kk * 2 : zero;
        }
      };
      auto b_addr = [&](int j, int t) -> const char* {
        if constexpr (FAST) {
          const int kk = k_begin + (t < nk ? t : nk - 1) * kBK;
          return b_src[j] + (BT ? (int64_t)kk * 2 : (int64_t)kk * p.ldb * 2);
        } else {
          const int kk = k_begin + t * kBK;
          const bool ok = ((b_ok >> j) & 1) && (kk + b_kc[j] < k_end);
          return ok ? b_src[j] + (BT ? (int64_t)kk * 2 : (int64_t)kk * p.ldb * 2) : zero;
        }
      };
      const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char_t*)smem;
      const uint32_t lds_a = lds0 + wave * (T::A_IPW * 1024);
      const uint32_t lds_b = lds0 + wave * (T::B_IPW * 1024);
      auto put_a = [&](int slot, int t, int j0, int j1) {
#pragma unroll
        for (int j = j0; j < j1; ++j) load_lds16_at(a_addr(j, t), lds_a + slot * PB + j * 1024);
      };
      auto put_b = [&](int slot, int t) {
#pragma unroll
        for (int j = 0; j < T::B_IPW; ++j) load_lds16_at(b_addr(j, t), lds_b + slot * PB + j * 1024);
      };
      u32x4_t fa[2][T::FM], fb[2][T::FN];
      put_a(0, 0, 0, L);
      put_b(1, 0);
      put_a(2, 1, 0, L);
      put_b(3, 1);
      wait_vmcnt<L + LB>();
      block_barrier();
      read_frags2(smem, smem + PB, 0, fa[0], fb[0]);
      int sa_slot = 0, sb_slot = 1;   // slots of A and B of k-tile it
      for (int it = 0; it < nk; ++it) {
        const char* sa = smem + sa_slot * PB;
        const char* sb = smem + sb_slot * PB;
        const int a_new = sb_slot + 3 >= 5 ? sb_slot - 2 : sb_slot + 3;   // slot of B of it-1
        const int na = sa_slot + 2 >= 5 ? sa_slot - 3 : sa_slot + 2;
        const int nb = sb_slot + 2 >= 5 ? sb_slot - 3 : sb_slot + 2;
#pragma unroll
        for (int s = 0; s < T::SUB; ++s) {
          int nv;
          if (s == T::SUB - 1) {
            wait_vmcnt<L>();
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            block_barrier();
            read_frags2(smem + na * PB, smem + nb * PB, 0, fa[0], fb[0]);
            put_b(sa_slot, it + 2);
            nv = LB;
          } else {
            const int j0 = s * L / SPREAD, j1 = (s + 1) * L / SPREAD;
            read_frags2(sa, sb, s + 1, fa[(s + 1) & 1], fb[(s + 1) & 1]);
            put_a(a_new, it + 2, j0, j1);
            nv = j1 - j0;
          }
          mfma_block(fa[s & 1], fb[s & 1]);
          // interleave: MFMA, LDS read, ... (all reads first: the next
          // substep waits on them), then MFMA, global->LDS load(s), ...
          constexpr int nr = kReadsPerSub < kMfmaPerSub ? kReadsPerSub : kMfmaPerSub;
          const int left = kMfmaPerSub - nr;
#pragma unroll
          for (int q = 0; q < nr; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          }
#pragma unroll
          for (int q = 0; q < left; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
            for (int r = q * nv / left; r < (q + 1) * nv / left; ++r)
              __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
          }
        }
        sa_slot = na;
        sb_slot = nb;
      }
    };
    if (interior) ring(BoolTag<true>{});
    else ring(BoolTag<false>{});
  } else {
  // ---- main loop ---------------------------------------------------------------
  // Fragment registers alternate between two sets: the LDS reads of substep
  // s+1 are in flight while the MFMAs of substep s run.  Once per k-tile the
  // workgroup synchronises ("sync"): each wave waits for its own loads of
  // the next k-tile (vmcnt), then a barrier makes that tile complete in LDS
  // and guarantees every wave is done with the stage the next issue reuses;
  // right after it the loads of a further k-tile are issued.
  //   MID_SYNC (>= 3 stages): sync in the middle of tile `it`, issue tile
  //     it+NST-1 into the stage of tile it-1; the reads of tile it+1 start
  //     during the last substep of tile it.
  //   2 stages: sync at the end of tile `it`, issue tile it+2 into the stage
  //     of tile it.
  // Every iteration issues exactly one k-tile of loads (past the end they
  // fetch zeros into a stage nobody reads again), so the vmcnt arithmetic is
  // the same in every iteration and the loop body has no branches.
  u32x4_t fa[2][T::FM], fb[2][T::FN];
  constexpr int kPre = T::MID_SYNC ? kStages - 1 : kStages;   // tiles issued up front
#pragma unroll
  for (int t = 0; t < kPre; ++t) issue(t, k_begin + t * kBK);
  wait_vmcnt<(kPre - 1) * T::LOADS>();
  block_barrier();
  read_frags(smem, 0, fa[0], fb[0]);
  int st_cur = 0;                              // stage of tile it
  int st_new = T::MID_SYNC ? kStages - 1 : 0;  // stage the next issue fills
  int t_new = kPre;                            // k-tile the next issue loads
  for (int it = 0; it < nk; ++it) {
    const char* cur = smem + st_cur * T::STAGE_BYTES;
    const int st_next = (st_cur + 1 == kStages) ? 0 : st_cur + 1;
#pragma unroll
    for (int s = 0; s < T::SUB; ++s) {
      if (s == T::SYNC_SUB) {
        wait_vmcnt<(kStages - 3 > 0 ? kStages - 3 : 0) * T::LOADS>();
        block_barrier();
        issue(st_new, k_begin + t_new * kBK);
      }
      if (s + 1 < T::SUB) read_frags(cur, s + 1, fa[(s + 1) & 1], fb[(s + 1) & 1]);
      else if (T::MID_SYNC) read_frags(smem + st_next * T::STAGE_BYTES, 0, fa[0], fb[0]);
      mfma_block(fa[s & 1], fb[s & 1]);
      // interleave: MFMA, global->LDS load (right after a sync), ...,
      // then MFMA, LDS read, MFMA, LDS read, ..., then the remaining MFMAs
      const int nv = (s == T::SYNC_SUB) ? (T::LOADS < kMfmaPerSub ? T::LOADS : kMfmaPerSub) : 0;
      const int left = kMfmaPerSub - nv;
      const int nr = kReadsPerSub < left ? kReadsPerSub : left;
#pragma unroll
      for (int q = 0; q < nv; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      }
#pragma unroll
      for (int q = 0; q < nr; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
#pragma unroll
      for (int q = 0; q < left - nr; ++q) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    if constexpr (!T::MID_SYNC) {
      wait_vmcnt<0>();
      block_barrier();
      issue(st_new, k_begin + t_new * kBK);
      read_frags(smem + st_next * T::STAGE_BYTES, 0, fa[0], fb[0]);
    }
    st_cur = st_next;
    st_new = (st_new + 1 == kStages) ? 0 : st_new + 1;
    ++t_new;
  }
  }
  // No LDS-bound load may still be in flight when the workgroup retires.
  wait_vmcnt<0>();

  // ---- epilogue --------------------------------------------------------------
  // acc[i][j][4q + e] holds C[m0 + wm*TM + i*32 + l32][n0 + wn*TN + j*32 + 8q + 4hi + e].
  //
  // Interior tiles with 16-byte aligned C rows go through LDS: every wave
  // writes its converted sub-tile into a [BM][BN] staging tile (16-byte
  // chunk c of row r at position c ^ (r % chunks-per-row), which spreads
  // the 32 rows one ds_write touches over the banks), then the workgroup
  // writes C row by row, 16 bytes per lane and whole rows per group of
  // lanes, instead of 16-byte pieces of 32 different rows per store.
  constexpr int kRowB = BN * 2;            // bytes of a staged C row
  constexpr int kChunks = kRowB / 16;      // 16-byte chunks per row
  static_assert(T::LDS_BYTES >= BM * kRowB, "LDS too small to stage the C tile");
  static_assert((kChunks & (kChunks - 1)) == 0 && T::THREADS % kChunks == 0, "staging layout");
  bool staged = false;
  if constexpr (!SPLIT) {
    staged = (m0 + BM <= M) && (n0 + BN <= N) && (p.ldc % 8) == 0 &&
             ((reinterpret_cast<uintptr_t>(p.c) & 15) == 0);
  }
  if (staged) {
    block_barrier();   // every wave's fragment reads and LDS-bound loads are done
#pragma unroll
    for (int i = 0; i < T::FM; ++i) {
      const int r = wm * T::TM + i * 32 + l32;
      char* row = smem + r * kRowB;
#pragma unroll
      for (int j = 0; j < T::FN; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = wn * T::TN + j * 32 + 8 * q;          // first column of the chunk
          const int pos = (c >> 3) ^ (r & (kChunks - 1));
          const f32x16_t& a = acc[i][j];
          u32x2_t v;
          v[0] = pack2<DT>(a[4 * q + 0], a[4 * q + 1]);
          v[1] = pack2<DT>(a[4 * q + 2], a[4 * q + 3]);
          *reinterpret_cast<u32x2_t*>(row + pos * 16 + hi * 8) = v;
        }
      }
    }
    block_barrier();
    constexpr int kRowsPerPass = T::THREADS / kChunks;
    const int ch = tid % kChunks;
    int r = tid / kChunks;
    int gi = m0 + r;
    int g = gi / p.rows.rows_per_group;
    int t = gi - g * p.rows.rows_per_group;
    uint16_t* cbase = static_cast<uint16_t*>(p.c) + n0 + ch * 8;
#pragma unroll 4
    for (; r < BM; r += kRowsPerPass) {
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(smem + r * kRowB + ((ch ^ (r & (kChunks - 1))) << 4));
      const int64_t crow = (int64_t)g * p.rows.c_group_rows + p.rows.c_row_off + t;
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(cbase + crow * p.ldc));   // C is not re-read: keep L2 for A and B
      t += kRowsPerPass;
      while (t >= p.rows.rows_per_group) {
        t -= p.rows.rows_per_group;
        ++g;
      }
    }
  } else if constexpr (!SPLIT) {
    const bool vec_ok = (N % 4) == 0 && (p.ldc % 4) == 0;
#pragma unroll
    for (int i = 0; i < T::FM; ++i) {
      const int gi = m0 + wm * T::TM + i * 32 + l32;
      if (gi >= M) continue;
      const int g = gi / p.rows.rows_per_group;
      const int t = gi - g * p.rows.rows_per_group;
      const int64_t crow = (int64_t)g * p.rows.c_group_rows + p.rows.c_row_off + t;
      uint16_t* cp = static_cast<uint16_t*>(p.c) + crow * p.ldc;
#pragma unroll
      for (int j = 0; j < T::FN; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int gn = n0 + wn * T::TN + j * 32 + 8 * q + 4 * hi;
          const f32x16_t& a = acc[i][j];
          if (vec_ok && gn + 3 < N) {
            u32x2_t v;
            v[0] = pack2<DT>(a[4 * q + 0], a[4 * q + 1]);
            v[1] = pack2<DT>(a[4 * q + 2], a[4 * q + 3]);
            *reinterpret_cast<u32x2_t*>(cp + gn) = v;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (gn + e < N) cp[gn + e] = cvt1<DT>(a[4 * q + e]);
          }
        }
      }
    }
  } else {
    // Split-K: this workgroup's fp32 partial tile goes to partials[split];
    // splitk_reduce_kernel sums the splits afterwards.
    float* part = p.partials + (int64_t)split * M * N;
    const bool vec_ok = (N % 4) == 0;
#pragma unroll
    for (int i = 0; i < T::FM; ++i) {
      const int gi = m0 + wm * T::TM + i * 32 + l32;
      if (gi >= M) continue;
      float* prow = part + (int64_t)gi * N;
#pragma unroll
      for (int j = 0; j < T::FN; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int gn = n0 + wn * T::TN + j * 32 + 8 * q + 4 * hi;
          const f32x16_t& a = acc[i][j];
          if (vec_ok && gn + 3 < N) {
            *reinterpret_cast<f32x4_t*>(prow + gn) =
                f32x4_t{a[4 * q + 0], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (gn + e < N) prow[gn + e] = a[4 * q + e];
          }
        }
      }
    }
  }
}

// Part-ring GEMM on v_mfma_f32_16x16x32_{bf16,f16}: the tiles, LDS layouts,
// part ring, synchronisation, load paths and epilogue of the part-ring form
// of gemm_mfma_kernel, with each wave's sub-tile computed as 16x16 blocks and
// a 64-deep k-tile as two k32 steps.  With random bf16 operands the chip is
// power-limited, and this instruction holds a higher clock than the 32x32x16
// one for the same work (measured raw MFMA throughput on MI355X: 1.88 against
// 1.65 PFLOP/s, 1.97 against 1.64 GHz).
// Fragments (lane l, g = l / 16, i = l % 16), B is the first operand:
//   A (second operand): A[m = i][k = 8g .. 8g+7] of a 16-row block
//   B (first operand):  B[k = 8g .. 8g+7][n = i] of a 16-column block
//   result:             C[m = i][n = 4g .. 4g+3] of the 16x16 block
template <int BM, int BN, int BK, int DT, bool BT, bool SPLIT, int WAVES, int OCC>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
void gemm_m16_kernel(GemmProblem p) {
  using T = GemmTile<BM, BN, BK, DT, BT, 5, WAVES, kLoopParts>;
  constexpr int kBK = BK;
  constexpr int FM = T::TM / 16, FN = T::TN / 16;   // 16x16 blocks per wave
  constexpr int STEPS = BK / 32;                    // k32 steps per k-tile
  static_assert(BK == 64, "two k32 steps per k-tile");
  __shared__ __attribute__((aligned(1024))) char smem[T::LDS_BYTES];

#include "gemm_m16_loop.inc"

  // ---- epilogue: acc[i][j][e] = C[m0 + wm*TM + 16i + i16][n0 + wn*TN + 16j + 4g4 + e]
  const int hi = g4 & 1;   // which half of a 16-byte (8-column) chunk
  constexpr int kRowB = BN * 2;
  constexpr int kChunks = kRowB / 16;
  // staged C rows: chunk c of row r at c ^ (r mod kSwz), kSwz the largest
  // power of two dividing the chunks per row (so positions stay in the row)
  constexpr int kSwz = kChunks & -kChunks;
  static_assert(T::LDS_BYTES >= BM * kRowB, "LDS too small to stage the C tile");
  bool staged = false;
  if constexpr (!SPLIT) {
    staged = (m0 + BM <= M) && (n0 + BN <= N) && (p.ldc % 8) == 0 &&
             ((reinterpret_cast<uintptr_t>(p.c) & 15) == 0);
  }
  if (staged) {
    block_barrier();
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = wm * T::TM + i * 16 + i16;
      char* row = smem + r * kRowB;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int c = wn * T::TN + j * 16 + 4 * g4;
        const int pos = (c >> 3) ^ (r & (kSwz - 1));
        u32x2_t v;
        v[0] = pack2<DT>(acc[i][j][0], acc[i][j][1]);
        v[1] = pack2<DT>(acc[i][j][2], acc[i][j][3]);
        *reinterpret_cast<u32x2_t*>(row + pos * 16 + hi * 8) = v;
      }
    }
    block_barrier();
    constexpr int kRowsPerPass = T::THREADS / kChunks;   // threads past whole rows stay idle
    const int ch = tid % kChunks;
    int r = tid < kRowsPerPass * kChunks ? tid / kChunks : BM;
    int gi = m0 + r;
    int g = gi / p.rows.rows_per_group;
    int t = gi - g * p.rows.rows_per_group;
    uint16_t* cbase = static_cast<uint16_t*>(p.c) + n0 + ch * 8;
#pragma unroll 4
    for (; r < BM; r += kRowsPerPass) {
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(smem + r * kRowB + ((ch ^ (r & (kSwz - 1))) << 4));
      const int64_t crow = (int64_t)g * p.rows.c_group_rows + p.rows.c_row_off + t;
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(cbase + crow * p.ldc));
      t += kRowsPerPass;
      while (t >= p.rows.rows_per_group) {
        t -= p.rows.rows_per_group;
        ++g;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int gi = m0 + wm * T::TM + i * 16 + i16;
      if (gi >= M) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int gn = n0 + wn * T::TN + j * 16 + 4 * g4;
        const f32x4_t& a = acc[i][j];
        if constexpr (SPLIT) {
          float* prow = p.partials + ((int64_t)split * M + gi) * N;
          if ((N % 4) == 0 && gn + 3 < N) {
            *reinterpret_cast<f32x4_t*>(prow + gn) = a;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (gn + e < N) prow[gn + e] = a[e];
          }
        } else {
          const int g = gi / p.rows.rows_per_group;
          const int t = gi - g * p.rows.rows_per_group;
          uint16_t* cp = static_cast<uint16_t*>(p.c) + ((int64_t)g * p.rows.c_group_rows + p.rows.c_row_off + t) * p.ldc;
          if ((N % 4) == 0 && (p.ldc % 4) == 0 && gn + 3 < N) {
            u32x2_t v;
            v[0] = pack2<DT>(a[0], a[1]);
            v[1] = pack2<DT>(a[2], a[3]);
            *reinterpret_cast<u32x2_t*>(cp + gn) = v;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (gn + e < N) cp[gn + e] = cvt1<DT>(a[e]);
          }
        }
      }
    }
  }
}

// Sum of the split-K partials in split order 0, 1, ..., S-1 (fixed, so the
// result does not depend on which workgroup finished first), cast to the
// output dtype, scattered to C rows through the row map.  Four consecutive
// columns per thread.
template <int DT>
__global__ __launch_bounds__(256) void splitk_reduce_kernel(GemmProblem p) {
  const int M = p.m, N = p.n;
  const int n4 = (N + 3) / 4;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= (int64_t)M * n4) return;
  const int row = (int)(idx / n4);
  const int col = (int)(idx - (int64_t)row * n4) * 4;
  const int g = row / p.rows.rows_per_group;
  const int t = row - g * p.rows.rows_per_group;
  const int64_t crow = (int64_t)g * p.rows.c_group_rows + p.rows.c_row_off + t;
  uint16_t* cp = static_cast<uint16_t*>(p.c) + crow * p.ldc;
  const int64_t plane = (int64_t)M * N;
  const float* src = p.partials + (int64_t)row * N + col;
  if ((N % 4) == 0) {
    // Up to 8 partial vectors are loaded before any is added, then added in
    // split order.
    f32x4_t s = *reinterpret_cast<const f32x4_t*>(src);
    for (int sp0 = 1; sp0 < p.splits; sp0 += 8) {
      f32x4_t v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (sp0 + q < p.splits) v[q] = *reinterpret_cast<const f32x4_t*>(src + (sp0 + q) * plane);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (sp0 + q < p.splits) s += v[q];
    }
    u32x2_t v;
    v[0] = pack2<DT>(s[0], s[1]);
    v[1] = pack2<DT>(s[2], s[3]);
    if ((p.ldc % 4) == 0) {
      *reinterpret_cast<u32x2_t*>(cp + col) = v;
    } else {
      for (int e = 0; e < 4; ++e) cp[col + e] = cvt1<DT>(s[e]);
    }
  } else {
    for (int e = 0; e < 4 && col + e < N; ++e) {
      float s = src[e];
      for (int sp = 1; sp < p.splits; ++sp) s += src[sp * plane + e];
      cp[col + e] = cvt1<DT>(s);
    }
  }
}

template <int BM, int BN, int BK, int DT, bool BT, int NST, int WAVES, int OCC, int LOOP = kLoopStages>
hipError_t launch_one(const GemmProblem& p, hipStream_t stream) {
  const int ntiles = p.order.num_rb * p.order.num_cb;
  if (p.splits > 1) {
    hipLaunchKernelGGL((gemm_mfma_kernel<BM, BN, BK, DT, BT, true, NST, WAVES, OCC, LOOP>),
                       dim3(ntiles * p.splits), dim3(64 * WAVES), 0, stream, p);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const int64_t work = (int64_t)p.m * ((p.n + 3) / 4);
    hipLaunchKernelGGL((splitk_reduce_kernel<DT>), dim3((unsigned)((work + 255) / 256)), dim3(256),
                       0, stream, p);
  } else {
    hipLaunchKernelGGL((gemm_mfma_kernel<BM, BN, BK, DT, BT, false, NST, WAVES, OCC, LOOP>),
                       dim3(ntiles), dim3(64 * WAVES), 0, stream, p);
  }
  return hipGetLastError();
}

template <int BM, int BN, int BK, int NST, int WAVES, int OCC, int LOOP = kLoopStages>
hipError_t launch_tile(const GemmProblem& p, int dtype, bool bt, hipStream_t s) {
  if (dtype == kDtypeBf16)
    return bt ? launch_one<BM, BN, BK, kDtypeBf16, true, NST, WAVES, OCC, LOOP>(p, s)
              : launch_one<BM, BN, BK, kDtypeBf16, false, NST, WAVES, OCC, LOOP>(p, s);
  return bt ? launch_one<BM, BN, BK, kDtypeFp16, true, NST, WAVES, OCC, LOOP>(p, s)
            : launch_one<BM, BN, BK, kDtypeFp16, false, NST, WAVES, OCC, LOOP>(p, s);
}

template <int BM, int BN, int BK, int DT, bool BT, int WAVES, int OCC>
hipError_t launch_m16_one(const GemmProblem& p, hipStream_t stream) {
  const int ntiles = p.order.num_rb * p.order.num_cb;
  if (p.splits > 1) {
    hipLaunchKernelGGL((gemm_m16_kernel<BM, BN, BK, DT, BT, true, WAVES, OCC>),
                       dim3(ntiles * p.splits), dim3(64 * WAVES), 0, stream, p);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const int64_t work = (int64_t)p.m * ((p.n + 3) / 4);
    hipLaunchKernelGGL((splitk_reduce_kernel<DT>), dim3((unsigned)((work + 255) / 256)), dim3(256),
                       0, stream, p);
  } else {
    hipLaunchKernelGGL((gemm_m16_kernel<BM, BN, BK, DT, BT, false, WAVES, OCC>),
                       dim3(ntiles), dim3(64 * WAVES), 0, stream, p);
  }
  return hipGetLastError();
}

// B stored n x k only (tiles whose B rows are not a power-of-two of chunks)
template <int BM, int BN, int BK, int WAVES, int OCC>
hipError_t launch_m16_bt(const GemmProblem& p, int dtype, hipStream_t s) {
  return dtype == kDtypeBf16 ? launch_m16_one<BM, BN, BK, kDtypeBf16, true, WAVES, OCC>(p, s)
                             : launch_m16_one<BM, BN, BK, kDtypeFp16, true, WAVES, OCC>(p, s);
}

template <int BM, int BN, int BK, int WAVES, int OCC>
hipError_t launch_m16(const GemmProblem& p, int dtype, bool bt, hipStream_t s) {
  if (dtype == kDtypeBf16)
    return bt ? launch_m16_one<BM, BN, BK, kDtypeBf16, true, WAVES, OCC>(p, s)
              : launch_m16_one<BM, BN, BK, kDtypeBf16, false, WAVES, OCC>(p, s);
  return bt ? launch_m16_one<BM, BN, BK, kDtypeFp16, true, WAVES, OCC>(p, s)
            : launch_m16_one<BM, BN, BK, kDtypeFp16, false, WAVES, OCC>(p, s);
}

}  // namespace

// Compiled tile configurations: output tile, k-depth of an LDS stage,
// stages in the LDS ring, waves per workgroup, waves per SIMD.
struct TileInfo { int bm, bn, bk, stages, waves, occ; };
constexpr TileInfo kTiles[kTileCount] = {
    {256, 256, 32, 4, 4, 1},   // kTile256x256:      128 KiB LDS, 3 k-tiles in flight
    {128, 128, 32, 4, 4, 2},   // kTile128x128:      64 KiB, two workgroups per CU
    {256, 128, 32, 3, 4, 2},   // kTile256x128:      72 KiB, two workgroups per CU
    {128, 64, 32, 4, 4, 1},    // kTile128x64:       48 KiB; B stored n x k only (skinny m)
    {128, 64, 32, 8, 4, 1},    // kTile128x64s8:     96 KiB, 7 k-tiles in flight; B n x k only
    {256, 256, 64, 5, 4, 1},   // kTile256x256r5:    160 KiB part ring, 64-deep k-tiles
    {128, 128, 64, 5, 4, 2},   // kTile128x128r5:    80 KiB part ring, two workgroups per CU
    {128, 64, 64, 5, 4, 2},    // kTile128x64r5:     80 KiB part ring; B stored n x k only
    {256, 256, 64, 5, 4, 1},   // kTile256x256m16:   part ring on 16x16x32 MFMAs
    {128, 128, 64, 5, 4, 2},   // kTile128x128m16:   same, two workgroups per CU
    {32, 32, 64, 4, 8, 1},     // kTileSkinny:       skinny kernel, whole k (launch_skinny_fullk)
    {256, 224, 64, 5, 4, 1},   // kTile256x224m16:   16x16x32 part ring, 7 column blocks per wave; B n x k only
};

constexpr bool all_tiles_described() {
  for (const TileInfo& t : kTiles)
    if (t.bm <= 0 || t.bn <= 0 || t.bk <= 0 || t.waves <= 0 || t.occ <= 0) return false;
  return true;
}
static_assert(all_tiles_described(), "every tile configuration needs its row of kTiles");

int tile_bm(int cfg) { return kTiles[cfg].bm; }
int tile_bn(int cfg) { return kTiles[cfg].bn; }
int tile_bk(int cfg) { return kTiles[cfg].bk; }
int tile_occ(int cfg) { return kTiles[cfg].occ; }

hipError_t launch_gemm_mfma(const GemmProblem& p, int tile_cfg, int dtype, bool rhs_transpose,
                            hipStream_t stream) {
  if (dtype != kDtypeBf16 && dtype != kDtypeFp16) return hipErrorInvalidValue;
  // an n-contiguous B tile of 64 columns is too narrow for its LDS swizzle
  if (tile_needs_bt(tile_cfg) && !rhs_transpose) return hipErrorInvalidValue;
  switch (tile_cfg) {
    case kTile256x256: return launch_tile<256, 256, 32, 4, 4, 1>(p, dtype, rhs_transpose, stream);
    case kTile128x128: return launch_tile<128, 128, 32, 4, 4, 2>(p, dtype, rhs_transpose, stream);
    case kTile256x128: return launch_tile<256, 128, 32, 3, 4, 2>(p, dtype, rhs_transpose, stream);
    case kTile128x64:
      return dtype == kDtypeBf16 ? launch_one<128, 64, 32, kDtypeBf16, true, 4, 4, 1>(p, stream)
                                 : launch_one<128, 64, 32, kDtypeFp16, true, 4, 4, 1>(p, stream);
    case kTile128x64s8:
      return dtype == kDtypeBf16 ? launch_one<128, 64, 32, kDtypeBf16, true, 8, 4, 1>(p, stream)
                                 : launch_one<128, 64, 32, kDtypeFp16, true, 8, 4, 1>(p, stream);
    case kTile256x256r5:
      return launch_tile<256, 256, 64, 5, 4, 1, kLoopParts>(p, dtype, rhs_transpose, stream);
    case kTile128x128r5:
      return launch_tile<128, 128, 64, 5, 4, 2, kLoopParts>(p, dtype, rhs_transpose, stream);
    case kTile128x64r5:
      return dtype == kDtypeBf16 ? launch_one<128, 64, 64, kDtypeBf16, true, 5, 4, 2, kLoopParts>(p, stream)
                                 : launch_one<128, 64, 64, kDtypeFp16, true, 5, 4, 2, kLoopParts>(p, stream);
    case kTile256x256m16: return launch_m16<256, 256, 64, 4, 1>(p, dtype, rhs_transpose, stream);
    case kTile128x128m16: return launch_m16<128, 128, 64, 4, 2>(p, dtype, rhs_transpose, stream);
    case kTile256x224m16: return launch_m16_bt<256, 224, 64, 4, 1>(p, dtype, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_splitk_reduce(const GemmProblem& p, int dtype, hipStream_t stream) {
  if (dtype != kDtypeBf16 && dtype != kDtypeFp16) return hipErrorInvalidValue;
  if (p.splits < 1 || p.partials == nullptr) return hipErrorInvalidValue;
  const int64_t blocks = ((int64_t)p.m * ((p.n + 3) / 4) + 255) / 256;
  if (blocks < 1 || blocks > INT32_MAX) return hipErrorInvalidValue;
  if (dtype == kDtypeBf16)
    hipLaunchKernelGGL((splitk_reduce_kernel<kDtypeBf16>), dim3((unsigned)blocks), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((splitk_reduce_kernel<kDtypeFp16>), dim3((unsigned)blocks), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace agmm
