// Device code shared by the MFMA GEMM kernels of the library (gfx950): tile
// order, global -> LDS loads, LDS swizzles, waits and the tied 16x16x32 MFMA.
// gemm_mfma.hip describes the design.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "agmm_kernels.h"

namespace agmm {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));

typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
typedef __attribute__((address_space(3))) char lds_char_t;

// 16 zero bytes: the source of every out-of-range 16-byte chunk.
__device__ __attribute__((aligned(64))) const uint32_t g_zero_chunk[16] = {0};


// Position of 16-byte chunk groups in a k-contiguous LDS row (BK elements,
// 2*BK bytes).  Both choices were measured free of LDS bank conflicts for
// the MFMA fragment reads on gfx950 (64 banks, 16 lanes per ds_read_b128
// cycle).
template <int BK>
__device__ __forceinline__ int swz_k(int row) {
  if constexpr (BK == 32) return (row >> 2) & 3;
  else return (row ^ (row >> 3)) & 7;
}
__device__ __forceinline__ int swz_n(int krow) {
  // 0, 4, 10, 14 for krow % 4 = 0..3
  const int r = krow & 3;
  return (r << 2) ^ ((r >> 1) << 1);
}

// Swizzles of the 16x16x32-MFMA kernel.  Its fragment reads differ from the
// 32x32x16 ones: a ds_read_b128 covers 16 rows x 4 chunks (lane 16g + i
// reads row i, chunk g) instead of 32 rows x 2 chunks, and a transposed B
// read covers k-rows 8g + 0..3 for g = 0..3.  Rocprof counters showed the
// 32x32 swizzles costing this kernel LDS bank-conflict stalls on ~16% of
// its cycles (against 0.3% in the 32x32 kernel).  Both patterns agree with
// the LDS serving a b128 read in passes of lanes 8p..8p+7 with
// 32+8p..32+8p+7, and a b64 read in passes of 32 lanes.  Under that
// grouping:
//  * k-contiguous rows of 128 bytes: chunk c of row r at c ^ swz_k16(r).
//    A pass reads 8 consecutive rows x chunks {g, g ^ 2}; the 4 rows of one
//    parity (one 128-byte bank half) get swizzles 0, 1, 4, 5 (first 8 rows
//    of 16) or 2, 3, 6, 7 (last 8), so the 8 chunks they need are distinct.
//    Any 16 consecutive rows use 8 distinct swizzles per parity as well.
//  * n-contiguous B k-rows: the 32x32 swizzle of k-row r (by r % 4), plus
//    a flip of chunk bit 1 for k-rows with bit 3 set, which puts k-rows r
//    and r + 8 (read in the same pass) on disjoint bank sets.
__device__ __forceinline__ int swz_k16(int row) {
  return ((row >> 1) & 1) | (row & 4) | ((row >> 2) & 2);
}
__device__ __forceinline__ int swz_n16(int krow) { return swz_n(krow) ^ ((krow >> 2) & 2); }

template <int DT>
__device__ __forceinline__ f32x16_t mfma32(u32x4_t a, u32x4_t b, f32x16_t c) {
  if constexpr (DT == kDtypeBf16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  }
}

// fp32 -> 16-bit storage, round to nearest even (subnormals kept for fp16).
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == kDtypeBf16) {
    __bf16 a = (__bf16)lo, b = (__bf16)hi;
    return (uint32_t)__builtin_bit_cast(uint16_t, a) | ((uint32_t)__builtin_bit_cast(uint16_t, b) << 16);
  } else {
    _Float16 a = (_Float16)lo, b = (_Float16)hi;
    return (uint32_t)__builtin_bit_cast(uint16_t, a) | ((uint32_t)__builtin_bit_cast(uint16_t, b) << 16);
  }
}

template <int DT>
__device__ __forceinline__ uint16_t cvt1(float v) {
  if constexpr (DT == kDtypeBf16) {
    __bf16 a = (__bf16)v;
    return __builtin_bit_cast(uint16_t, a);
  } else {
    _Float16 a = (_Float16)v;
    return __builtin_bit_cast(uint16_t, a);
  }
}

// One 16-byte-per-lane global -> LDS load: lane i of the wave writes bytes
// [16i, 16i+16) of the 1 KiB LDS block at `lds_block` (wave-uniform).
// Issued as inline assembly on purpose: the compiler cannot tell which LDS
// bytes such a load writes, so it would otherwise wait for every one of
// them (vmcnt(0)) before the next LDS read anywhere in the kernel, which
// defeats the multi-stage pipeline.  The kernel instead waits explicitly for
// exactly the k-tile it is about to read (wait_vmcnt + barrier).
__device__ __forceinline__ void load_lds16(const void* gsrc, char* lds_block) {
  const uint32_t lds = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_char_t*)lds_block);
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(gsrc), "s"(lds)
               : "m0");
}

// Same, with the LDS destination given as a 32-bit LDS address (no generic
// pointer conversion per load).
__device__ __forceinline__ void load_lds16_at(const void* gsrc, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(gsrc), "s"(__builtin_amdgcn_readfirstlane(lds_addr))
               : "m0");
}

// Buffer-descriptor form of the same load: the 64-bit base sits in the
// scalar descriptor, each lane adds a 32-bit offset (`voff`) and the wave a
// scalar one (`soff`).  Interior tiles use it: their per-lane offsets stay
// fixed over the k loop, so a load costs no vector address arithmetic (the
// flat form adds a 64-bit k offset to every lane's pointer per load), and the
// descriptor's record count bounds every lane's offset.  LDS placement is the
// flat form's: lane i writes bytes [16i, 16i+16) of a 1 KiB block.
// The load goes into block R (0..3) of a 4 KiB LDS group: the instruction's
// offset field, R KiB, moves the LDS destination and the memory address
// alike, so `voff` is the lane's offset less R KiB.  With SET the load first
// writes the group's base into M0; without it M0 must already hold that
// base (the previous load of the group set it, and nothing between writes
// M0).  Writing M0 right before a DMA load costs the issuing wave about nine
// cycles beside its MFMA stream, against about one for the load alone
// (measured on MI355X), so one write serves four loads.
template <int R, bool SET>
__device__ __forceinline__ void load_lds16_buf_grp(const u32x4_t& rsrc, uint32_t voff, uint32_t soff,
                                                   uint32_t group_lds) {
  static_assert(R >= 0 && R < 4, "block of a 4 KiB group");
  if constexpr (SET)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %3 offen offset:%4 lds"
                 :
                 : "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(group_lds)),
                   "s"(__builtin_amdgcn_readfirstlane(soff)), "n"(R * 1024)
                 : "m0");
  else
    asm volatile("buffer_load_dwordx4 %0, %1, %2 offen offset:%3 lds"
                 :
                 : "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(soff)), "n"(R * 1024)
                 : "memory");
}

// Load j of a part: block j % 4 of group j / 4; M0 is written at the first
// block of each group.  A part's loads are issued in increasing j with no
// other M0 write between them.
__device__ __forceinline__ void load_lds16_buf_j(int j, const u32x4_t& rsrc, uint32_t voff_shifted,
                                                 uint32_t soff, uint32_t part_lds) {
  const uint32_t grp = part_lds + (uint32_t)(j & ~3) * 1024u;
  switch (j & 3) {
    case 0: load_lds16_buf_grp<0, true>(rsrc, voff_shifted, soff, grp); break;
    case 1: load_lds16_buf_grp<1, false>(rsrc, voff_shifted, soff, grp); break;
    case 2: load_lds16_buf_grp<2, false>(rsrc, voff_shifted, soff, grp); break;
    default: load_lds16_buf_grp<3, false>(rsrc, voff_shifted, soff, grp); break;
  }
}

// Raw buffer descriptor (stride 0, so the record count is in bytes) over
// `bytes` bytes from `base`; the last word is the gfx9 data-format word.
__device__ __forceinline__ u32x4_t buffer_rsrc(const void* base, uint64_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  u32x4_t r;
  r[0] = __builtin_amdgcn_readfirstlane((uint32_t)b);
  r[1] = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32) & 0xFFFFu);
  r[2] = __builtin_amdgcn_readfirstlane((uint32_t)bytes);
  r[3] = 0x00020000u;
  return r;
}

__device__ __forceinline__ u32x2_t read_tr(const char* p) {
  i16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(lds_char_t*)p);
  return __builtin_bit_cast(u32x2_t, v);
}

// vmcnt(n) with the other counters left alone (gfx9 encoding).
// The scheduling barrier keeps the wait where it is written: the compiler
// would otherwise hoist it above independent MFMAs and stall them.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// Workgroup barrier without the release/acquire fence of __syncthreads():
// that fence would also wait for the in-flight global->LDS loads of the
// next k-tiles.  Completion of the loads a k-tile needs is awaited
// explicitly (wait_vmcnt) before this barrier; the empty asm statements keep
// the compiler from moving LDS accesses across it.
__device__ __forceinline__ void block_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Logical tile visited by this workgroup.
__device__ __forceinline__ void tile_coords(const TileOrder& o, int wg, int nwg, int& rb, int& cb) {
  if (o.xcd_remap) {
    // Workgroups are dispatched round-robin over the 8 XCDs; give XCD x a
    // contiguous range of logical tiles so neighbours share its L2.
    const int xcd = wg & 7, local = wg >> 3;
    const int per = nwg >> 3, rem = nwg & 7;
    wg = xcd * per + (xcd < rem ? xcd : rem) + local;
  }
  const int gsz = o.group_m * o.num_cb;
  const int grp = wg / gsz;
  const int first = grp * o.group_m;
  const int rows_here = min(o.num_rb - first, o.group_m);
  const int in = wg - grp * gsz;
  const int rbi = first + in % rows_here;
  cb = in / rows_here;
  rb = o.rb_order ? o.rb_order[rbi] : rbi;
}

// Main-loop forms.
//   kLoopStages:   ring of NST stages, each one k-tile of A and B.
//   kLoopParts:    ring of NST slots, each holding one operand of one k-tile
//                  ("part"); the parts alternate A, B, A, B, ...  With an odd
//                  slot count this keeps 2.5 k-tiles of 64-deep operands in
//                  LDS, i.e. 128-byte row pieces per load (a whole L2 line)
//                  with a load depth that whole stages could not fit.
template <bool B>
struct BoolTag {
  static constexpr bool value = B;
};
template <int V>
struct IntTag {
  static constexpr int value = V;
};

constexpr int kLoopStages = 0;
constexpr int kLoopParts = 2;

template <int BM, int BN, int BK, int DT, bool BT, int NST, int WAVES, int LOOP = kLoopStages>
struct GemmTile {
  static constexpr int kStages = NST;
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int WM = 2, WN = WAVES / 2;      // wave grid over the output tile
  static constexpr int TM = BM / WM, TN = BN / WN;     // per-wave tile
  static constexpr int FM = TM / 32, FN = TN / 32;     // 32x32 MFMA blocks per wave
  static constexpr int KROW = BK * 2;                  // bytes of a k-contiguous LDS row
  static constexpr int CPR = BK / 8;                   // 16-byte chunks per such row
  static constexpr int RPI = 1024 / KROW;              // rows one 1 KiB load instruction fills
  static constexpr int SUB = BK / 16;                  // k16 MFMA substeps per k-tile
  static constexpr int A_BYTES = BM * KROW;
  static constexpr int B_BYTES = BN * KROW;            // same size in both B layouts
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int PART_BYTES = A_BYTES > B_BYTES ? A_BYTES : B_BYTES;
  static constexpr int LDS_BYTES = LOOP == kLoopParts ? kStages * PART_BYTES : kStages * STAGE_BYTES;
  static constexpr int A_IPW = A_BYTES / 1024 / WAVES; // 1 KiB load instructions per wave
  static constexpr int B_IPW = B_BYTES / 1024 / WAVES;
  static constexpr int LOADS = A_IPW + B_IPW;          // per wave per k-tile
  static constexpr int B_ROW = BN * 2;                 // bytes of an n-contiguous k-row
  // Where in a k-tile the workgroup synchronises: in the middle when at
  // least 3 stages leave a tile of slack, else at the end of the tile.
  static constexpr bool MID_SYNC = NST >= 3;
  static constexpr int SYNC_SUB = MID_SYNC ? SUB / 2 : SUB;
  static_assert(BK == 32 || BK == 64, "BK");
  static_assert(WAVES == 4 || WAVES == 8, "waves");
  static_assert(FM >= 1 && FN >= 1, "tile too small");
  static_assert(A_IPW >= 1 && B_IPW >= 1, "tile too small for the load split");
  static_assert(LDS_BYTES <= 160 * 1024, "LDS budget");
  static_assert(LOOP == kLoopParts || (NST - 1) * LOADS < 64, "vmcnt range");
  static_assert(NST >= 2 && NST <= 8, "stages");
  // part ring: 5 slots (parts 2t, 2t+1 = A, B of k-tile t live in slots
  // (2t) % 5 and (2t+1) % 5), at most 2 A parts and one B part in flight
  static_assert(LOOP != kLoopParts || (NST == 5 && A_IPW >= B_IPW && SUB >= 2 && 2 * A_IPW + B_IPW < 64),
                "part ring layout");
};

// acc += B-fragment x A-fragment on one 16x16 block, accumulator tied to its
// AGPRs.  Written as inline assembly because the compiler gives the builtin
// for this shape a separate destination and copies every accumulator once
// per use (four register moves per MFMA); with the operand tied read-write
// the 64 accumulators of a 128x128 sub-tile stay in place.  Being opaque to
// the hazard recognizer, the caller keeps the rules the compiler would:
// fragment registers come straight from LDS reads (waitcnt covers those),
// and the accumulators are touched by no other instruction between the
// mfma16_drain() calls around the main loop.
template <int DT>
__device__ __forceinline__ void mfma16(f32x4_t& c, const u32x4_t& b, const u32x4_t& a) {
  if constexpr (DT == kDtypeBf16)
    asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
  else
    asm("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
}

template <int DT>
__device__ __forceinline__ f32x4_t mfma16_builtin(u32x4_t b, u32x4_t a, f32x4_t c) {
  if constexpr (DT == kDtypeBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, b),
                                                   __builtin_bit_cast(bf16x8_t, a), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, b),
                                                  __builtin_bit_cast(f16x8_t, a), c, 0, 0, 0);
}

// Wait states between MFMAs and any other instruction that reads or writes
// their accumulators (more than the longest MFMA-to-VALU dependency).  The
// empty statements tie every accumulator on both sides, so no read or write
// of one can be placed across the wait.
template <int FM, int FN>
__device__ __forceinline__ void mfma16_drain(f32x4_t (&acc)[FM][FN]) {
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) asm volatile("" : "+a"(acc[i][j]));
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) asm volatile("" : "+a"(acc[i][j]));
}

}  // namespace

}  // namespace agmm
