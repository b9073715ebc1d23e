// Block-scaled 8-bit quantiser (gfx950): the operands of the block-scaled
// product from bf16, fp16 or fp32 matrices.
//
//     s = max(max_{block} |x| / F, 2^-126)      (finite elements only)
//     q = rne8(x * (1 / s))                     F = 448 (e4m3), 57344 (e5m2)
//
// with one block per 128 consecutive elements of a row (block_rows 1) or per
// 128 x 128 tile (block_rows 128), of x, of x transposed, or of both from one
// read of x.  s and 1 / s are correctly rounded fp32 quotients and the product
// is rounded once to fp32 before its rounding to 8 bits, so the result is
// the same on every path.  |x * (1 / s)| <= F (1 + 2^-22), which rounds to at
// most F; non-finite elements do not enter a maximum and come out as NaN
// (e4m3) or as themselves (e5m2), never as a finite number.
//
// Bound: HBM.  Each element is read once and written once (twice for
// "both").
//
//  * quantize_rows_kernel (block_rows 1, x as it stands): a lane holds 8
//    consecutive elements, 16 lanes a block, so the maximum is four DPP steps
//    within a row of 16 lanes; a wave takes 512 columns and RPW rows, all of
//    its loads in flight before the first is used.  The scales of a
//    workgroup's rows are neighbours in [block][row] order.
//  * quantize_tile_kernel (transposed outputs, 128 x 128 blocks): one 128 x
//    128 tile per workgroup, 8 rows x 8 columns per thread, so that a thread
//    holds 8 consecutive elements of both orders; the transposed bytes pass
//    through 16 KiB of LDS and leave as whole 128-byte rows.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "agmm_kernels.h"

namespace agmm {

namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x8_t __attribute__((ext_vector_type(8)));

constexpr float kTinyScale = 1.17549435082228750797e-38f;   // 2^-126: 1 / s stays finite

template <int FMT>
__device__ __forceinline__ float top_value() { return FMT == kFmtE4M3 ? 448.0f : 57344.0f; }

// 8 consecutive elements from column c of a row; elements at or past `left`
// (columns that remain) are zero.  VEC: 16-byte aligned rows.
template <int DT, bool VEC>
__device__ __forceinline__ f32x8_t load8(const char* row, int64_t c, int64_t left) {
  f32x8_t v;
  if constexpr (DT == kDtypeFp32) {
    const float* s = reinterpret_cast<const float*>(row) + c;
    if (VEC && left >= 8) {
      const f32x4_t a = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(s));
      const f32x4_t b = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(s) + 1);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = a[e];
        v[4 + e] = b[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < left ? s[e] : 0.0f;
    }
  } else {
    const uint16_t* s = reinterpret_cast<const uint16_t*>(row) + c;
    uint32_t w[4];
    if (VEC && left >= 8) {
      const u32x4_t a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(s));
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = a[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = (2 * e < left ? (uint32_t)s[2 * e] : 0u) | (2 * e + 1 < left ? (uint32_t)s[2 * e + 1] << 16 : 0u);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (DT == kDtypeBf16) {
        v[2 * e] = __builtin_bit_cast(float, w[e] << 16);
        v[2 * e + 1] = __builtin_bit_cast(float, w[e] & 0xFFFF0000u);
      } else {
        v[2 * e] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[e] & 0xFFFFu));
        v[2 * e + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[e] >> 16));
      }
    }
  }
  return v;
}

// Bits of |x| (they order like |x|), 0 for infinities and NaN.
__device__ __forceinline__ uint32_t size_bits(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}

// Maximum over the 16 lanes of a DPP row, in every lane: rotations by 8, 4, 2, 1.
__device__ __forceinline__ uint32_t max16(uint32_t b) {
  b = max(b, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x128, 0xF, 0xF, true));
  b = max(b, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x124, 0xF, 0xF, true));
  b = max(b, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x122, 0xF, 0xF, true));
  b = max(b, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x121, 0xF, 0xF, true));
  return b;
}

template <int FMT>
__device__ __forceinline__ float scale_of(uint32_t bits) {
  return fmaxf(__builtin_bit_cast(float, bits) / top_value<FMT>(), kTinyScale);
}

// Four fp32 values (already scaled) to four 8-bit ones.
template <int FMT>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int w = 0;
  if constexpr (FMT == kFmtE4M3) {
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  } else {
    w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
  }
  return (uint32_t)w;
}

template <int DT, int FMT, bool VEC, int RPW>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantProblem p) {
  constexpr int ES = DT == kDtypeFp32 ? 4 : 2;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t cw = (p.cols + 511) / 512;                     // 512-column pieces of a row
  const int64_t piece = blockIdx.x % cw, rgrp = blockIdx.x / cw;
  const int64_t c = piece * 512 + lane * 8, left = p.cols - c;
  const int64_t r0 = (rgrp * 4 + wave) * RPW;
  f32x8_t v[RPW];
#pragma unroll
  for (int i = 0; i < RPW; ++i)
    if (r0 + i < p.rows && left > 0)
      v[i] = load8<DT, VEC>(static_cast<const char*>(p.x) + (r0 + i) * p.ldx * ES, c, left);
    else
      v[i] = f32x8_t{};
  const int64_t block = c >> 7;
#pragma unroll
  for (int i = 0; i < RPW; ++i) {
    uint32_t b = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) b = max(b, size_bits(v[i][e]));
    const float s = scale_of<FMT>(max16(b));
    const float inv = 1.0f / s;
    if (r0 + i >= p.rows) break;
    if (c < p.cols16)
      *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(p.q) + (r0 + i) * p.ldq + c) =
          u32x2_t{pack4<FMT>(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv),
                  pack4<FMT>(v[i][4] * inv, v[i][5] * inv, v[i][6] * inv, v[i][7] * inv)};
    if ((lane & 15) == 0 && left > 0) p.scale[block * p.rows + r0 + i] = s;
  }
}

// One 128 x 128 tile; p.q and p.qt either may be null.
template <int DT, int FMT, bool VEC, bool SQUARE>
__global__ __launch_bounds__(256) void quantize_tile_kernel(QuantProblem p) {
  constexpr int ES = DT == kDtypeFp32 ? 4 : 2;
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * 128];
  __shared__ uint32_t cmax[4][128];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t kb = (p.cols + 127) / 128, rb = (p.rows + 127) / 128;
  const int64_t tb = blockIdx.x % kb, tr = blockIdx.x / kb;
  const int cl = tid & 15, rl = tid >> 4;                      // 8-column and 8-row piece of this thread
  const int64_t c0 = tb * 128 + cl * 8, r0 = tr * 128 + rl * 8;
  const int64_t left = p.cols - c0;
  f32x8_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + i < p.rows && left > 0)
      v[i] = load8<DT, VEC>(static_cast<const char*>(p.x) + (r0 + i) * p.ldx * ES, c0, left);
    else
      v[i] = f32x8_t{};

  uint32_t colb[8] = {};
  uint32_t rowb[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    rowb[i] = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = size_bits(v[i][e]);
      rowb[i] = max(rowb[i], b);
      colb[e] = max(colb[e], b);
    }
  }
  // Column maxima (or the tile's one): over the wave's four 8-row pieces,
  // then over the four waves in LDS.
  float cs[8], cinv[8];
  if constexpr (SQUARE) {
    uint32_t b = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) b = max(b, colb[e]);
    b = max16(b);
    b = max(b, (uint32_t)__shfl_xor((int)b, 16));
    b = max(b, (uint32_t)__shfl_xor((int)b, 32));
    if (lane == 0) cmax[wave][0] = b;
    __syncthreads();
    b = max(max(cmax[0][0], cmax[1][0]), max(cmax[2][0], cmax[3][0]));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cs[e] = e ? cs[0] : scale_of<FMT>(b);
      cinv[e] = e ? cinv[0] : 1.0f / cs[0];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      colb[e] = max(colb[e], (uint32_t)__shfl_xor((int)colb[e], 16));
      colb[e] = max(colb[e], (uint32_t)__shfl_xor((int)colb[e], 32));
      if (lane < 16) cmax[wave][cl * 8 + e] = colb[e];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = cl * 8 + e;
      cs[e] = scale_of<FMT>(max(max(cmax[0][c], cmax[1][c]), max(cmax[2][c], cmax[3][c])));
      cinv[e] = 1.0f / cs[e];
    }
  }

  if (p.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s, inv;
      if constexpr (SQUARE) {
        s = cs[0];
        inv = cinv[0];
      } else {
        s = scale_of<FMT>(max16(rowb[i]));
        inv = 1.0f / s;
      }
      if (r0 + i < p.rows && c0 < p.cols16)
        *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(p.q) + (r0 + i) * p.ldq + c0) =
            u32x2_t{pack4<FMT>(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv),
                    pack4<FMT>(v[i][4] * inv, v[i][5] * inv, v[i][6] * inv, v[i][7] * inv)};
      if (!SQUARE && cl == 0 && r0 + i < p.rows) p.scale[tb * p.rows + r0 + i] = s;
    }
    if (SQUARE && tid == 0) p.scale[tb * rb + tr] = cs[0];
  }
  if (p.qt) {
    // 8 rows of one column are 8 consecutive bytes of the transposed tile:
    // 8-byte piece rl of tile row c sits at piece rl ^ (c / 8).
#pragma unroll
    for (int e = 0; e < 8; ++e)
      *reinterpret_cast<u32x2_t*>(tile + (cl * 8 + e) * 128 + (rl ^ cl) * 8) =
          u32x2_t{pack4<FMT>(v[0][e] * cinv[e], v[1][e] * cinv[e], v[2][e] * cinv[e], v[3][e] * cinv[e]),
                  pack4<FMT>(v[4][e] * cinv[e], v[5][e] * cinv[e], v[6][e] * cinv[e], v[7][e] * cinv[e])};
    if constexpr (SQUARE) {
      if (tid == 0) p.scale_t[tr * kb + tb] = cs[0];
    } else {
      if (rl == 0)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c0 + e < p.cols) p.scale_t[tr * p.cols + c0 + e] = cs[e];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = i * 16 + rl;                                // column of x, row of the output
      const int64_t gc = tb * 128 + c, gr = tr * 128 + cl * 8;
      if (gc < p.cols && gr < p.rows16)
        *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(p.qt) + gc * p.ldqt + gr) =
            *reinterpret_cast<const u32x2_t*>(tile + c * 128 + (cl ^ (c >> 3)) * 8);
    }
  }
}

template <int DT, int FMT, bool VEC>
hipError_t launch(const QuantProblem& p, hipStream_t stream) {
  if (p.block_rows == 1 && !p.qt) {
    const int64_t cw = (p.cols + 511) / 512;
    // 8 rows per wave where that still gives every CU several workgroups,
    // else 1: a small call is bound by latency, and more waves hide it.
    const bool deep = cw * ((p.rows + 31) / 32) >= 1024;
    const int64_t grid = cw * ((p.rows + (deep ? 32 : 4) - 1) / (deep ? 32 : 4));
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    if (deep) hipLaunchKernelGGL((quantize_rows_kernel<DT, FMT, VEC, 8>), dim3((unsigned)grid), dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((quantize_rows_kernel<DT, FMT, VEC, 1>), dim3((unsigned)grid), dim3(256), 0, stream, p);
  } else {
    const int64_t grid = ((p.cols + 127) / 128) * ((p.rows + 127) / 128);
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    if (p.block_rows == 1)
      hipLaunchKernelGGL((quantize_tile_kernel<DT, FMT, VEC, false>), dim3((unsigned)grid), dim3(256), 0, stream, p);
    else
      hipLaunchKernelGGL((quantize_tile_kernel<DT, FMT, VEC, true>), dim3((unsigned)grid), dim3(256), 0, stream, p);
  }
  return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const QuantProblem& p, hipStream_t s) {
  constexpr int ES = DT == kDtypeFp32 ? 4 : 2;
  const bool vec = (p.ldx * ES) % 16 == 0 && (reinterpret_cast<uintptr_t>(p.x) & 15) == 0;
  if (p.format == kFmtE4M3) return vec ? launch<DT, kFmtE4M3, true>(p, s) : launch<DT, kFmtE4M3, false>(p, s);
  return vec ? launch<DT, kFmtE5M2, true>(p, s) : launch<DT, kFmtE5M2, false>(p, s);
}

}  // namespace

hipError_t launch_quantize(const QuantProblem& p, hipStream_t stream) {
  switch (p.dtype) {
    case kDtypeBf16: return launch_dt<kDtypeBf16>(p, stream);
    case kDtypeFp16: return launch_dt<kDtypeFp16>(p, stream);
    case kDtypeFp32: return launch_dt<kDtypeFp32>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace agmm
