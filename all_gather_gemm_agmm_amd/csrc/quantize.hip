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

template <int I>
struct Row {
  static constexpr int value = I;
};

constexpr float kTinyScale = 1.17549435082228750797e-38f;   // 2^-126: 1 / s stays finite

template <int FMT>
__device__ __forceinline__ float top_value() { return FMT == kFmtE4M3 ? 448.0f : 57344.0f; }

// 8 consecutive elements of a row, as they are stored.  Sizes (the bits of
// |x|, which order like |x|) are kept two to a word for the 16-bit types.
template <int DT>
struct Eight {
  static constexpr bool kWide = DT == kDtypeFp32;
  static constexpr int W = kWide ? 8 : 4;
  uint32_t w[W];

  // from column c of a row; elements at or past `left` (columns that remain)
  // are zero.  VEC: 16-byte aligned rows.
  template <bool VEC>
  __device__ __forceinline__ void load(const char* row, int64_t c, int64_t left) {
    if (VEC && left >= 8) {
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const u32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(row + c * (kWide ? 4 : 2)) + q);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * q + e] = v[e];
      }
    } else if constexpr (kWide) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = e < left ? reinterpret_cast<const uint32_t*>(row)[c + e] : 0u;
    } else {
      const uint16_t* s = reinterpret_cast<const uint16_t*>(row) + c;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = (2 * e < left ? (uint32_t)s[2 * e] : 0u) | (2 * e + 1 < left ? (uint32_t)s[2 * e + 1] << 16 : 0u);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < W; ++e) w[e] = 0;
  }
  __device__ __forceinline__ float value(int e) const {
    if constexpr (kWide) {
      return __builtin_bit_cast(float, w[e]);
    } else if constexpr (DT == kDtypeBf16) {
      return __builtin_bit_cast(float, e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
    } else {
      const uint16_t h = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      return (float)__builtin_bit_cast(_Float16, h);
    }
  }
};

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

// Sizes of word q, infinities and NaN included.
template <int DT>
__device__ __forceinline__ uint32_t sizes(uint32_t w) {
  return w & (Eight<DT>::kWide ? 0x7FFFFFFFu : 0x7FFF7FFFu);
}
template <int DT>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  if constexpr (Eight<DT>::kWide)
    return max(a, b);
  else
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}
// Whether a word of sizes holds an infinity or NaN, and the word without them.
template <int DT>
__device__ __forceinline__ bool odd_sizes(uint32_t s) {
  constexpr uint32_t kInf = DT == kDtypeFp32 ? 0x7F800000u : DT == kDtypeBf16 ? 0x7F80u : 0x7C00u;
  return Eight<DT>::kWide ? s >= kInf : (s & 0xFFFFu) >= kInf || (s >> 16) >= kInf;
}
template <int DT>
__device__ __forceinline__ uint32_t finite_sizes(uint32_t s) {
  constexpr uint32_t kInf = DT == kDtypeFp32 ? 0x7F800000u : DT == kDtypeBf16 ? 0x7F80u : 0x7C00u;
  if constexpr (Eight<DT>::kWide) return s < kInf ? s : 0u;
  else return ((s & 0xFFFFu) < kInf ? s & 0xFFFFu : 0u) | ((s >> 16) < kInf ? s & 0xFFFF0000u : 0u);
}
// The larger half of a word, and its value (a size of the type) as fp32.
template <int DT>
__device__ __forceinline__ uint32_t one_size(uint32_t s) {
  return Eight<DT>::kWide ? s : max(s & 0xFFFFu, s >> 16);
}
template <int DT>
__device__ __forceinline__ float size_value(uint32_t s) {
  if constexpr (DT == kDtypeFp32) return __builtin_bit_cast(float, s);
  else if constexpr (DT == kDtypeBf16) return __builtin_bit_cast(float, s << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)s);
}

// Maximum over the 16 lanes of a DPP row, in every lane: rotations by 8, 4, 2, 1.
template <int DT>
__device__ __forceinline__ uint32_t max16(uint32_t b) {
  b = larger<DT>(b, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x128, 0xF, 0xF, true));
  b = larger<DT>(b, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x124, 0xF, 0xF, true));
  b = larger<DT>(b, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x122, 0xF, 0xF, true));
  b = larger<DT>(b, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, 0x121, 0xF, 0xF, true));
  return b;
}

// The value of lane I of each DPP row, in the row's every lane.
template <int I>
__device__ __forceinline__ float row_lane(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x150 + I, 0xF, 0xF, true));
}

template <int FMT>
__device__ __forceinline__ float scale_of(float size) {
  return fmaxf(size / top_value<FMT>(), kTinyScale);
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

template <int FMT, int DT>
__device__ __forceinline__ u32x2_t pack8(const Eight<DT>& v, float inv) {
  return u32x2_t{pack4<FMT>(v.value(0) * inv, v.value(1) * inv, v.value(2) * inv, v.value(3) * inv),
                 pack4<FMT>(v.value(4) * inv, v.value(5) * inv, v.value(6) * inv, v.value(7) * inv)};
}

template <int DT, int FMT, bool VEC, int RPW>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantProblem p) {
  constexpr int ES = DT == kDtypeFp32 ? 4 : 2;
  using E = Eight<DT>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cw = (int)((p.cols + 511) / 512);                  // 512-column pieces of a row
  const int piece = blockIdx.x % cw, rgrp = blockIdx.x / cw;
  const int64_t c = (int64_t)piece * 512 + lane * 8, left = p.cols - c;
  const int64_t r0 = ((int64_t)rgrp * 4 + wave) * RPW;
  E v[RPW];
#pragma unroll
  for (int i = 0; i < RPW; ++i)
    if (r0 + i < p.rows && left > 0) v[i].template load<VEC>(static_cast<const char*>(p.x) + (r0 + i) * p.ldx * ES, c, left);
    else v[i].zero();
#pragma unroll
  for (int i = 0; i < RPW; ++i) {
    uint32_t b = sizes<DT>(v[i].w[0]);
#pragma unroll
    for (int e = 1; e < E::W; ++e) b = larger<DT>(b, sizes<DT>(v[i].w[e]));
    if (odd_sizes<DT>(b)) {
      b = 0;
#pragma unroll
      for (int e = 0; e < E::W; ++e) b = larger<DT>(b, finite_sizes<DT>(sizes<DT>(v[i].w[e])));
    }
    const float s = scale_of<FMT>(size_value<DT>(one_size<DT>(max16<DT>(b))));
    const float inv = 1.0f / s;
    if (r0 + i >= p.rows) break;
    if (c < p.cols16)
      *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(p.q) + (r0 + i) * p.ldq + c) = pack8<FMT>(v[i], inv);
    if ((lane & 15) == 0 && left > 0) p.scale[(c >> 7) * p.rows + r0 + i] = s;
  }
}

// One 128 x 128 tile; p.q and p.qt either may be null.  A quotient costs as
// much as the rest of the work on an element, so each scale and its inverse
// are computed once per row (by one lane of 16, then broadcast) and once per
// column (by one thread, then read from LDS).
template <int DT, int FMT, bool VEC, bool SQUARE>
__global__ __launch_bounds__(256) void quantize_tile_kernel(QuantProblem p) {
  constexpr int ES = DT == kDtypeFp32 ? 4 : 2;
  using E = Eight<DT>;
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * 128];
  __shared__ __attribute__((aligned(16))) uint32_t cmax[4][16][E::W];   // column sizes: wave, 8-column piece, word
  __shared__ __attribute__((aligned(16))) float cinv[128];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t kb = (p.cols + 127) / 128, rb = (p.rows + 127) / 128;
  const int64_t tb = blockIdx.x % (uint32_t)kb, tr = blockIdx.x / (uint32_t)kb;
  const int cl = tid & 15, rl = tid >> 4;                      // 8-column and 8-row piece of this thread
  const int64_t c0 = tb * 128 + cl * 8, r0 = tr * 128 + rl * 8;
  const int64_t left = p.cols - c0;
  E v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + i < p.rows && left > 0) v[i].template load<VEC>(static_cast<const char*>(p.x) + (r0 + i) * p.ldx * ES, c0, left);
    else v[i].zero();

  uint32_t col[E::W], row[8];   // sizes of the piece's columns (by words) and rows
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < E::W; ++e) {
      const uint32_t b = sizes<DT>(v[i].w[e]);
      row[i] = e ? larger<DT>(row[i], b) : b;
      col[e] = i ? larger<DT>(col[e], b) : b;
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) most = larger<DT>(most, row[i]);
  if (odd_sizes<DT>(most)) {   // some infinity or NaN: once more, without them
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < E::W; ++e) {
        const uint32_t b = finite_sizes<DT>(sizes<DT>(v[i].w[e]));
        row[i] = e ? larger<DT>(row[i], b) : b;
        col[e] = i ? larger<DT>(col[e], b) : b;
      }
  }

  float inv_all = 0.0f;        // SQUARE: of the tile
  if constexpr (SQUARE) {
    uint32_t b = row[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) b = larger<DT>(b, row[i]);
    b = max16<DT>(b);
    b = larger<DT>(b, (uint32_t)__shfl_xor((int)b, 16));
    b = larger<DT>(b, (uint32_t)__shfl_xor((int)b, 32));
    if (lane == 0) cmax[wave][0][0] = b;
    __syncthreads();
    b = larger<DT>(larger<DT>(cmax[0][0][0], cmax[1][0][0]), larger<DT>(cmax[2][0][0], cmax[3][0][0]));
    const float s = scale_of<FMT>(size_value<DT>(one_size<DT>(b)));
    inv_all = 1.0f / s;
    if (tid == 0) {
      if (p.q) p.scale[tb * rb + tr] = s;
      if (p.qt) p.scale_t[tr * kb + tb] = s;
    }
  } else if (p.qt) {
#pragma unroll
    for (int e = 0; e < E::W; ++e) {
      col[e] = larger<DT>(col[e], (uint32_t)__shfl_xor((int)col[e], 16));
      col[e] = larger<DT>(col[e], (uint32_t)__shfl_xor((int)col[e], 32));
      if (lane < 16) cmax[wave][cl][e] = col[e];
    }
    __syncthreads();
    if (tid < 128) {
      uint32_t b = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) b = larger<DT>(b, cmax[w][tid >> 3][E::kWide ? tid & 7 : (tid & 7) >> 1]);
      if (!E::kWide) b = tid & 1 ? b >> 16 : b & 0xFFFFu;
      const float s = scale_of<FMT>(size_value<DT>(b));
      cinv[tid] = 1.0f / s;
      if (tb * 128 + tid < p.cols) p.scale_t[tr * p.cols + tb * 128 + tid] = s;
    }
    __syncthreads();
  }

  if (p.q) {
    float inv = inv_all;
    if constexpr (!SQUARE) {
      // lane cl of 16 takes row cl % 8: its size, scale and inverse
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = one_size<DT>(max16<DT>(row[i]));
        mine = (cl & 7) == i ? b : mine;
      }
      const float s = scale_of<FMT>(size_value<DT>(mine));
      inv = 1.0f / s;
      if (cl < 8 && r0 + cl < p.rows) p.scale[tb * p.rows + r0 + cl] = s;
    }
    const auto put = [&](auto row_tag) {
      constexpr int I = decltype(row_tag)::value;
      const float f = SQUARE ? inv_all : row_lane<I>(inv);
      if (r0 + I < p.rows && c0 < p.cols16)
        *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(p.q) + (r0 + I) * p.ldq + c0) = pack8<FMT>(v[I], f);
    };
    put(Row<0>{});
    put(Row<1>{});
    put(Row<2>{});
    put(Row<3>{});
    put(Row<4>{});
    put(Row<5>{});
    put(Row<6>{});
    put(Row<7>{});
  }
  if (p.qt) {
    // 8 rows of one column are 8 consecutive bytes of the transposed tile:
    // 8-byte piece rl of tile row c sits at piece rl ^ (c / 8).
    float ci[8];
    if constexpr (SQUARE) {
#pragma unroll
      for (int e = 0; e < 8; ++e) ci[e] = inv_all;
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const f32x4_t c4 = *reinterpret_cast<const f32x4_t*>(cinv + cl * 8 + 4 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e) ci[4 * q + e] = c4[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      *reinterpret_cast<u32x2_t*>(tile + (cl * 8 + e) * 128 + (rl ^ cl) * 8) =
          u32x2_t{pack4<FMT>(v[0].value(e) * ci[e], v[1].value(e) * ci[e], v[2].value(e) * ci[e], v[3].value(e) * ci[e]),
                  pack4<FMT>(v[4].value(e) * ci[e], v[5].value(e) * ci[e], v[6].value(e) * ci[e], v[7].value(e) * ci[e])};
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
