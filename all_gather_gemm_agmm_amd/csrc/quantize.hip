// Block-scaled 8-bit quantiser (gfx950): the operands of the block-scaled
// product from bf16, fp16 or fp32 matrices.
//
//     s = max(max_{block} |x| / F, 2^-126)      (finite elements only)
//     q = rne8(x / s)                           F = 448 (e4m3), 57344 (e5m2)
//
// with one block per 128 consecutive elements of a row (block_rows 1) or per
// 128 x 128 tile (block_rows 128), of x, of x transposed, or of both from one
// read of x.  s is the correctly rounded fp32 quotient, q the format's value
// nearest to the real quotient x / s (the even one of two).  t = x * (1 / s) in
// fp32 is within 2 units of that, so only near the midpoint of two values can
// rounding t to 8 bits go wrong:
//  * 16-bit x (quotient16): F x / max is a ratio of short integers, so either
//    it is a midpoint or it lies 2^-20 or more (relative) from one.  Where it is
//    one, x / s lies on the side that the rounding of s took it to, for the
//    whole block, and 1 / s moved two units that way puts every such t on that
//    side and changes no other.  Where s is exact, one Newton step makes t
//    exact wherever x / s is an fp32 number, midpoints among them.  (Without
//    this about one bf16 element in 300 went to the wrong side.)
//  * fp32 x (exact8): a t within 4 units of a midpoint, about one in a
//    million, is decided by the sign of the exact remainder x - midpoint * s.
// |t| <= F (1 + 2^-20) rounds to at most F; non-finite elements do not enter
// a maximum and come out as NaN (e4m3) or as themselves (e5m2), never as a
// finite number.
//
// Bound: HBM.  Each element is read once and written once (twice for
// "both").  Measured: 8192 x 8192 bf16, rows and transposed rows, 52 us, 5.2
// TB/s read and written (a plain copy of 2 GiB reaches 5.0); 7168 x 8192 fp32
// in square blocks, both orders, 71 us, 5.0 TB/s; 128 x 4096 bf16 by rows 2.8
// us, a launch.
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

#include "ops_kernels.h"

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

typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));

// 8 consecutive elements of a row, as they are stored.  Sizes (the bits of
// |x|, which order like |x|) are kept two to a word for the 16-bit types.
template <int DT>
struct Eight {
  static constexpr bool kWide = DT == kDtypeFp32;
  static constexpr int W = kWide ? 8 : 4;
  uint32_t w[W];

  // from column c of a row; elements at or past `left` (columns that remain)
  // are zero.  Rows need element alignment only: 16-byte accesses to global
  // memory may start at any address.
  __device__ __forceinline__ void load(const char* row, int64_t c, int64_t left) {
    if (left >= 8) {
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const u32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any_t*>(row + c * (kWide ? 4 : 2)) + q);
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

// What dividing a block by its scale takes: the scale, its inverse (16-bit x:
// moved two units where s is not exact), and the factor of the Newton step (the
// inverse where s is exact, else 0).
struct Divisor {
  float s, inv, step;
};

template <int FMT, int DT>
__device__ __forceinline__ Divisor divisor(float size) {
  Divisor d;
  d.s = scale_of<FMT>(size);
  d.inv = 1.0f / d.s;
  d.step = 0.0f;
  if constexpr (DT != kDtypeFp32) {
    // the sign of s * F - max, exact; at the smallest scale the product with
    // its inverse, a power of two, is exact already
    const float off = __builtin_fmaf(d.s, top_value<FMT>(), -size);
    const int32_t move = d.s > kTinyScale ? (off > 0.0f ? -2 : off < 0.0f ? 2 : 0) : 0;
    d.step = move ? 0.0f : d.inv;
    d.inv = __builtin_bit_cast(float, __builtin_bit_cast(int32_t, d.inv) + move);
  }
  return d;
}

template <int FMT>
__device__ __forceinline__ float quotient16(float x, const Divisor& d) {
  const float t = x * d.inv, r = __builtin_fmaf(__builtin_fmaf(-t, d.s, x), d.step, t);
  // the step makes NaN of an infinity, which e5m2 keeps
  return FMT == kFmtE5M2 && !(__builtin_fabsf(t) < __builtin_inff()) ? t : r;
}

// How far the bits of t are from 4 units below a midpoint, in the upper bits.
template <int FMT>
__device__ __forceinline__ uint32_t beyond_midpoint(float t) {
  constexpr int kShift = FMT == kFmtE4M3 ? 12 : 11;   // the bits below the format's mantissa to the top
  return (__builtin_bit_cast(uint32_t, t) << kShift) + ((4u << kShift) - 0x80000000u);
}

// The same of the binade above the smallest normal value, whose spacing is
// that of everything below it.
template <int FMT>
__device__ __forceinline__ float low_binade(float size) {
  return size + (FMT == kFmtE4M3 ? 0.015625f : 6.103515625e-05f);
}

// Eight quotients by one divisor.  fp32: `near` tells whether one of them may
// be on the wrong side of a midpoint (then exact8 does it over).
template <int FMT, int DT, class X>
__device__ __forceinline__ u32x2_t pack8(X&& x, const Divisor& d, bool& near) {
  float t[8];
  if constexpr (DT != kDtypeFp32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = quotient16<FMT>(x(e), d);
  } else {
    uint32_t least = 0xFFFFFFFFu;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      t[e] = x(e) * d.inv;
      least = min(least, min(beyond_midpoint<FMT>(t[e]), beyond_midpoint<FMT>(low_binade<FMT>(__builtin_fabsf(t[e])))));
    }
    near = least <= (8u << (FMT == kFmtE4M3 ? 12 : 11));
  }
  return u32x2_t{pack4<FMT>(t[0], t[1], t[2], t[3]), pack4<FMT>(t[4], t[5], t[6], t[7])};
}

// fp32: up to eight elements `step` apart once more, each a byte, `out_step` apart.  Rare
// (about one group of eight in 10^5), so it reads them again and is not
// unrolled.
template <int FMT>
__device__ __forceinline__ void exact8(const float* x, int64_t step, int count, const Divisor& d, uint8_t* out, int out_step) {
  constexpr uint32_t kBelow = FMT == kFmtE4M3 ? 0xFFFFFu : 0x1FFFFFu;
#pragma unroll 1
  for (int e = 0; e < count; ++e) {
    const float v = x[e * step], t = v * d.inv, size = __builtin_fabsf(t);
    const bool low = size < low_binade<FMT>(0.0f);
    const float w = low ? low_binade<FMT>(size) : size;
    float r = t;
    if (beyond_midpoint<FMT>(w) <= (8u << (FMT == kFmtE4M3 ? 12 : 11)) && size < __builtin_inff()) {
      const float mid = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, w) & ~kBelow) | ((kBelow + 1) / 2)) -
                        (low ? low_binade<FMT>(0.0f) : 0.0f);
      const float rest = __builtin_fmaf(-mid, d.s, __builtin_fabsf(v));
      const uint32_t m = __builtin_bit_cast(uint32_t, mid);   // just above or below the midpoint, or on it
      r = __builtin_copysignf(rest == 0.0f ? mid : __builtin_bit_cast(float, rest > 0.0f ? m + 1 : m - 1), v);
    }
    out[e * out_step] = (uint8_t)pack4<FMT>(r, r, r, r);
  }
}

template <int DT, int FMT, int RPW>
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
    if (r0 + i < p.rows && left > 0) v[i].load(static_cast<const char*>(p.x) + (r0 + i) * p.ldx * ES, c, left);
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
    const Divisor d = divisor<FMT, DT>(size_value<DT>(one_size<DT>(max16<DT>(b))));
    if (r0 + i >= p.rows) break;
    if (c < p.cols16) {
      uint8_t* out = static_cast<uint8_t*>(p.q) + (r0 + i) * p.ldq + c;
      bool near = false;
      *reinterpret_cast<u32x2_t*>(out) = pack8<FMT, DT>([&](int e) { return v[i].value(e); }, d, near);
      if (DT == kDtypeFp32 && near && left > 0)
        exact8<FMT>(static_cast<const float*>(p.x) + (r0 + i) * p.ldx + c, 1, (int)min(left, (int64_t)8), d, out, 1);
    }
    if ((lane & 15) == 0 && left > 0) p.scale[(c >> 7) * p.rows + r0 + i] = d.s;
  }
}

// One 128 x 128 tile; p.q and p.qt either may be null.  A quotient costs as
// much as the rest of the work on an element, so each scale and its inverse
// are computed once per row (by one lane of 16, then broadcast) and once per
// column (by one thread, then read from LDS).
template <int DT, int FMT, bool SQUARE>
__global__ __launch_bounds__(256) void quantize_tile_kernel(QuantProblem p) {
  constexpr int ES = DT == kDtypeFp32 ? 4 : 2;
  using E = Eight<DT>;
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * 128];
  __shared__ __attribute__((aligned(16))) uint32_t cmax[4][16][E::W];   // column sizes: wave, 8-column piece, word
  __shared__ __attribute__((aligned(16))) float cs[128], cinv[128], cstep[128];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t kb = (p.cols + 127) / 128, rb = (p.rows + 127) / 128;
  const int64_t tb = blockIdx.x % (uint32_t)kb, tr = blockIdx.x / (uint32_t)kb;
  const int cl = tid & 15, rl = tid >> 4;                      // 8-column and 8-row piece of this thread
  const int64_t c0 = tb * 128 + cl * 8, r0 = tr * 128 + rl * 8;
  const int64_t left = p.cols - c0;
  E v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + i < p.rows && left > 0) v[i].load(static_cast<const char*>(p.x) + (r0 + i) * p.ldx * ES, c0, left);
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

  Divisor all{};               // SQUARE: of the tile
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
    all = divisor<FMT, DT>(size_value<DT>(one_size<DT>(b)));
    if (tid == 0) {
      if (p.q) p.scale[tb * rb + tr] = all.s;
      if (p.qt) p.scale_t[tr * kb + tb] = all.s;
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
      const Divisor d = divisor<FMT, DT>(size_value<DT>(b));
      cs[tid] = d.s;
      cinv[tid] = d.inv;
      cstep[tid] = d.step;
      if (tb * 128 + tid < p.cols) p.scale_t[tr * p.cols + tb * 128 + tid] = d.s;
    }
    __syncthreads();
  }

  // 8 rows of one column are 8 consecutive bytes of the transposed tile:
  // 8-byte piece rl of tile row c sits at piece rl ^ (c / 8).
  const auto piece = [&](int e) { return tile + (cl * 8 + e) * 128 + (rl ^ cl) * 8; };
  const auto row_out = [&](int i) { return static_cast<uint8_t*>(p.q) + (r0 + i) * p.ldq + c0; };
  const auto row_in = [&](int i) { return static_cast<const float*>(p.x) + (r0 + i) * p.ldx + c0; };
  const int count = (int)max((int64_t)0, min(left, (int64_t)8));   // columns of x in this piece
  if constexpr (SQUARE) {
    // one divisor, so one set of bytes, turned for the transposed output
    u32x2_t q[8];
    uint32_t near_rows = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bool near = false;
      q[i] = pack8<FMT, DT>([&](int e) { return v[i].value(e); }, all, near);
      near_rows |= (uint32_t)(near && r0 + i < p.rows) << i;
    }
    if (p.q && c0 < p.cols16)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r0 + i < p.rows) *reinterpret_cast<u32x2_t*>(row_out(i)) = q[i];
    if (p.qt)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint32_t col[2][4];   // of rows 0-3 and 4-7: 4 x 4 bytes turned by eight permutes
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a = q[4 * h][w], b = q[4 * h + 1][w], c = q[4 * h + 2][w], d = q[4 * h + 3][w];
          const uint32_t ab0 = __builtin_amdgcn_perm(b, a, 0x05010400), ab1 = __builtin_amdgcn_perm(b, a, 0x07030602);
          const uint32_t cd0 = __builtin_amdgcn_perm(d, c, 0x05010400), cd1 = __builtin_amdgcn_perm(d, c, 0x07030602);
          col[h][0] = __builtin_amdgcn_perm(cd0, ab0, 0x05040100);
          col[h][1] = __builtin_amdgcn_perm(cd0, ab0, 0x07060302);
          col[h][2] = __builtin_amdgcn_perm(cd1, ab1, 0x05040100);
          col[h][3] = __builtin_amdgcn_perm(cd1, ab1, 0x07060302);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<u32x2_t*>(piece(4 * w + e)) = u32x2_t{col[0][e], col[1][e]};
      }
    if constexpr (DT == kDtypeFp32)
      if (near_rows && count > 0)
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          if (!(near_rows >> i & 1)) continue;
          if (p.q) exact8<FMT>(row_in(i), 1, count, all, row_out(i), 1);
          if (p.qt) exact8<FMT>(row_in(i), 1, count, all, piece(0) + i, 128);
        }
  } else {
    if (p.q) {
      // lane cl of 16 takes row cl % 8: its size and divisor
      uint32_t size = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = one_size<DT>(max16<DT>(row[i]));
        size = (cl & 7) == i ? b : size;
      }
      const Divisor mine = divisor<FMT, DT>(size_value<DT>(size));
      if (cl < 8 && r0 + cl < p.rows) p.scale[tb * p.rows + r0 + cl] = mine.s;
      uint32_t near_rows = 0;
      const auto put = [&](auto row_tag) {
        constexpr int I = decltype(row_tag)::value;
        const Divisor d{row_lane<I>(mine.s), row_lane<I>(mine.inv), row_lane<I>(mine.step)};
        if (r0 + I < p.rows && c0 < p.cols16) {
          bool near = false;
          *reinterpret_cast<u32x2_t*>(row_out(I)) = pack8<FMT, DT>([&](int e) { return v[I].value(e); }, d, near);
          near_rows |= (uint32_t)near << I;
        }
      };
      put(Row<0>{});
      put(Row<1>{});
      put(Row<2>{});
      put(Row<3>{});
      put(Row<4>{});
      put(Row<5>{});
      put(Row<6>{});
      put(Row<7>{});
      if constexpr (DT == kDtypeFp32)
        if (__any(near_rows != 0 && count > 0))
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const int src = (lane & 48) + i;                   // the lane that holds row i's divisor
            const Divisor d{__shfl(mine.s, src), __shfl(mine.inv, src), 0.0f};
            if ((near_rows >> i & 1) && count > 0) exact8<FMT>(row_in(i), 1, count, d, row_out(i), 1);
          }
    }
    if (p.qt) {
      uint32_t near_cols = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const Divisor d{cs[cl * 8 + e], cinv[cl * 8 + e], cstep[cl * 8 + e]};
        bool near = false;
        *reinterpret_cast<u32x2_t*>(piece(e)) = pack8<FMT, DT>([&](int i) { return v[i].value(e); }, d, near);
        near_cols |= (uint32_t)near << e;
      }
      if constexpr (DT == kDtypeFp32)
        if (near_cols && r0 < p.rows)
#pragma unroll 1
          for (int e = 0; e < count; ++e) {
            if (!(near_cols >> e & 1)) continue;
            const Divisor d{cs[cl * 8 + e], cinv[cl * 8 + e], 0.0f};
            exact8<FMT>(row_in(0) + e, p.ldx, (int)min(p.rows - r0, (int64_t)8), d, piece(e), 1);
          }
    }
  }
  if (p.qt) {
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

template <int DT, int FMT>
hipError_t launch(const QuantProblem& p, hipStream_t stream) {
  if (p.block_rows == 1 && !p.qt) {
    const int64_t cw = (p.cols + 511) / 512;
    // 8 rows per wave where that still gives every CU several workgroups,
    // else 1: a small call is bound by latency, and more waves hide it.
    const bool deep = cw * ((p.rows + 31) / 32) >= 1024;
    const int64_t grid = cw * ((p.rows + (deep ? 32 : 4) - 1) / (deep ? 32 : 4));
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    if (deep) hipLaunchKernelGGL((quantize_rows_kernel<DT, FMT, 8>), dim3((unsigned)grid), dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((quantize_rows_kernel<DT, FMT, 1>), dim3((unsigned)grid), dim3(256), 0, stream, p);
  } else {
    const int64_t grid = ((p.cols + 127) / 128) * ((p.rows + 127) / 128);
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    if (p.block_rows == 1)
      hipLaunchKernelGGL((quantize_tile_kernel<DT, FMT, false>), dim3((unsigned)grid), dim3(256), 0, stream, p);
    else
      hipLaunchKernelGGL((quantize_tile_kernel<DT, FMT, true>), dim3((unsigned)grid), dim3(256), 0, stream, p);
  }
  return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const QuantProblem& p, hipStream_t s) {
  return p.format == kFmtE4M3 ? launch<DT, kFmtE4M3>(p, s) : launch<DT, kFmtE5M2>(p, s);
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
