// Device code shared by the feed-forward block's kernels: activations, 8-bit
// pre-activations, and accesses to rows of any alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "feed_kernels.h"
#include "gemm_device.h"

namespace agmm {

namespace {

// Vectors in global memory that need element alignment only.
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
typedef u32x2_t u32x2_any_t __attribute__((aligned(2)));

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// The normal distribution function.  With z = |x| / sqrt 2 the smaller tail is
// erfc(z) / 2 = exp(-z^2) erfcx(z) / 2; erfcx, which is smooth and between 1
// and 1 / (z sqrt pi), is fitted as t * polynomial(t), t = 1 / (1 + 0.38 z)
// (least relative error over 0 <= z <= 10: 1.0e-6, in fp32 1.3e-6; the results
// are rounded to 16 bits, 2^-11 at best).  So both tails keep their relative
// precision, which 1 + erf does not.  Beyond |x| = 13.2 exp(-z^2) is 0.
__device__ __forceinline__ float normal_share(float x) {
  const float z = __builtin_fabsf(x);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(z, 0.26870057685088806f, 1.0f));
  float q = -0.5f * 0.12520186603069305f;
  q = __builtin_fmaf(q, t, 0.5f * 0.33520618081092834f);
  q = __builtin_fmaf(q, t, 0.5f * -0.0686253011226654f);
  q = __builtin_fmaf(q, t, 0.5f * 0.2468075305223465f);
  q = __builtin_fmaf(q, t, 0.5f * 0.1810360699892044f);
  q = __builtin_fmaf(q, t, 0.5f * 0.21648065745830536f);
  q = __builtin_fmaf(q, t, 0.5f * 0.21429570019245148f);
  q = q * t * __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2e));
  return x >= 0.0f ? 1.0f - q : q;
}

// x is cut in the cubic term, where it may be infinite.
__device__ __forceinline__ float logistic_share(float x, float c1, float c3) {
  const float q = fminf(__builtin_fabsf(x), 1e9f);
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * __builtin_fmaf(c3 * kLog2e * q, q, c1 * kLog2e)));
}
__device__ __forceinline__ float silu_share(float x) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -kLog2e)); }

// act(x).  A NaN stays one in every kind; the limits at -infinity are those of
// the arithmetic (x times a share of 0: NaN), as for the formula in IEEE numbers.
template <int KIND>
__device__ __forceinline__ float act_value(float x, float c1, float c3) {
  if constexpr (KIND == kActSilu) return x * silu_share(x);
  else if constexpr (KIND == kActLogistic) return x * logistic_share(x, c1, c3);
  else if constexpr (KIND == kActNormal) return x * normal_share(x);
  else if constexpr (KIND == kActRelu) return x < 0.0f ? 0.0f : x;
  else return x;
}

// act(x) and its derivative.  The derivative's second term vanishes beyond 128
// in every kind, so x is cut there: its limits at the infinities are 0 and 1.
template <int KIND>
__device__ __forceinline__ void act_both(float x, float c1, float c3, float& value, float& slope) {
  const float near = fminf(fmaxf(x, -128.0f), 128.0f);
  if constexpr (KIND == kActSilu) {
    const float s = silu_share(x);
    value = x * s;
    slope = __builtin_fmaf(near * s, 1.0f - s, s);
  } else if constexpr (KIND == kActLogistic) {
    const float s = logistic_share(x, c1, c3);
    value = x * s;
    slope = __builtin_fmaf(near * s, (1.0f - s) * __builtin_fmaf(3.0f * c3 * near, near, c1), s);
  } else if constexpr (KIND == kActNormal) {
    const float s = normal_share(x);
    value = x * s;
    slope = __builtin_fmaf(near * 0.3989422804014327f, exp_of(-0.5f * x * x), s);
  } else if constexpr (KIND == kActRelu) {
    value = x < 0.0f ? 0.0f : x;
    slope = x > 0.0f ? 1.0f : x == x ? 0.0f : x;
  } else {
    value = x;
    slope = 1.0f;
  }
}

// Biased exponent of the smallest power of two s >= 2^-126 with size <= 448 s
// (448 = 1.75 * 2^8 is e4m3's largest value), for finite size >= 0: that of
// size, less 8, and one more where its fraction is above 1.75.
__device__ __forceinline__ uint32_t scale_code(float size) {
  const int e = (int)((__builtin_bit_cast(uint32_t, size) + 0x001FFFFFu) >> 23) - 8;
  return (uint32_t)(e > 1 ? e : 1);
}
__device__ __forceinline__ float scale_value(uint32_t code) { return __builtin_bit_cast(float, code << 23); }
// 1 / s, exact: s is between 2^-126 and 2^120.
__device__ __forceinline__ float scale_inverse(uint32_t code) { return __builtin_bit_cast(float, (254u - code) << 23); }

// The largest finite |x| so far.
__device__ __forceinline__ float larger_finite(float size, float x) {
  x = __builtin_fabsf(x);
  return x < __builtin_inff() ? fmaxf(size, x) : size;
}

// Four values over their scale as e4m3, rounded once to nearest even (the
// products are exact but for results below fp32's normal range, which are 0 in
// e4m3 either way).  An infinity becomes NaN, which is all that e4m3 has.
__device__ __forceinline__ uint32_t pack4_e4m3(float a, float b, float c, float d, float inv) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
  return (uint32_t)w;
}

// 16-bit storage to fp32.
template <int DT>
__device__ __forceinline__ float value16(uint32_t bits) {
  if constexpr (DT == kDtypeBf16) return __builtin_bit_cast(float, bits << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}
template <int DT>
__device__ __forceinline__ float low16(uint32_t w) {
  if constexpr (DT == kDtypeBf16) return __builtin_bit_cast(float, w << 16);
  else return value16<DT>(w & 0xFFFFu);
}
template <int DT>
__device__ __forceinline__ float high16(uint32_t w) {
  if constexpr (DT == kDtypeBf16) return __builtin_bit_cast(float, w & 0xFFFF0000u);
  else return value16<DT>(w >> 16);
}

// Eight 16-bit elements of a row of any alignment, zeros past `left` of them.
__device__ __forceinline__ u32x4_t load8(const uint16_t* x, int left) {
  if (left >= 8) return *reinterpret_cast<const u32x4_any_t*>(x);
  u32x4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) v[e >> 1] |= (uint32_t)x[e] << (16 * (e & 1));
  return v;
}
__device__ __forceinline__ void store8(uint16_t* x, u32x4_t v, int left) {
  if (left >= 8) {
    *reinterpret_cast<u32x4_any_t*>(x) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) x[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
  }
}
__device__ __forceinline__ void store4(uint16_t* x, u32x2_t v, int left) {
  if (left >= 4) {
    *reinterpret_cast<u32x2_any_t*>(x) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) x[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
  }
}
// Four 16-bit elements as fp32, zeros past `left`.
template <int DT>
__device__ __forceinline__ f32x4_t load4(const uint16_t* x, int left) {
  u32x2_t v = {0u, 0u};
  if (left >= 4) {
    v = *reinterpret_cast<const u32x2_any_t*>(x);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) v[e >> 1] |= (uint32_t)x[e] << (16 * (e & 1));
  }
  return f32x4_t{low16<DT>(v[0]), high16<DT>(v[0]), low16<DT>(v[1]), high16<DT>(v[1])};
}

// Calls f with the activation's kind as a constant.
template <class F>
__device__ __forceinline__ void with_kind(int kind, F&& f) {
  if (kind == kActSilu) f(IntTag<kActSilu>{});
  else if (kind == kActLogistic) f(IntTag<kActLogistic>{});
  else if (kind == kActNormal) f(IntTag<kActNormal>{});
  else if (kind == kActRelu) f(IntTag<kActRelu>{});
  else f(IntTag<kActLinear>{});
}

// Eight columns of a row of the product, bias added: what is kept of them, and
// y.  Four neighbouring lanes hold the 32 columns from `col` rounded down on,
// and all of them come here together.
template <int DT, bool GATED, int KIND>
__device__ __forceinline__ void finish8(const FeedProblem& fp, const float (&v)[GATED ? 2 : 1][8], int64_t row, bool in, int col) {
  constexpr int PARTS = GATED ? 2 : 1;
  const int left = fp.n - col;
  const int64_t wide = fp.kept.wide;
  if (fp.kept.values && col < wide) {
#pragma unroll
    for (int h = 0; h < PARTS; ++h) {
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = v[h][e];
      if (left < 8)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e >= left) w[e] = 0.0f;
      const int64_t out = (row * PARTS + h) * wide + col;
      if (!fp.kept.scales) {
        if (in)
          *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(fp.kept.values) + out) =
              u32x4_t{pack2<DT>(w[0], w[1]), pack2<DT>(w[2], w[3]), pack2<DT>(w[4], w[5]), pack2<DT>(w[6], w[7])};
      } else {
        // the maximum passes over NaN; an infinite one is taken anew
        float size = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) size = fmaxf(size, __builtin_fabsf(w[e]));
        if (size == __builtin_inff()) {
          size = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) size = larger_finite(size, w[e]);
        }
        size = fmaxf(size, __shfl_xor(size, 1));
        size = fmaxf(size, __shfl_xor(size, 2));
        const uint32_t code = scale_code(size);
        const float inv = scale_inverse(code);
        if (in) {
          *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(fp.kept.values) + out) =
              u32x2_t{pack4_e4m3(w[0], w[1], w[2], w[3], inv), pack4_e4m3(w[4], w[5], w[6], w[7], inv)};
          if (col % kKeptBlock == 0) fp.kept.scales[out / kKeptBlock] = (uint8_t)code;
        }
      }
    }
  }
  if (!in || left <= 0) return;
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    y[e] = act_value<KIND>(v[0][e], fp.act.c1, fp.act.c3);
    if constexpr (GATED) y[e] *= v[1][e];
  }
  if (!GATED && fp.residual) {
    const u32x4_t b = load8(static_cast<const uint16_t*>(fp.residual) + row * fp.ldr + col, left);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] += e & 1 ? high16<DT>(b[e >> 1]) : low16<DT>(b[e >> 1]);
  }
  store8(static_cast<uint16_t*>(fp.y) + row * fp.ldy + col,
         u32x4_t{pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3]), pack2<DT>(y[4], y[5]), pack2<DT>(y[6], y[7])}, left);
}

// The bias of eight columns of each part, zeros where there is none.
template <int DT, bool GATED>
__device__ __forceinline__ void bias8(const FeedProblem& fp, int col, float (&bias)[GATED ? 2 : 1][8]) {
  const int left = fp.n - col;
#pragma unroll
  for (int h = 0; h < (GATED ? 2 : 1); ++h) {
    u32x4_t b = {0u, 0u, 0u, 0u};
    if (fp.bias && left > 0) b = load8(static_cast<const uint16_t*>(fp.bias) + (int64_t)h * fp.n + col, left);
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[h][e] = e & 1 ? high16<DT>(b[e >> 1]) : low16<DT>(b[e >> 1]);
  }
}

}  // namespace

}  // namespace agmm
