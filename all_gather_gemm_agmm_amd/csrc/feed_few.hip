// Product with an epilogue, and the gated product: few rows (gfx950).
//
// 16 FM rows x YC columns of y per workgroup, whose waves share out k, 64
// elements at a time, and load their operands straight into registers: 16-byte
// accesses to global memory may start at any word, which loads into LDS may not,
// so k and the strides may be anything and nothing is copied first.  The waves' sums are added in LDS in a fixed order, wave w
// taking row block w, and bias, activation, product, residual and rounding
// follow there (feed_tiles.hip says how).  Gated, blocks of 16 rows of the
// first n rows of B and of the second n take turns.  Where the blocks leave CUs
// idle and k is long, it is cut into ranges as well, whose fp32 sums a second
// launch adds in order and finishes (63 x 3814 -> 2 x 381: 20 us in one launch,
// 12 so; 128 x 2834 -> 2 x 252: 15 and 11; 8 x 1001 -> 700 is faster in one, 5).
//
// ODD (a stride is odd): rows that start in the middle of a word are read from
// that word on, with one word more, and shifted; accesses that start there take
// three times as long.
//
// Bound: what a CU streams in, 22 bytes a cycle, its columns of W and the rows
// of A again per workgroup, and a launch.  Blocks of 8 columns fill the CUs of a
// short y.  Measured (us, calls back to back in a graph): 8 x 4096 -> 1792 bf16 7.8
// (8.4 under a profiler), of which W at 4.5 TB/s is 3.3; gated, twice the W, 9.4;
// 8 x 8192 -> 3584 16; 128 x 4096 -> 7168 35, where tiles of 128 take 22 and are
// chosen.
#include "feed_device.h"

namespace agmm {

namespace {

// YC: columns of y per workgroup.  FN = 1 with YC = 8 fills twice the CUs of a
// short y: plain, both halves of the block read the same 8 rows of B (the same
// cache lines); gated, its halves are 8 rows of each part.
template <int DT, int FM, int YC, int UN, int WAVES, bool ODD, bool GATED>
__global__ __launch_bounds__(64 * WAVES) void feed_few_kernel(FeedProblem fp) {
  const GemmProblem& p = fp.gemm;
  constexpr int PARTS = GATED ? 2 : 1;
  constexpr bool HALF = YC == 8;
  constexpr int FN = HALF ? 1 : YC / 16 * PARTS, FQ = HALF ? 1 : YC / 16;
  __shared__ float part[WAVES][FM][FN][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g4 = lane >> 4, i16 = lane & 15;
  const int blocks = p.order.num_rb * p.order.num_cb, range = (int)blockIdx.x / blocks, id = (int)blockIdx.x - range * blocks;
  const int cb = id / p.order.num_rb, rb = id - cb * p.order.num_rb;
  const bool whole = p.splits == 1;            // not one of several ranges of k
  const int k0 = range * p.k_per_split;
  const int M = p.m, NC = fp.n, K = min(p.k - k0, p.k_per_split);
  const int m0 = rb * 16 * FM, y0 = cb * YC;
  // rows and columns past the end read the last one and are never used
  const uint16_t *a[FM], *b[FN];
  if constexpr (FM == 1) {
    // the shards' addresses of up to 16 rows by scalar loads and a choice per
    // lane: a load per lane from the kernel's arguments, on whose result the
    // rows' own loads wait, takes as long as those
    const int rpg = p.rows.rows_per_group, i = min(m0 + i16, M - 1), g = i / rpg, first = m0 / rpg;
    const void* base = p.rows.a_group[first];
#pragma unroll
    for (int q = 1; q < 16; ++q) {
      const void* other = p.rows.a_group[min(first + q, p.rows.num_groups - 1)];
      if (g == first + q) base = other;
    }
    a[0] = static_cast<const uint16_t*>(base) + (int64_t)(i - g * rpg) * p.rows.a_ld + k0 + 8 * g4;
  } else {
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      const int i = min(m0 + 16 * f + i16, M - 1), g = i / p.rows.rows_per_group;
      a[f] = static_cast<const uint16_t*>(p.rows.a_group[g]) + (int64_t)(i - g * p.rows.rows_per_group) * p.rows.a_ld + k0 + 8 * g4;
    }
  }
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    const int h = HALF ? (GATED ? i16 >> 3 : 0) : f % PARTS, c = HALF ? i16 & 7 : 16 * (f / PARTS) + i16;
    b[f] = static_cast<const uint16_t*>(p.b) + k0 + 8 * g4 + ((int64_t)h * NC + min(y0 + c, NC - 1)) * p.ldb;
  }

  // what the epilogue adds, on its way early
  f32x4_t bias[FN], res[FQ];
  const int row = m0 + 16 * wave + i16;       // wave w ends with row block w
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int h = HALF ? (GATED ? g4 >> 1 : 0) : j % PARTS, c = y0 + (HALF ? 4 * (g4 & 1) : 16 * (j / PARTS) + 4 * g4);
    bias[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (fp.bias && whole && wave < FM) bias[j] = load4<DT>(static_cast<const uint16_t*>(fp.bias) + (int64_t)h * NC + c, NC - c);
  }
#pragma unroll
  for (int q = 0; q < FQ; ++q) {
    const int c = y0 + (HALF ? 4 * (g4 & 1) : 16 * q + 4 * g4);
    res[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (!GATED && fp.residual && whole && wave < FM && row < M)
      res[q] = load4<DT>(static_cast<const uint16_t*>(fp.residual) + (int64_t)row * fp.ldr + c, NC - c);
  }

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const auto multiply = [&](const u32x4_t (&fa)[FM], const u32x4_t (&fb)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = mfma16_builtin<DT>(fb[j], fa[i], acc[i][j]);
  };
  // halves 2u, 2u + 1 of piece c + u: elements 64 (c + u) + 32 h + 8 g4 on;
  // ODD: their words and the one behind
  constexpr int W = ODD ? 2 * UN : 1;
  typedef u32x4_t u32x4_word_t __attribute__((aligned(4)));
  const auto load = [&](int c, u32x4_t (&fa)[2 * UN][FM], u32x4_t (&fb)[2 * UN][FN], uint32_t (&wa)[W][FM], uint32_t (&wb)[W][FN]) {
    const auto one = [&](const uint16_t* x, u32x4_t& v, uint32_t& w) {
      if constexpr (ODD) {
        const char* q = reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(x) & ~uintptr_t(2));
        v = *reinterpret_cast<const u32x4_word_t*>(q);
        w = *reinterpret_cast<const uint32_t*>(q + 16);
      } else {
        v = *reinterpret_cast<const u32x4_word_t*>(x);
      }
    };
    // B first: it comes from furthest.  Lanes without a row of their own load
    // nothing (the way into a CU is what bounds 8 rows); what they hold reaches
    // no result that is used.
    if (!HALF || GATED || i16 < 8) {
#pragma unroll
      for (int h = 0; h < 2 * UN; ++h)
#pragma unroll
        for (int j = 0; j < FN; ++j) one(b[j] + (int64_t)c * 64 + 32 * h, fb[h][j], wb[ODD ? h : 0][j]);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FM; ++i)
      if (16 * i + i16 < M - m0)
#pragma unroll
        for (int h = 0; h < 2 * UN; ++h) one(a[i] + (int64_t)c * 64 + 32 * h, fa[h][i], wa[ODD ? h : 0][i]);
  };
  const auto shift = [&](const uint16_t* x, u32x4_t& v, uint32_t w) {
    const uint32_t by = (uint32_t)reinterpret_cast<uintptr_t>(x) & 2;
    v = u32x4_t{__builtin_amdgcn_alignbyte(v[1], v[0], by), __builtin_amdgcn_alignbyte(v[2], v[1], by),
                __builtin_amdgcn_alignbyte(v[3], v[2], by), __builtin_amdgcn_alignbyte(w, v[3], by)};
  };
  const auto use = [&](u32x4_t (&fa)[2 * UN][FM], u32x4_t (&fb)[2 * UN][FN], const uint32_t (&wa)[W][FM], const uint32_t (&wb)[W][FN]) {
#pragma unroll
    for (int h = 0; h < 2 * UN; ++h) {
      if constexpr (ODD) {
#pragma unroll
        for (int j = 0; j < FN; ++j) shift(b[j], fb[h][j], wb[h][j]);
#pragma unroll
        for (int i = 0; i < FM; ++i) shift(a[i], fa[h][i], wa[h][i]);
      }
      multiply(fa[h], fb[h]);
    }
  };
  const int pieces = (ODD ? max(K - 2, 0) : K) / 64, groups = pieces / UN;   // the word behind lies in the row
  u32x4_t fa[2][2 * UN][FM] = {}, fb[2][2 * UN][FN] = {};
  uint32_t wa[2][W][FM] = {}, wb[2][W][FN] = {};
  // workgroups begin at different places of k, so that they do not ask the same
  // memory channel for rows a power of two apart all at once (8 x 4096 -> 2 x
  // 7168: 29 -> 24 us)
  const int rot = groups > 1 ? (int)((blockIdx.x * 7u) % (unsigned)groups) : 0;
  const auto piece_of = [&](int c) { return (c + rot >= groups ? c + rot - groups : c + rot) * UN; };
  if (wave < groups) load(piece_of(wave), fa[0], fb[0], wa[0], wb[0]);
  for (int c = wave; c < groups; c += 2 * WAVES) {
    // two groups per turn; all of a group's loads are issued before the other's
    // products
    if (c + WAVES < groups) load(piece_of(c + WAVES), fa[1], fb[1], wa[1], wb[1]);
    __builtin_amdgcn_sched_barrier(0);
    use(fa[0], fb[0], wa[0], wb[0]);
    if (c + WAVES >= groups) break;
    if (c + 2 * WAVES < groups) load(piece_of(c + 2 * WAVES), fa[0], fb[0], wa[0], wb[0]);
    __builtin_amdgcn_sched_barrier(0);
    use(fa[1], fb[1], wa[1], wb[1]);
  }
  // what is left: halves of 32 elements, shared out over the waves, those
  // past k elementwise and zero
  for (int at = groups * UN * 64 + 32 * wave; at < K; at += 32 * WAVES) {
    u32x4_t ta[FM], tb[FN];
    const int left = K - at - 8 * g4;
#pragma unroll
    for (int j = 0; j < FN; ++j) tb[j] = load8(b[j] + at, left);
#pragma unroll
    for (int i = 0; i < FM; ++i) ta[i] = load8(a[i] + at, left);
    multiply(ta, tb);
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[wave][i][j][e][lane] = acc[i][j][e];
  __syncthreads();
  if (wave >= FM) return;
  const bool in = row < M;
  float x[FN][4];
#pragma unroll
  for (int j = 0; j < FN; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float t = part[0][wave][j][e][lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) t += part[w][wave][j][e][lane];
      x[j][e] = t + bias[j][e];
    }
  }
  if (!HALF && !whole) {
    // fp32 sums [range][m][tile columns rounded up to 16] for launch_feed_join
    const int64_t ld = (p.n + 15) & ~15;
    float* out = p.partials + ((int64_t)range * M + row) * ld + PARTS * y0 + 4 * g4;
    if (in)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        if (PARTS * y0 + 16 * j < ld) *reinterpret_cast<f32x4_t*>(out + 16 * j) = f32x4_t{x[j][0], x[j][1], x[j][2], x[j][3]};
    return;
  }
  if (YC >= kKeptBlock && fp.kept.values) {
    const int64_t wide = fp.kept.wide;
    // blocks of 32 columns of a part: two accumulator blocks 
#pragma unroll
    for (int h = 0; h < PARTS; ++h)
#pragma unroll
      for (int q = 0; q + 1 < FQ; q += 2) {
        float w[2][4], size = 0.0f;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[s][e] = y0 + 16 * (q + s) + 4 * g4 + e < NC ? x[PARTS * (q + s) + h][e] : 0.0f;
            size = larger_finite(size, w[s][e]);
          }
        size = fmaxf(size, __shfl_xor(size, 16));
        size = fmaxf(size, __shfl_xor(size, 32));
        const uint32_t code = scale_code(size);
        const float inv = scale_inverse(code);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int c = y0 + 16 * (q + s) + 4 * g4;
          const int64_t out = ((int64_t)row * PARTS + h) * wide + c;
          if (!in || c >= wide) continue;
          if (fp.kept.scales)
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(fp.kept.values) + out) =
                pack4_e4m3(w[s][0], w[s][1], w[s][2], w[s][3], inv);
          else
            *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(fp.kept.values) + out) =
                u32x2_t{pack2<DT>(w[s][0], w[s][1]), pack2<DT>(w[s][2], w[s][3])};
          if (fp.kept.scales && s == 0 && g4 == 0) fp.kept.scales[out / kKeptBlock] = (uint8_t)code;
        }
      }
  }
  float factor[4];   // YC 8: the second part's, from the lane that holds it
  if constexpr (HALF && GATED)
#pragma unroll
    for (int e = 0; e < 4; ++e) factor[e] = __shfl_xor(x[0][e], 32);
  if (!in || (HALF && g4 >= 2)) return;
  with_kind(fp.act.kind, [&](auto kind) {
    constexpr int KIND = decltype(kind)::value;
#pragma unroll
    for (int q = 0; q < FQ; ++q) {
      const int c = y0 + 16 * q + 4 * g4, left = NC - c;
      if (left <= 0) continue;
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[e] = act_value<KIND>(x[HALF ? 0 : PARTS * q][e], fp.act.c1, fp.act.c3);
        if constexpr (GATED) y[e] *= HALF ? factor[e] : x[HALF ? 0 : PARTS * q + PARTS - 1][e];
      }
      if (!GATED && fp.residual)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += res[q][e];
      store4(static_cast<uint16_t*>(fp.y) + (int64_t)row * fp.ldy + c, u32x2_t{pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3])}, left);
    }
  });
}

template <int DT, int FM, int YC, int UN, int WAVES, bool GATED>
void launch_shape(const FeedProblem& p, unsigned grid, hipStream_t s) {
  const bool odd = p.gemm.ldb % 2 != 0 || p.gemm.rows.a_ld % 2 != 0;
  if (odd) hipLaunchKernelGGL((feed_few_kernel<DT, FM, YC, UN, WAVES, true, GATED>), dim3(grid), dim3(64 * WAVES), 0, s, p);
  else hipLaunchKernelGGL((feed_few_kernel<DT, FM, YC, UN, WAVES, false, GATED>), dim3(grid), dim3(64 * WAVES), 0, s, p);
}

template <int DT>
hipError_t launch_type(const FeedProblem& p, int fm, int yc, unsigned grid, hipStream_t s) {
  if (p.gated) {
    if (fm == 1 && yc == 8) launch_shape<DT, 1, 8, 4, 8, true>(p, grid, s);
    else if (fm == 1 && yc == 16) launch_shape<DT, 1, 16, 2, 8, true>(p, grid, s);
    else if (fm == 1) launch_shape<DT, 1, 32, 2, 4, true>(p, grid, s);
    else if (yc == 16) launch_shape<DT, 4, 16, 1, 4, true>(p, grid, s);
    else launch_shape<DT, 4, 32, 1, 4, true>(p, grid, s);
  } else {
    if (fm == 1 && yc == 8) launch_shape<DT, 1, 8, 4, 8, false>(p, grid, s);
    else if (fm == 1 && yc == 16) launch_shape<DT, 1, 16, 4, 8, false>(p, grid, s);
    else if (fm == 1) launch_shape<DT, 1, 64, 2, 4, false>(p, grid, s);
    else if (yc == 16) launch_shape<DT, 4, 16, 2, 4, false>(p, grid, s);
    else launch_shape<DT, 4, 64, 1, 4, false>(p, grid, s);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_feed_few(const FeedProblem& p, int fm, int yc, int dtype, hipStream_t stream) {
  const GemmProblem& g = p.gemm;
  const int64_t grid = (int64_t)g.order.num_rb * g.order.num_cb * g.splits;
  const int most = p.gated ? 32 : 64;
  if ((fm != 1 && fm != 4) || (yc != 8 && yc != 16 && yc != most) || (yc == 8 && fm != 1) || (p.gated && p.residual) ||
      p.gemm.order.num_rb != (p.gemm.m + 16 * fm - 1) / (16 * fm) || p.gemm.order.num_cb != (p.n + (int64_t)yc - 1) / yc ||
      grid < 1 || grid >= kFeedGrid || (int64_t)p.gemm.rows.num_groups * p.gemm.rows.rows_per_group != p.gemm.m ||
      g.splits < 1 || (g.splits == 1 && g.k_per_split < g.k) ||
      (g.splits > 1 && (yc == 8 || !g.partials || g.k_per_split % 64 != 0 || (int64_t)g.splits * g.k_per_split < g.k ||
                        (int64_t)(g.splits - 1) * g.k_per_split >= g.k ||
                        g.n != (p.gated ? 2 * (((int64_t)p.n + 15) / 16 * 16) : p.n))) ||
      (p.kept.values && ((g.splits == 1 && yc != most) || p.kept.wide != ((int64_t)p.n + kKeptBlock - 1) / kKeptBlock * kKeptBlock)))
    return hipErrorInvalidValue;
  const hipError_t err = dtype == kDtypeBf16 ? launch_type<kDtypeBf16>(p, fm, yc, (unsigned)grid, stream)
                       : dtype == kDtypeFp16 ? launch_type<kDtypeFp16>(p, fm, yc, (unsigned)grid, stream) : hipErrorInvalidValue;
  return err == hipSuccess && g.splits > 1 ? launch_feed_join(p, dtype, stream) : err;
}

}  // namespace agmm
