// The way back through the product with an epilogue and the gated product,
// elementwise part (gfx950):
//
//     d = dy act'(p)     or, gated,     d_0 = dy p_1 act'(p_0),  d_1 = dy act(p_0)
//
// from the kept pre-activations, as 16-bit operands of the two gradient
// products, by rows [m][parts * n] for dA = d W and transposed [parts * n][m]
// for dW = d^T A, and the column sums of d for the bias.  A workgroup takes 128
// (few: 32) rows x 64 columns of y: 16-byte pieces of rows in, d by rows out of the same
// registers, and through LDS and transposing reads out again by columns.  Bound:
// HBM, every value read once and d written twice (that the matrix cores can
// read both operands along k).  d is rounded to the operands' type, as every
// other operand of these products is; its sums are taken before that, in fp32.
//
// Measured: 8192 x 2 x 3584 bf16 from 8 bits 76-80 us, 355 MB at 4.5 TB/s; 2048 x
// 1024 bf16, tanh's gelu 6.4, in blocks of 32 rows, so that there are enough; 111 x
// 2 x 2051 fp16, with the copies that the products need, 6.3.  y again (recompute),
// 8192 x 2 x 3584 bf16: 22 us from 8 bits, 30 from 16, 119 and 176 MB.
//
// What is read again as fp32 sums over ranges of k, or over blocks of rows, is
// added in a fixed order.
#include "feed_device.h"

namespace agmm {

namespace {

// Eight kept pre-activations of one part.
template <int DT>
__device__ __forceinline__ void kept8(const KeptRows& k, int64_t at, float (&v)[8]) {
  if (k.scales) {
    const u32x2_t q = *reinterpret_cast<const u32x2_t*>(static_cast<const uint8_t*>(k.values) + at);
    const float s = scale_value(k.scales[at / kKeptBlock]);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      v[4 * w + 0] = __builtin_amdgcn_cvt_f32_fp8((int)q[w], 0) * s;
      v[4 * w + 1] = __builtin_amdgcn_cvt_f32_fp8((int)q[w], 1) * s;
      v[4 * w + 2] = __builtin_amdgcn_cvt_f32_fp8((int)q[w], 2) * s;
      v[4 * w + 3] = __builtin_amdgcn_cvt_f32_fp8((int)q[w], 3) * s;
    }
  } else {
    const u32x4_t q = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(k.values) + at);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e & 1 ? high16<DT>(q[e >> 1]) : low16<DT>(q[e >> 1]);
  }
}

template <int DT>
__device__ __forceinline__ void unpack8(u32x4_t q, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e & 1 ? high16<DT>(q[e >> 1]) : low16<DT>(q[e >> 1]);
}
template <int DT>
__device__ __forceinline__ u32x4_t pack8(const float (&v)[8]) {
  return u32x4_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
}

// One thread's share of a copy: every `step`-th 16-byte piece of its output.
__device__ __forceinline__ void copy_rows(const PadRows& c, int64_t first, int64_t step) {
  const int64_t all = c.num_groups * c.rows * c.chunks;
  const auto from = [&](int64_t u, int64_t& row, int& col) {
    row = u / (uint32_t)c.chunks;
    col = (int)(u - row * c.chunks) * 8;
    const int64_t g = row / (uint32_t)c.rows;
    return static_cast<const uint16_t*>(c.group[g]) + (row - g * c.rows) * c.ld + col;
  };
#pragma unroll 1
  for (int64_t u = first; u < all; u += 4 * step) {
    u32x4_t v[4];                              // on their way together
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      int64_t row;
      int col;
      if (u + q * step < all) {
        const uint16_t* x = from(u + q * step, row, col);
        v[q] = load8(x, (int)c.cols - col);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (u + q * step < all) *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(c.out) + (u + q * step) * 8) = v[q];
  }
}

// Workgroups of 256 of a copy: 16 KiB each, as many as fill the chip.
int64_t copy_groups(const PadRows& c) {
  const int64_t pieces = c.num_groups * c.rows * c.chunks, want = (pieces + 1023) / 1024;
  return want < 8192 ? want : 8192;
}

__device__ __forceinline__ void copy_block(const FeedCopies& c, int64_t block, int64_t a_groups, int64_t w_groups) {
  const bool w = block >= a_groups;
  const int64_t step = (w ? w_groups : a_groups) * 256;
  copy_rows(w ? c.w : c.a, (w ? block - a_groups : block) * 256 + threadIdx.x, step);
}

__global__ __launch_bounds__(256) void feed_copies_kernel(FeedCopies c, int32_t a_groups, int32_t w_groups) {
  copy_block(c, blockIdx.x, a_groups, w_groups);
}

// What a thread loads of a row: eight columns of dy and of the parts kept.
template <bool GATED>
struct RawRow {
  u32x4_t dy, p[GATED ? 2 : 1];
  uint32_t code[GATED ? 2 : 1];
};

// ROWS rows x 64 columns of y per workgroup: 128, or 32 where that leaves CUs
// idle.  The loop over a thread's rows is not unrolled: a small launch waits for
// its instructions (111 x 2051 gated took 12.6 us unrolled), a large one has
// enough other waves; the next row's loads are on their way meanwhile.
template <int DT, bool GATED, int ROWS>
__global__ __launch_bounds__(256) void feed_d_kernel(FeedDProblem p, FeedCopies copies, int32_t blocks, int32_t a_groups, int32_t w_groups) {
  if ((int)blockIdx.x >= blocks) {
    copy_block(copies, (int)blockIdx.x - blocks, a_groups, w_groups);
    return;
  }
  constexpr int PARTS = GATED ? 2 : 1, RB = kDCols * 2, CH = RB / 16;
  __shared__ __attribute__((aligned(1024))) char smem[PARTS * ROWS * RB];
  __shared__ float sums[4][PARTS][kDCols];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int ncb = (p.n + kDCols - 1) / kDCols;
  const int64_t rb = blockIdx.x / (unsigned)ncb;
  const int cb = (int)(blockIdx.x - rb * ncb);
  const int64_t m0 = rb * ROWS;
  const int c = tid & 7, col = cb * kDCols + 8 * c, left = p.n - col;
  const int kind = p.act.kind;
  const bool need_p = kind != kActLinear || GATED, bytes = p.kept.scales != nullptr;
  const float c1 = p.act.c1, c3 = p.act.c3;
  float total[PARTS][8] = {};
  const auto load = [&](int r, RawRow<GATED>& x) {
    const int64_t row = m0 + r;
    if (row >= p.m || left <= 0) return;
    x.dy = load8(static_cast<const uint16_t*>(p.dy) + row * p.lddy + col, left);
    if (!need_p) return;
#pragma unroll
    for (int h = 0; h < PARTS; ++h) {
      const int64_t at = (row * PARTS + h) * p.kept.wide + col;
      if (bytes) {
        const u32x2_t q = *reinterpret_cast<const u32x2_t*>(static_cast<const uint8_t*>(p.kept.values) + at);
        x.p[h][0] = q[0];
        x.p[h][1] = q[1];
        x.code[h] = p.kept.scales[at / kKeptBlock];
      } else {
        x.p[h] = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p.kept.values) + at);
      }
    }
  };
  const auto values = [&](const RawRow<GATED>& x, int h, float (&v)[8]) {
    if (bytes) {
      const float s = scale_value(x.code[h]);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int q = (int)x.p[h][w];
        v[4 * w + 0] = __builtin_amdgcn_cvt_f32_fp8(q, 0) * s;
        v[4 * w + 1] = __builtin_amdgcn_cvt_f32_fp8(q, 1) * s;
        v[4 * w + 2] = __builtin_amdgcn_cvt_f32_fp8(q, 2) * s;
        v[4 * w + 3] = __builtin_amdgcn_cvt_f32_fp8(q, 3) * s;
      }
    } else {
      unpack8<DT>(x.p[h], v);
    }
  };
  RawRow<GATED> raw = {}, next = {};
  load(tid >> 3, raw);
#pragma unroll 1
  for (int r = tid >> 3; r < ROWS; r += 32) {
    if (r + 32 < ROWS) load(r + 32, next);
    __builtin_amdgcn_sched_barrier(0);
    const int64_t row = m0 + r;
    float d[PARTS][8] = {};
    if (row < p.m && left > 0) {
      float dy[8], x[8], u[8];
      unpack8<DT>(raw.dy, dy);
      values(raw, 0, x);
      if constexpr (GATED) values(raw, 1, u);
      if (!need_p) {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[0][e] = dy[e];
      } else {
        with_kind(kind, [&](auto tag) {
          constexpr int KIND = decltype(tag)::value;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float value, slope;
            act_both<KIND>(x[e], c1, c3, value, slope);
            d[0][e] = dy[e] * (GATED ? u[e] * slope : slope);
            if constexpr (GATED) d[1][e] = dy[e] * value;
          }
        });
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e >= left)
#pragma unroll
          for (int h = 0; h < PARTS; ++h) d[h][e] = 0.0f;
    }
#pragma unroll
    for (int h = 0; h < PARTS; ++h) {
      const u32x4_t w = pack8<DT>(d[h]);
#pragma unroll
      for (int e = 0; e < 8; ++e) total[h][e] += d[h][e];
      if (p.dt) *reinterpret_cast<u32x4_t*>(smem + (h * ROWS + r) * RB + ((c ^ (r & (CH - 1))) << 4)) = w;
      if (p.d && row < p.m && left > 0) {
        uint16_t* out = static_cast<uint16_t*>(p.d) + row * p.ldd + (int64_t)h * p.n;
        store8(out + col, w, left);
        if (h == PARTS - 1 && left <= 8)       // the row's end, up to a whole 16-byte piece
          for (int64_t e = p.n; (h * (int64_t)p.n + e) % 8 != 0; ++e) out[e] = 0;
      }
    }
    raw = next;
  }
  if (p.sums) {
    // over the rows of the wave (lanes 8 apart hold the same columns), then the waves
#pragma unroll
    for (int h = 0; h < PARTS; ++h)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float t = total[h][e];
        t += __shfl_xor(t, 8);
        t += __shfl_xor(t, 16);
        t += __shfl_xor(t, 32);
        if (lane < 8) sums[wave][h][8 * c + e] = t;
      }
  }
  __syncthreads();
  if (p.sums && tid < PARTS * kDCols) {
    const int h = tid / kDCols, x = tid % kDCols;
    if (cb * kDCols + x < p.n)
      p.sums[(rb * PARTS + h) * p.n + cb * kDCols + x] = (sums[0][h][x] + sums[1][h][x]) + (sums[2][h][x] + sums[3][h][x]);
  }
  if (p.dt) {
    // Transposing reads: a wave takes 16 columns x 32 rows at a time, lane (g4,
    // i16) the rows 8 g4 .. 8 g4 + 7 of column i16 (two reads of four rows, each
    // lane of a group giving the address of row i16 / 4, columns 4 (i16 % 4) ..
    // + 3 of the 4 x 16 block), 16 bytes of the column's row.
    const int g4 = lane >> 4, i16 = lane & 15;
    constexpr int UNITS = PARTS * (kDCols / 16) * (ROWS / 32);
#pragma unroll 2
    for (int q = 0; q < UNITS / 4; ++q) {
      const int u = q * 4 + wave, h = u / (UNITS / PARTS), v = u % (UNITS / PARTS);
      const int nb = (v / (ROWS / 32)) * 16, mb = (v % (ROWS / 32)) * 32 + 8 * g4;
      u32x2_t half[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int r = mb + 4 * s + (i16 >> 2), x = nb + 4 * (i16 & 3);
        half[s] = read_tr(smem + (h * ROWS + r) * RB + (((x >> 3) ^ (r & (CH - 1))) << 4) + (x & 4) * 2);
      }
      const int x = cb * kDCols + nb + i16;
      if (x < p.n && m0 + mb < p.ldt)
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p.dt) + ((int64_t)h * p.n + x) * p.ldt + m0 + mb) =
            u32x4_t{half[0][0], half[0][1], half[1][0], half[1][1]};
    }
  }
}

// y once more from the kept pre-activations, eight columns per thread.
template <int DT>
__global__ __launch_bounds__(256) void feed_again_kernel(FeedAgainProblem p) {
  const uint32_t pieces = (uint32_t)((p.n + 7) / 8);
  const int64_t all = p.m * pieces;
  with_kind(p.act.kind, [&](auto kind) {
    constexpr int KIND = decltype(kind)::value;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < all; u += (int64_t)gridDim.x * 256) {
      const int64_t row = u / pieces;
      const int col = (int)(u - row * pieces) * 8;
      float x[8], f[8], y[8];
      const int64_t at = row * (p.gated ? 2 : 1) * p.kept.wide + col;
      kept8<DT>(p.kept, at, x);
      if (p.gated) kept8<DT>(p.kept, at + p.kept.wide, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = act_value<KIND>(x[e], p.act.c1, p.act.c3);
        if (p.gated) y[e] *= f[e];
      }
      store8(static_cast<uint16_t*>(p.y) + row * p.ldy + col, pack8<DT>(y), p.n - col);
    }
  });
}

struct SumPair {
  SumRanges a, b;
  int64_t a_pieces, pieces;
};

template <int DT>
__global__ __launch_bounds__(256) void sum_ranges_kernel(SumPair s) {
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < s.pieces; u += (int64_t)gridDim.x * 256) {
    const bool second = u >= s.a_pieces;
    const SumRanges& c = second ? s.b : s.a;
    const int64_t at = second ? u - s.a_pieces : u;
    const int64_t n4 = (c.cols + 3) / 4, row = at / n4, col = (at - row * n4) * 4;
    const int64_t plane = c.rows * n4 * 4;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    // eight ranges are on their way at a time, added in order
    for (int q0 = 0; q0 < c.ranges; q0 += 8) {
      f32x4_t w[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q0 + q < c.ranges) w[q] = *reinterpret_cast<const f32x4_t*>(c.sums + at * 4 + (q0 + q) * plane);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q0 + q < c.ranges) v += w[q];
    }
    store4(static_cast<uint16_t*>(c.out) + row * c.ldo + col, u32x2_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])},
           (int)(c.cols - col < 4 ? c.cols - col : 4));
  }
}

// 64 columns per workgroup, whose 16 waves share out the groups.
__global__ __launch_bounds__(1024) void sum_columns_kernel(SumColumns p) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;
  float t = 0.0f;
  if (col < p.cols) {
    int64_t g = wave;
    for (; g + 112 < p.groups; g += 128) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = p.sums[(g + 16 * q) * p.cols + col];
#pragma unroll
      for (int q = 0; q < 8; ++q) t += v[q];
    }
    for (; g < p.groups; g += 16) t += p.sums[g * p.cols + col];
  }
  part[wave][lane] = t;
  __syncthreads();
  if (wave || col >= p.cols) return;
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < 16; ++w) s += part[w][lane];
  const bool second = col >= p.first;
  void* out = second ? p.out2 : p.out;
  const int64_t at = second ? col - p.first : col;
  if (!out) return;
  if (p.dtype == kDtypeFp32) static_cast<float*>(out)[at] = s;
  else static_cast<uint16_t*>(out)[at] = p.dtype == kDtypeBf16 ? cvt1<kDtypeBf16>(s) : cvt1<kDtypeFp16>(s);
}

constexpr int64_t kLoopGrid = 1 << 16;   // workgroups of the kernels that loop over their work

}  // namespace

static bool copies_valid(const FeedCopies& c) {
  for (const PadRows* r : {&c.a, &c.w})
    if (r->num_groups != 0 && (r->num_groups < 1 || r->num_groups > kMaxGroups || r->rows < 1 || r->rows > INT32_MAX || r->chunks < 1 ||
                               r->chunks > INT32_MAX || r->cols < 1 || r->cols > r->chunks * 8 || r->cols > INT32_MAX || !r->out))
      return false;
  return true;
}

hipError_t launch_feed_copies(const FeedCopies& c, hipStream_t s) {
  if (!copies_valid(c)) return hipErrorInvalidValue;
  const int64_t a = copy_groups(c.a), w = copy_groups(c.w);
  if (a + w < 1) return hipErrorInvalidValue;
  hipLaunchKernelGGL(feed_copies_kernel, dim3((unsigned)(a + w)), dim3(256), 0, s, c, (int32_t)a, (int32_t)w);
  return hipGetLastError();
}

hipError_t launch_feed_d(const FeedDProblem& p, const FeedCopies& copies, int dtype, hipStream_t s) {
  const int parts = p.gated ? 2 : 1;
  const int64_t blocks = (p.m + p.block - 1) / p.block * ((p.n + kDCols - 1) / kDCols);
  const int64_t a = copy_groups(copies.a), w = copy_groups(copies.w);
  if (p.m < 1 || p.n < 1 || (p.block != 32 && p.block != 128) || blocks >= kFeedGrid - 16384 || !copies_valid(copies) ||
      (!p.kept.values && (p.gated || p.act.kind != kActLinear)) ||
      (p.kept.values && p.kept.wide != ((int64_t)p.n + kKeptBlock - 1) / kKeptBlock * kKeptBlock) ||
      (p.d && (p.ldd % 8 != 0 || p.ldd < (int64_t)parts * p.n)) || (p.dt && (p.ldt % 8 != 0 || p.ldt < p.m)) ||
      (dtype != kDtypeBf16 && dtype != kDtypeFp16))
    return hipErrorInvalidValue;
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks + a + w)), dim3(256), 0, s, p, copies, (int32_t)blocks, (int32_t)a, (int32_t)w);
  };
  const auto rows = [&](auto dt, auto gated) {
    constexpr int DT = decltype(dt)::value;
    constexpr bool G = decltype(gated)::value;
    p.block == 128 ? go(feed_d_kernel<DT, G, 128>) : go(feed_d_kernel<DT, G, 32>);
  };
  if (dtype == kDtypeBf16) p.gated ? rows(IntTag<kDtypeBf16>{}, BoolTag<true>{}) : rows(IntTag<kDtypeBf16>{}, BoolTag<false>{});
  else p.gated ? rows(IntTag<kDtypeFp16>{}, BoolTag<true>{}) : rows(IntTag<kDtypeFp16>{}, BoolTag<false>{});
  return hipGetLastError();
}

hipError_t launch_feed_again(const FeedAgainProblem& p, int dtype, hipStream_t s) {
  if (p.m < 1 || p.n < 1 || !p.kept.values || (dtype != kDtypeBf16 && dtype != kDtypeFp16) ||
      p.kept.wide != ((int64_t)p.n + kKeptBlock - 1) / kKeptBlock * kKeptBlock)
    return hipErrorInvalidValue;
  const int64_t blocks = (p.m * ((p.n + 7) / 8) + 255) / 256;
  const dim3 grid((unsigned)(blocks < kLoopGrid ? blocks : kLoopGrid));
  if (dtype == kDtypeBf16) hipLaunchKernelGGL((feed_again_kernel<kDtypeBf16>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((feed_again_kernel<kDtypeFp16>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_sum_ranges(const SumRanges* a, const SumRanges* b, int dtype, hipStream_t s) {
  SumPair c{};
  if (a) c.a = *a, c.a_pieces = a->rows * ((a->cols + 3) / 4);
  c.pieces = c.a_pieces;
  if (b) c.b = *b, c.pieces += b->rows * ((b->cols + 3) / 4);
  if (c.pieces < 1 || (dtype != kDtypeBf16 && dtype != kDtypeFp16)) return hipErrorInvalidValue;
  const int64_t blocks = (c.pieces + 255) / 256;
  const dim3 grid((unsigned)(blocks < kLoopGrid ? blocks : kLoopGrid));
  if (dtype == kDtypeBf16) hipLaunchKernelGGL((sum_ranges_kernel<kDtypeBf16>), grid, dim3(256), 0, s, c);
  else hipLaunchKernelGGL((sum_ranges_kernel<kDtypeFp16>), grid, dim3(256), 0, s, c);
  return hipGetLastError();
}

hipError_t launch_sum_columns(const SumColumns& p, hipStream_t s) {
  const int64_t grid = (p.cols + 63) / 64;
  if (p.cols < 1 || p.groups < 1 || grid >= kFeedGrid / 4) return hipErrorInvalidValue;
  hipLaunchKernelGGL(sum_columns_kernel, dim3((unsigned)grid), dim3(1024), 0, s, p);
  return hipGetLastError();
}

}  // namespace agmm
