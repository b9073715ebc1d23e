// Layer norm over rows, forward and backward (gfx950).
//
//     y = (x - mean) rstd w + b                     mean, var over the row, rstd = 1 / sqrt(var + eps)
//     dx = rstd (g - mean(g) - h mean(g h)),        g = dy w,  h = (x - mean) rstd
//     dw = sum over rows of dy h,  db = sum over rows of dy
//
// A row is held in registers by THREADS lanes, CH 16-byte pieces each, so that
// x is read once: the mean first, then the sums of x - mean, which is what the
// mean's rounding left, and of its square (the difference of two large sums
// would lose the variance of rows far from 0).
// Rows longer than 1024 threads hold are read again for each sum.
//
// Backward, a workgroup takes as many rows at a time as 1024 threads hold, and
// every `groups`-th such set; a lane's columns stay the same, so the two column
// sums are registers too, and leave once at the end as [groups][2][columns],
// which sum_columns_kernel adds in order (one group: as dw and db at once).  The
// next row's loads are on their way while a row is reduced.
//
// Bound: HBM; few rows: a launch.  Statistics and sums are fp32; results are
// rounded once.  Measured: forward 8192 x 8192 bf16, fp32 weights 53-55 us, 4.9
// TB/s (weights are loaded once per workgroup of three a CU, not per row: 80 us);
// 128 x 4096 4; backward 8192 x 8192 77-80 us, 5.1 TB/s, and 4 for the sums; 1011
// x 4035 fp16 11 and 3 (1011 x 4096: 10.6; rows at odd addresses cost little).
// Backward past 8192 16-bit columns x and dy are read three times: 4096 x 16384
// bf16 59, 119 and 5.
#include "feed_device.h"

namespace agmm {

namespace {

template <int DT>
struct Elem {
  static constexpr int kBytes = DT == kDtypeFp32 ? 4 : 2;
  static constexpr int V = 16 / kBytes;        // of a piece
};

// A lane's piece of a row of `cols`, at column `col`, of any alignment: zeros
// past the row's end, in two steps.  load(): 16 bytes of the row, the piece
// itself or, at its end, the last 16, unconditionally: a condition would make
// every later wait for a load one for all stores too.  settle(), where the
// values are needed, shifts out what lies before the piece.  SHORT rows, of less
// than 16 bytes, are loaded by element.
template <int DT, bool SHORT>
struct Piece {
  static constexpr int V = Elem<DT>::V;
  int64_t at;              // column of the 16 bytes
  int over;                // elements of them before the piece
  int64_t col, cols;
  __device__ __forceinline__ Piece(int64_t col, int64_t cols) : col(col), cols(cols) {
    const int64_t last = SHORT ? 0 : cols - V;
    at = col < last ? col : last;
    over = SHORT ? 0 : col - at < V ? (int)(col - at) : V;
  }
  __device__ __forceinline__ u32x4_t load(const void* row) const {
    if constexpr (!SHORT) {
      return *reinterpret_cast<const u32x4_any_t*>(static_cast<const char*>(row) + at * Elem<DT>::kBytes);
    } else {
      u32x4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (col + e < cols) {
          if constexpr (DT == kDtypeFp32) v[e] = static_cast<const uint32_t*>(row)[col + e];
          else v[e >> 1] |= (uint32_t)static_cast<const uint16_t*>(row)[col + e] << (16 * (e & 1));
        }
      return v;
    }
  }
  __device__ __forceinline__ u32x4_t settle(u32x4_t v) const {
    if (!SHORT && over) {
      if (DT != kDtypeFp32 && (over & 1))
        v = u32x4_t{__builtin_amdgcn_alignbyte(v[1], v[0], 2), __builtin_amdgcn_alignbyte(v[2], v[1], 2),
                    __builtin_amdgcn_alignbyte(v[3], v[2], 2), v[3] >> 16};
      const int words = DT != kDtypeFp32 ? over >> 1 : over;
      if (words & 1) v = u32x4_t{v[1], v[2], v[3], 0u};
      if (words & 2) v = u32x4_t{v[2], v[3], 0u, 0u};
      if (words & 4) v = u32x4_t{0u, 0u, 0u, 0u};
    }
    return v;
  }
};
template <int DT>
__device__ __forceinline__ u32x4_t load_piece(const void* x, int64_t col, int64_t cols) {
  if (cols < Elem<DT>::V) return Piece<DT, true>(col, cols).load(x);
  const Piece<DT, false> p(col, cols);
  return p.settle(p.load(x));
}
// Row r, `ld` elements apart.
template <int DT>
__device__ __forceinline__ const void* row_of(const void* x, int64_t r, int64_t ld) {
  return static_cast<const char*>(x) + r * ld * Elem<DT>::kBytes;
}
template <int DT>
__device__ __forceinline__ float piece_value(const u32x4_t& v, int e) {
  const uint32_t w = v[e];   // a bit cast of the vector's element itself takes element 0
  if constexpr (DT == kDtypeFp32) return __builtin_bit_cast(float, w);
  else return e & 1 ? high16<DT>(v[e >> 1]) : low16<DT>(v[e >> 1]);
}
template <int DT>
__device__ __forceinline__ void store_piece(void* x, int64_t at, int64_t left, const float* v) {
  if constexpr (DT == kDtypeFp32) {
    typedef f32x4_t f32x4_word_t __attribute__((aligned(4)));
    float* p = static_cast<float*>(x) + at;
    if (left >= 4) {
      *reinterpret_cast<f32x4_word_t*>(p) = f32x4_t{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) p[e] = v[e];
    }
  } else {
    store8(static_cast<uint16_t*>(x) + at, u32x4_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])},
           left < 8 ? (int)left : 8);
  }
}
// V consecutive weights (of the rows' type or fp32) as fp32, `none` where there
// are no weights or past the end.
template <int WT, int V>
__device__ __forceinline__ void load_weights(const void* w, int64_t col, int64_t cols, float none, float (&v)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = none;
  if (!w) return;
  constexpr int U = Elem<WT>::V < V ? Elem<WT>::V : V;
#pragma unroll
  for (int s = 0; s < V / U; ++s) {
    if (col + s * U >= cols) break;
    const u32x4_t q = load_piece<WT>(w, col + s * U, cols);
#pragma unroll
    for (int e = 0; e < U; ++e)
      if (col + s * U + e < cols) v[s * U + e] = piece_value<WT>(q, e);
  }
}

// Sums of N values over the lanes of a workgroup, in every lane, in a fixed
// order.  Two buffers in turn: one barrier a call.
template <int THREADS, int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*buf)[N], int& turn) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2)
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] += __shfl_xor(v[q], d);
  if constexpr (THREADS > 64) {
    constexpr int W = THREADS / 64;
    float(*b)[N] = buf + turn * W;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int q = 0; q < N; ++q) b[threadIdx.x >> 6][q] = v[q];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < N; ++q) {
      v[q] = b[0][q];
#pragma unroll
      for (int w = 1; w < W; ++w) v[q] += b[w][q];
    }
  }
}

template <int DT, int WT, int THREADS, int CH, bool SHORT = false>
__global__ __launch_bounds__(THREADS) void norm_forward_kernel(NormProblem p) {
  constexpr int V = Elem<DT>::V;
  constexpr bool HOLD = THREADS <= 512;             // the weights stay in registers from row to row
  __shared__ float buf[2 * THREADS / 64][1], buf2[2 * THREADS / 64][2];
  int turn = 0, turn2 = 0;
  const auto col_of = [&](int c) { return ((int64_t)c * THREADS + threadIdx.x) * V; };
  u32x4_t x[CH], next[CH];
  const auto piece = [&](int c) { return Piece<DT, SHORT>(col_of(c), p.cols); };
  const auto load = [&](int64_t row, u32x4_t (&to)[CH]) {   // past the last row: that one again
    const void* at = row_of<DT>(p.x, row < p.rows ? row : p.rows - 1, p.ldx);
#pragma unroll
    for (int c = 0; c < CH; ++c) to[c] = piece(c).load(at);
  };
  int64_t row = blockIdx.x;
  load(row, x);
  float w[HOLD ? CH : 1][V], b[HOLD ? CH : 1][V];
  if constexpr (HOLD)
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      load_weights<WT>(p.weight, col_of(c), p.cols, 1.0f, w[c]);
      load_weights<WT>(p.bias, col_of(c), p.cols, 0.0f, b[c]);
    }
  for (; row < p.rows; row += gridDim.x) {
    load(row + gridDim.x, next);               // on its way while this row is reduced
    __builtin_amdgcn_sched_barrier(0);
    float s[1] = {0.0f}, t[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) x[c] = piece(c).settle(x[c]);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < V; ++e) s[0] += piece_value<DT>(x[c], e);
    block_sum<THREADS>(s, buf, turn);
    const float near = s[0] / (float)p.cols;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t left = p.cols - col_of(c);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = e < left ? piece_value<DT>(x[c], e) - near : 0.0f;
        t[0] += d;
        t[1] = __builtin_fmaf(d, d, t[1]);
      }
    }
    block_sum<THREADS>(t, buf2, turn2);
    const float rest = t[0] / (float)p.cols, var = __builtin_fmaf(-rest, rest, t[1] / (float)p.cols);
    const float rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = near + rest;
      if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t col = col_of(c), left = p.cols - col;
      if (left > 0) {
        float y[V];
        if constexpr (!HOLD) {
          load_weights<WT>(p.weight, col, p.cols, 1.0f, w[0]);
          load_weights<WT>(p.bias, col, p.cols, 0.0f, b[0]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
          y[e] = __builtin_fmaf((piece_value<DT>(x[c], e) - near - rest) * rstd, w[HOLD ? c : 0][e], b[HOLD ? c : 0][e]);
        store_piece<DT>(p.y, row * p.ldy + col, left, y);
      }
      x[c] = next[c];
    }
  }
}

// Rows of any length, 1024 threads each, read once for every sum.
template <int DT, int WT>
__global__ __launch_bounds__(1024) void norm_forward_long_kernel(NormProblem p) {
  constexpr int V = Elem<DT>::V;
  __shared__ float buf[32][1], buf2[32][2];
  int turn = 0, turn2 = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const void* at = row_of<DT>(p.x, row, p.ldx);
    float s[1] = {0.0f}, t[2] = {0.0f, 0.0f};
    for (int64_t col = (int64_t)threadIdx.x * V; col < p.cols; col += 1024 * V) {
      const u32x4_t x = load_piece<DT>(at, col, p.cols);
#pragma unroll
      for (int e = 0; e < V; ++e) s[0] += piece_value<DT>(x, e);
    }
    block_sum<1024>(s, buf, turn);
    const float near = s[0] / (float)p.cols;
    for (int64_t col = (int64_t)threadIdx.x * V; col < p.cols; col += 1024 * V) {
      const u32x4_t x = load_piece<DT>(at, col, p.cols);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = e < p.cols - col ? piece_value<DT>(x, e) - near : 0.0f;
        t[0] += d;
        t[1] = __builtin_fmaf(d, d, t[1]);
      }
    }
    block_sum<1024>(t, buf2, turn2);
    const float rest = t[0] / (float)p.cols, var = __builtin_fmaf(-rest, rest, t[1] / (float)p.cols);
    const float rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = near + rest;
      if (p.rstd) p.rstd[row] = rstd;
    }
    for (int64_t col = (int64_t)threadIdx.x * V; col < p.cols; col += 1024 * V) {
      const int64_t left = p.cols - col;
      const u32x4_t x = load_piece<DT>(at, col, p.cols);
      float w[V], b[V], y[V];
      load_weights<WT>(p.weight, col, p.cols, 1.0f, w);
      load_weights<WT>(p.bias, col, p.cols, 0.0f, b);
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] = __builtin_fmaf((piece_value<DT>(x, e) - near - rest) * rstd, w[e], b[e]);
      store_piece<DT>(p.y, row * p.ldy + col, left, y);
    }
  }
}

// THREADS lanes a row, CH pieces each, 1024 / THREADS rows at a time, whose
// column sums are added at the end.
template <int DT, int WT, int THREADS, int CH, bool SHORT = false>
__global__ __launch_bounds__(1024) void norm_backward_kernel(NormProblem p) {
  constexpr int V = Elem<DT>::V, ROWS = 1024 / THREADS, W = THREADS / 64;
  __shared__ float buf[2][16][2];
  __shared__ float more[ROWS > 1 ? 2 * THREADS * V * CH : 1];
  int turn = 0;
  const int lane = threadIdx.x % THREADS, sub = threadIdx.x / THREADS;
  const auto col_of = [&](int c) { return ((int64_t)c * THREADS + lane) * V; };
  float w[CH][V], dw[CH][V] = {}, db[CH][V] = {};
#pragma unroll
  for (int c = 0; c < CH; ++c) load_weights<WT>(p.weight, col_of(c), p.cols, 1.0f, w[c]);
  u32x4_t x[CH], dy[CH];
  float mean = 0.0f, rstd = 0.0f;
  const auto piece = [&](int c) { return Piece<DT, SHORT>(col_of(c), p.cols); };
  const auto load = [&](int64_t row) {         // past the last row: that one again
    row = row < p.rows ? row : p.rows - 1;
    const void *ax = row_of<DT>(p.x, row, p.ldx), *ady = row_of<DT>(p.dy, row, p.lddy);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      x[c] = piece(c).load(ax);
      dy[c] = piece(c).load(ady);
    }
    mean = p.mean[row];
    rstd = p.rstd[row];
  };
  const float inv = 1.0f / (float)p.cols;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  load((int64_t)blockIdx.x * ROWS + sub);
  for (int64_t first = (int64_t)blockIdx.x * ROWS; first < p.rows; first += step) {
    const int64_t row = first + sub;
    float g[CH][V], h[CH][V], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      x[c] = piece(c).settle(x[c]);
      dy[c] = row < p.rows ? piece(c).settle(dy[c]) : u32x4_t{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = piece_value<DT>(dy[c], e);
        h[c][e] = col_of(c) + e < p.cols && row < p.rows ? (piece_value<DT>(x[c], e) - mean) * rstd : 0.0f;
        g[c][e] = d * w[c][e];
        s[0] += g[c][e];
        s[1] = __builtin_fmaf(g[c][e], h[c][e], s[1]);
        dw[c][e] = __builtin_fmaf(d, h[c][e], dw[c][e]);
        db[c][e] += d;
      }
    const float scale = rstd;
    load(row + step);                          // on its way while this row is reduced
    __builtin_amdgcn_sched_barrier(0);
    if (!p.dx) continue;
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
#pragma unroll
      for (int q = 0; q < 2; ++q) s[q] += __shfl_xor(s[q], d);
    if constexpr (W > 1) {
      if ((threadIdx.x & 63) == 0) {
        buf[turn][threadIdx.x >> 6][0] = s[0];
        buf[turn][threadIdx.x >> 6][1] = s[1];
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        s[q] = buf[turn][sub * W][q];
#pragma unroll
        for (int v = 1; v < W; ++v) s[q] += buf[turn][sub * W + v][q];
      }
      turn ^= 1;                               // two buffers in turn: one barrier a row
    }
    if (row < p.rows) {
      const float a = s[0] * inv, b = s[1] * inv;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (col_of(c) >= p.cols) continue;
        float v[V];
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = scale * (g[c][e] - __builtin_fmaf(h[c][e], b, a));
        store_piece<DT>(p.dx, row * p.lddx + col_of(c), p.cols - col_of(c), v);
      }
    }
  }
  if (!p.sums && !p.dweight && !p.dbias) return;
  if constexpr (ROWS > 1)
#pragma unroll 1
    for (int r = 1; r < ROWS; ++r) {
      if (sub == r)
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            more[((c * V + e) * 2 + 0) * THREADS + lane] = dw[c][e];
            more[((c * V + e) * 2 + 1) * THREADS + lane] = db[c][e];
          }
      __syncthreads();
      if (sub == 0)
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            dw[c][e] += more[((c * V + e) * 2 + 0) * THREADS + lane];
            db[c][e] += more[((c * V + e) * 2 + 1) * THREADS + lane];
          }
      __syncthreads();
    }
  if (sub) return;
  if (!p.sums) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t col = col_of(c);
      if (col >= p.cols) continue;
      constexpr int U = Elem<WT>::V < V ? Elem<WT>::V : V;
#pragma unroll
      for (int s = 0; s < V / U; ++s) {
        if (p.dweight) store_piece<WT>(p.dweight, col + U * s, p.cols - col - U * s, dw[c] + U * s);
        if (p.dbias) store_piece<WT>(p.dbias, col + U * s, p.cols - col - U * s, db[c] + U * s);
      }
    }
    return;
  }
  float* out = p.sums + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int64_t col = col_of(c);
    if (col >= p.cols) continue;
#pragma unroll
    for (int s = 0; s < V / 4; ++s) {
      store_piece<kDtypeFp32>(out, col + 4 * s, p.cols - col - 4 * s, dw[c] + 4 * s);
      store_piece<kDtypeFp32>(out + p.cols, col + 4 * s, p.cols - col - 4 * s, db[c] + 4 * s);
    }
  }
}

// Rows of any length: dx by rows, read twice.
template <int DT, int WT>
__global__ __launch_bounds__(1024) void norm_dx_long_kernel(NormProblem p) {
  constexpr int V = Elem<DT>::V;
  __shared__ float buf[32][2];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float mean = p.mean[row], rstd = p.rstd[row];
    const auto piece = [&](int64_t col, float (&g)[V], float (&h)[V]) {
      const int64_t left = p.cols - col;
      const u32x4_t x = load_piece<DT>(row_of<DT>(p.x, row, p.ldx), col, p.cols),
                    dy = load_piece<DT>(row_of<DT>(p.dy, row, p.lddy), col, p.cols);
      float w[V];
      load_weights<WT>(p.weight, col, p.cols, 1.0f, w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        h[e] = e < left ? (piece_value<DT>(x, e) - mean) * rstd : 0.0f;
        g[e] = piece_value<DT>(dy, e) * w[e];
      }
    };
    float s[2] = {0.0f, 0.0f};
    for (int64_t col = (int64_t)threadIdx.x * V; col < p.cols; col += 1024 * V) {
      float g[V], h[V];
      piece(col, g, h);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s[0] += g[e];
        s[1] = __builtin_fmaf(g[e], h[e], s[1]);
      }
    }
    block_sum<1024>(s, buf, turn);
    const float a = s[0] / (float)p.cols, b = s[1] / (float)p.cols;
    for (int64_t col = (int64_t)threadIdx.x * V; col < p.cols; col += 1024 * V) {
      float g[V], h[V], v[V];
      piece(col, g, h);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = rstd * (g[e] - __builtin_fmaf(h[e], b, a));
      store_piece<DT>(p.dx, row * p.lddx + col, p.cols - col, v);
    }
  }
}

// and the column sums: 256 V columns of every `groups`-th row per workgroup.
template <int DT>
__global__ __launch_bounds__(256) void norm_sums_long_kernel(NormProblem p) {
  constexpr int V = Elem<DT>::V;
  const int64_t strips = (p.cols + 256 * V - 1) / (256 * V);
  const int64_t group = blockIdx.x / strips, col = ((blockIdx.x - group * strips) * 256 + threadIdx.x) * V, left = p.cols - col;
  if (left <= 0) return;
  float dw[V] = {}, db[V] = {};
#pragma unroll 4
  for (int64_t row = group; row < p.rows; row += p.groups) {
    const u32x4_t x = load_piece<DT>(row_of<DT>(p.x, row, p.ldx), col, p.cols),
                    dy = load_piece<DT>(row_of<DT>(p.dy, row, p.lddy), col, p.cols);
    const float mean = p.mean[row], rstd = p.rstd[row];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float d = piece_value<DT>(dy, e);
      dw[e] = __builtin_fmaf(d, (piece_value<DT>(x, e) - mean) * rstd, dw[e]);
      db[e] += d;
    }
  }
  float* out = p.sums + group * 2 * p.cols;
#pragma unroll
  for (int s = 0; s < V / 4; ++s) {
    store_piece<kDtypeFp32>(out, col + 4 * s, left - 4 * s, dw + 4 * s);
    store_piece<kDtypeFp32>(out + p.cols, col + 4 * s, left - 4 * s, db + 4 * s);
  }
}

int64_t pieces_of(int64_t cols, int dtype) { return (cols + (dtype == kDtypeFp32 ? 3 : 7)) / (dtype == kDtypeFp32 ? 4 : 8); }

// Pieces of the longest rows that the backward kernel holds in registers.
int64_t held_pieces(int dtype) { return dtype == kDtypeFp32 ? 2048 : 1024; }

template <int DT, int WT>
hipError_t forward_type(const NormProblem& p, hipStream_t s) {
  const int64_t pieces = pieces_of(p.cols, DT);
  // workgroups that the CUs hold at a time, which take every so many-th row
  const auto go = [&](auto kernel, int threads, int per = 1) {
    const int64_t most = (int64_t)p.cus * per;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(p.rows < most ? p.rows : most)), dim3(threads), 0, s, p);
  };
  if (p.cols < Elem<DT>::V) go(norm_forward_kernel<DT, WT, 64, 1, true>, 64, 24);
  else if (pieces <= 64) go(norm_forward_kernel<DT, WT, 64, 1>, 64, 24);
  else if (pieces <= 128) go(norm_forward_kernel<DT, WT, 64, 2>, 64, 16);
  else if (pieces <= 256) go(norm_forward_kernel<DT, WT, 256, 1>, 256, 8);
  else if (pieces <= 512) go(norm_forward_kernel<DT, WT, 256, 2>, 256, 5);
  else if (pieces <= 1024) go(norm_forward_kernel<DT, WT, 256, 4>, 256, 3);
  else if (pieces <= 2048) go(norm_forward_kernel<DT, WT, 512, 4>, 512, 2);
  else if (pieces <= 4096) go(norm_forward_kernel<DT, WT, 1024, 4>, 1024, 2);
  else go(norm_forward_long_kernel<DT, WT>, 1024, 2);
  return hipGetLastError();
}

template <int DT, int WT>
hipError_t backward_type(const NormProblem& p, hipStream_t s) {
  const int64_t pieces = pieces_of(p.cols, DT);
  const auto go = [&](auto kernel, int64_t grid, int threads) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(threads), 0, s, p);
  };
  if (p.cols < Elem<DT>::V) go(norm_backward_kernel<DT, WT, 64, 1, true>, p.groups, 1024);
  else if (pieces <= 64) go(norm_backward_kernel<DT, WT, 64, 1>, p.groups, 1024);
  else if (pieces <= 128) go(norm_backward_kernel<DT, WT, 128, 1>, p.groups, 1024);
  else if (pieces <= 256) go(norm_backward_kernel<DT, WT, 256, 1>, p.groups, 1024);
  else if (pieces <= 512) go(norm_backward_kernel<DT, WT, 512, 1>, p.groups, 1024);
  else if (pieces <= 1024) go(norm_backward_kernel<DT, WT, 1024, 1>, p.groups, 1024);
  else if (DT == kDtypeFp32 && pieces <= 2048) go(norm_backward_kernel<DT, WT, 1024, DT == kDtypeFp32 ? 2 : 1>, p.groups, 1024);
  else {
    // the sums first: dx may overwrite dy
    if (p.sums) go(norm_sums_long_kernel<DT>, (pieces + 255) / 256 * p.groups, 256);
    if (p.dx) go(norm_dx_long_kernel<DT, WT>, p.rows < 2 * p.cus ? p.rows : 2 * p.cus, 1024);
  }
  return hipGetLastError();
}

bool valid(const NormProblem& p) {
  return p.rows >= 1 && p.rows < (int64_t(1) << 31) && p.cus >= 1 && p.cols >= 1 && p.cols < (int64_t(1) << 31) && p.x &&
         (p.wtype == p.dtype || p.wtype == kDtypeFp32);
}

template <class F>
hipError_t by_type(const NormProblem& p, F&& f) {
  const bool wide = p.wtype == kDtypeFp32;
  if (p.dtype == kDtypeBf16) return wide ? f(IntTag<kDtypeBf16>{}, IntTag<kDtypeFp32>{}) : f(IntTag<kDtypeBf16>{}, IntTag<kDtypeBf16>{});
  if (p.dtype == kDtypeFp16) return wide ? f(IntTag<kDtypeFp16>{}, IntTag<kDtypeFp32>{}) : f(IntTag<kDtypeFp16>{}, IntTag<kDtypeFp16>{});
  return p.dtype == kDtypeFp32 ? f(IntTag<kDtypeFp32>{}, IntTag<kDtypeFp32>{}) : hipErrorInvalidValue;
}

}  // namespace

bool norm_direct(int64_t cols, int dtype, int groups) { return groups == 1 && pieces_of(cols, dtype) <= held_pieces(dtype); }

int norm_groups(int64_t rows, int64_t cols, int dtype, int cus) {
  const int64_t pieces = pieces_of(cols, dtype);
  int64_t at_once = 1;                         // rows that a workgroup takes at a time
  while (at_once < 16 && pieces * at_once <= 512) at_once *= 2;
  // one workgroup a CU, whose sums are one row of [groups]; long rows: so many
  // strips that they fill the CUs four times
  int64_t groups = cus;
  if (pieces > held_pieces(dtype)) groups = 4 * cus / ((pieces + 255) / 256);
  else rows = (rows + at_once - 1) / at_once;
  // few rows: one workgroup writes the sums itself, which saves the launch that
  // adds groups (about 4 us, as long as four turns of a workgroup)
  if (pieces <= held_pieces(dtype) && rows <= 4) return 1;
  if (groups > rows) groups = rows;
  return (int)(groups < 1 ? 1 : groups);
}

hipError_t launch_norm_forward(const NormProblem& p, hipStream_t s) {
  if (!valid(p) || !p.y) return hipErrorInvalidValue;
  return by_type(p, [&](auto t, auto w) { return forward_type<decltype(t)::value, decltype(w)::value>(p, s); });
}

hipError_t launch_norm_backward(const NormProblem& p, hipStream_t s) {
  if (!valid(p) || !p.dy || !p.mean || !p.rstd || (!p.dx && !p.sums && !p.dweight && !p.dbias) || p.groups < 1 ||
      ((p.dweight || p.dbias) && (p.sums || p.groups != 1 || pieces_of(p.cols, p.dtype) > held_pieces(p.dtype))) || p.groups > p.rows)
    return hipErrorInvalidValue;
  return by_type(p, [&](auto t, auto w) { return backward_type<decltype(t)::value, decltype(w)::value>(p, s); });
}

}  // namespace agmm
