// C ABI of the operators around the all-gather matmul (host side): the
// block-scaled 8-bit quantiser.
#include <hip/hip_runtime.h>

#include "agmm.h"
#include "agmm_host.h"
#include "agmm_kernels.h"

namespace {

using agmm::hip_err;
using agmm::ok;
using agmm::set_err;

// Rows and columns of a quantised matrix, and their product: every launch
// then stays below 2^24 workgroups of 256 threads.
constexpr int64_t kQuantDim = int64_t(1) << 28;
constexpr int64_t kQuantElems = int64_t(1) << 37;

int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

}  // namespace

extern "C" {

int agmm_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, int format,
                  int block_rows, void* q, int64_t ldq, float* scale, void* qt, int64_t ldqt,
                  float* scale_t, void* stream) {
  if (!x) return set_err(AGMM_ERR_INVALID_ARG, "x is NULL");
  if (dtype != AGMM_BF16 && dtype != AGMM_FP16 && dtype != AGMM_FP32)
    return set_err(AGMM_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (format != AGMM_E4M3 && format != AGMM_E5M2)
    return set_err(AGMM_ERR_INVALID_ARG, "unknown 8-bit format %d", format);
  if (block_rows != 1 && block_rows != agmm::kScaleBlock)
    return set_err(AGMM_ERR_INVALID_ARG, "block_rows must be 1 or %d (got %d)", agmm::kScaleBlock, block_rows);
  if (rows < 1 || cols < 1)
    return set_err(AGMM_ERR_INVALID_ARG, "sizes must be >= 1 (rows=%lld, cols=%lld)", (long long)rows, (long long)cols);
  if (rows >= kQuantDim || cols >= kQuantDim || rows * cols >= kQuantElems)
    return set_err(AGMM_ERR_UNSUPPORTED, "matrix too large (rows=%lld, cols=%lld)", (long long)rows, (long long)cols);
  if (ldx < cols) return set_err(AGMM_ERR_INVALID_ARG, "ldx %lld is less than cols %lld", (long long)ldx, (long long)cols);
  if (!q && !qt) return set_err(AGMM_ERR_INVALID_ARG, "q and qt are both NULL");
  const int64_t es = dtype == AGMM_FP32 ? 4 : 2;
  if (!aligned(x, es)) return set_err(AGMM_ERR_UNSUPPORTED, "x is not aligned to its elements");
  agmm::QuantProblem p{};
  p.cols16 = round_up(cols, 16);
  p.rows16 = round_up(rows, 16);
  struct Out { const char* name; void* v; int64_t ld; float* s; int64_t need; };
  for (const Out& o : {Out{"q", q, ldq, scale, p.cols16}, Out{"qt", qt, ldqt, scale_t, p.rows16}}) {
    if (!o.v) continue;
    if (!o.s) return set_err(AGMM_ERR_INVALID_ARG, "%s has no scale array", o.name);
    if (o.ld < o.need)
      return set_err(AGMM_ERR_INVALID_ARG, "ld%s %lld is less than the row length rounded up to 16, %lld", o.name,
                     (long long)o.ld, (long long)o.need);
    if (!aligned(o.v, 16) || o.ld % 16 != 0 || !aligned(o.s, 4))
      return set_err(AGMM_ERR_UNSUPPORTED, "%s and its rows must be 16-byte aligned, its scales 4-byte aligned", o.name);
  }
  p.x = x;
  p.rows = rows;
  p.cols = cols;
  p.ldx = ldx;
  p.dtype = dtype;
  p.format = format;
  p.block_rows = block_rows;
  p.q = q;
  p.ldq = ldq;
  p.scale = scale;
  p.qt = qt;
  p.ldqt = ldqt;
  p.scale_t = scale_t;
  const hipError_t err = agmm::launch_quantize(p, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? ok() : hip_err(err, "quantiser launch");
}

}  // extern "C"
