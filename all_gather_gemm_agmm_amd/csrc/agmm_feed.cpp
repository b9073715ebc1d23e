// C ABI of the feed-forward block's operators (host side): the product with an
// epilogue and the gated product, their way back, and layer norm.  Their plans
// are used as those of agmm_ops.cpp are.
#include <initializer_list>
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <string>

#include "agmm.h"
#include "feed_kernels.h"
#include "ops_kernels.h"
#include "plan_base.h"

namespace {

using agmm::aligned;
using agmm::cdiv;
using agmm::check_ptr;
using agmm::check_sizes;
using agmm::Cut;
using agmm::group_rows;
using agmm::hip_err;
using agmm::kDimLimit;
using agmm::ok;
using agmm::PlanBase;
using agmm::round_up;
using agmm::set_err;

int validate_ff(int N, int64_t m_s, int64_t k, int64_t n, int dtype, int act, int gated) {
  const int rc = check_sizes(N, m_s, k, n);
  if (rc != AGMM_OK) return rc;
  if (dtype == AGMM_FP32)
    return set_err(AGMM_ERR_UNSUPPORTED, "the feed-forward product takes bf16 or fp16 operands");
  if (dtype != AGMM_BF16 && dtype != AGMM_FP16) return set_err(AGMM_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (act < AGMM_ACT_NONE || act > AGMM_ACT_SILU) return set_err(AGMM_ERR_INVALID_ARG, "unknown activation %d", act);
  if (gated != 0 && gated != 1) return set_err(AGMM_ERR_INVALID_ARG, "gated must be 0 or 1 (got %d)", gated);
  // every launch then stays within kFeedGrid by its smallest tile but the few-row
  // form, which is chosen only where it fits
  const int64_t m = N * m_s, cols = (1 + gated) * n;
  if (m >= (int64_t(1) << 27) || cols >= (int64_t(1) << 27) || m * cols >= (int64_t(1) << 36) || m * k >= (int64_t(1) << 36) ||
      cols * k >= (int64_t(1) << 36))
    return set_err(AGMM_ERR_UNSUPPORTED, "problem too large (m=%lld, k=%lld, n_local=%lld)", (long long)m, (long long)k, (long long)n);
  return ok();
}

agmm::Activation activation_of(int act) {
  const float c = 1.5957691216057308f;   // sqrt(8 / pi)
  switch (act) {
    case AGMM_ACT_RELU: return {agmm::kActRelu, 0.0f, 0.0f};
    case AGMM_ACT_GELU: return {agmm::kActNormal, 0.0f, 0.0f};
    case AGMM_ACT_GELU_TANH: return {agmm::kActLogistic, c, c * 0.044715f};   // x (1 + tanh u) / 2 = x / (1 + exp(-2 u))
    case AGMM_ACT_SILU: return {agmm::kActSilu, 0.0f, 0.0f};
    default: return {agmm::kActLinear, 0.0f, 0.0f};
  }
}

}  // namespace

struct agmm_ff_plan : PlanBase {
  int N = 0;
  int64_t m_s = 0, k = 0, n = 0, m = 0;
  int dtype = 0, act = 0, parts = 1;
  bool with_gradient = true;
  int64_t lda = 0, ldw = 0, ldr = 0, ldy = 0, lddy = 0, ldda = 0, lddw = 0;   // 0: dense
  int64_t tile_key = -1;                          // 64 (few rows), 128, 256; -1: automatic

  // What a call of a pass uses, derived from the settings.
  struct Layout {
    bool pad_a = false, pad_w = false;   // zero-padded copies
    int64_t kp = 0;                      // row length of a copy: whole 128-byte lines
    int tile = 256;                      // forward; 64: the few-row form, in
    int splits = 1;                      // ranges of k (tile 128)
    int64_t per = 0;
    int fm = 0, yc = 0;                  // blocks of 16 fm rows x yc columns of y (kept pre-activations: most_yc())
    int d_rows = 128;                    // rows of a workgroup of the elementwise part
    bool groups = false;                 // dW's product reads A in the shards
    int tile_grads = 256;
    int a_ranges = 1, w_ranges = 1;      // ranges of the gradient products' sums
    int64_t a_per = 0, w_per = 0;
    char *a = nullptr, *w = nullptr, *d = nullptr, *dt = nullptr;
    float *parts = nullptr, *a_sums = nullptr, *w_sums = nullptr, *b_sums = nullptr;
    size_t bytes = 0;
  };
  // those of the settings and the workspace: forward, forward with pre-activations
  // kept in 16 bits, in 8 bits, backward
  enum Pass { kForward, kKeep16, kKeep8, kBackward };
  Layout layouts[4];
  static Pass forward_pass(const void* saved, const void* scales) { return !saved ? kForward : scales ? kKeep8 : kKeep16; }
  int passes() const { return with_gradient ? kBackward + 1 : kBackward; }

  int64_t ld_a() const { return lda ? lda : k; }
  int64_t ld_w() const { return ldw ? ldw : k; }
  // Row lengths of d and d transposed: whole 128-byte lines.
  int64_t ld_d() const { return round_up(cols(), 64); }
  int64_t ld_dt() const { return round_up(m, 64); }
  int64_t cols() const { return parts * n; }
  int64_t wide() const { return round_up(n, agmm::kKeptBlock); }
  // Columns of the forward product's tiles (feed_kernels.h).
  int64_t tile_cols() const { return parts == 2 ? 2 * round_up(n, 16) : n; }

  // Microseconds of the products' tiles, measured on MI355X: of a launch of
  // `tiles` of them, each over `sum` elements of k.  A 256 x 256 tile has a CU to
  // itself, 17 and 1.1 per 64 of its sum, 0.93 where half the CUs have none, and
  // 256 x 224 seven eighths of that; a 128 x 128 one shares it, 5 and 0.92, in the
  // last round less, or has it alone, 0.48.  `lines`: the operands' rows start on
  // 128-byte lines; where they do not, a tile's loads take twice the lines
  // (1011 x 4040 -> 2 x 2051: 64 us, 40 at 4096).
  double tiles_us(int t, int64_t tiles, int64_t sum, bool lines) const {
    const double steps = (double)cdiv(sum, 64);
    if (t >= 224)
      return (double)cdiv(tiles, cu_count) * (17.0 + t / 256.0 * (2 * tiles <= cu_count ? 0.93 : 1.1) * steps * (lines ? 1.0 : 1.25));
    const int64_t rest = tiles % (2 * cu_count);
    const double by = steps * (lines ? 1.0 : tiles <= cu_count ? 1.55 : 1.4);
    const double last = rest <= cu_count ? 0.48 : 0.78 + 0.14 * ((double)rest / cu_count - 1.0);
    return (double)(tiles / (2 * cu_count)) * (5.0 + 0.92 * by) + (rest == 0 ? 0.0 : 5.0 + last * by);
  }

  // Microseconds of copies of A and W as rows of whole lines.
  double copy_us() const { return 5.0 + (double)(m + cols()) * (double)k * 4 / 6.5e6; }

  // The few-row form in blocks of yc columns of y: 4.5 and 21 per MB of a CU's
  // rows and columns (27 where four waves share out k, 1.7 times that for odd
  // strides), with 2.7 for every further workgroup of 64 rows on a CU, 4.9 where k
  // ends inside 64, or W at 4.5 TB/s, and a tenth of the other.  E.g. (us) 8 x 4096
  // -> 1792: 7.8 by 8 columns, 8.7 by 16, 21 by 64; 128 x 4096 -> 7168: 73 by 16,
  // 35 by 64, 22 in tiles of 128; 8 x 8192 -> 3584: 24 by 8, 16 by 16; 3000 x 130 ->
  // 6307: 114 by 64, 30 in tiles of 128.  (Calls back to back in a graph.)
  double few_us(int fm, int yc, int splits) const {
    const double mb = 2e-6 * (double)cdiv(k, splits) * (double)(std::min<int64_t>(m, 16 * fm) + parts * yc);
    const double each = (fm == 1 && yc <= 16 ? 21.0 : 27.0) * (ld_a() % 2 != 0 || ld_w() % 2 != 0 ? 1.7 : 1.0);
    const int64_t wgs = cdiv(m, 16 * fm) * cdiv(n, yc) * splits;
    const double turns = (double)cdiv(wgs, cu_count), more = fm == 1 ? 0.0 : (turns - 1.0) * (k % 64 == 0 ? 2.7 : 4.9);
    const double in = 4.5 + more + turns * each * mb, read = 2.0 + (double)cols() * (double)k * 2 / 4.5e6;
    return std::max(in, read) + 0.1 * std::min(in, read);
  }

  // Form of the forward product: the one that takes the least, with the copies
  // it needs.  Copies have rows of whole lines; rows that are whole 16-byte
  // vectors already are copied where that pays.  8-bit pre-activations of a gated
  // product come in no tile of 224 (feed_kernels.h): asked for, it is 256.
  void pick_tile(Layout& L, bool must_copy, Pass pass) const {
    const int64_t nc = tile_cols();
    const bool kept = pass != kForward, no_224 = pass == kKeep8 && parts == 2;
    const int64_t want = tile_key == 224 && no_224 ? 256 : tile_key;
    const bool lines = ld_a() % 64 == 0 && ld_w() % 64 == 0;
    double best = -1;
    const auto offer = [&](int tile, bool copied, int splits, double us) {
      if ((want > 0 && tile != want) || (tile == 224 && no_224)) return;
      us += copied ? copy_us() : 0.0;
      if (best >= 0 && us >= best) return;
      best = us;
      L.tile = tile;
      L.splits = splits;
      L.pad_a = L.pad_w = copied;
    };
    for (bool copied : {false, true}) {
      if (!copied && must_copy) continue;
      if (copied && !must_copy && lines) continue;
      for (int t : {256, 224}) offer(t, copied, 1, tiles_us(t, cdiv(m, 256) * cdiv(nc, t), k, lines || copied));
      const int64_t tiles = cdiv(m, 128) * cdiv(nc, 128);
      for (int s : {1, 2, 3, 4, 6, 8, 12, 16}) {
        if (s > 1 && (k < 256 * s || tiles * s > 4 * cu_count)) break;
        offer(128, copied, s, tiles_us(128, tiles * s, cdiv(k, s), lines || copied) + (s > 1 ? join_us(s, 4.0) : 0.0));
      }
    }
    L.fm = m <= 16 ? 1 : 4;
    if (!few_fits()) return;
    double few = -1;
    int ranges = 1;
    for (int yc : {8, 16, most_yc()}) {
      if (yc == 8 && L.fm > 1) continue;
      const int64_t blocks = cdiv(m, 16 * L.fm) * cdiv(n, yc);
      for (int s : {1, 2, 3, 4, 6, 8, 12, 16}) {
        if (s == 1 && kept && yc != most_yc()) continue;   // blocks of 32 kept columns lie in one workgroup
        if (s > 1 && (yc == 8 || k < 256 * s || blocks * s > 2 * cu_count)) break;
        const double us = few_us(L.fm, yc, s) + (s > 1 ? join_us(s, 5.0) : 0.0);
        if (few < 0 || us < few) few = us, L.yc = yc, ranges = s;
      }
    }
    offer(64, false, ranges, few);
  }

  // Microseconds of adding ranges of k: the launch (5 behind the few-row form, whose
  // own is short), and the sums written and read at 4 TB/s.
  double join_us(int splits, double launch) const { return launch + (double)(splits * m) * (double)tile_cols() * 8 / 4e6; }

  int most_yc() const { return parts == 2 ? 32 : 64; }

  // Whether every form of the few-row kernel stays within a launch.
  bool few_fits() const { return cdiv(m, m <= 16 ? 16 : 64) * cdiv(n, m <= 16 ? 8 : 16) < agmm::kFeedGrid; }

  Layout layout(Pass pass, char* base) const {
    Layout L;
    L.kp = round_up(k, 64);
    const bool must_a = k % 8 != 0 || ld_a() % 8 != 0, must_w = k % 8 != 0 || ld_w() % 8 != 0;   // not whole 16-byte vectors
    Cut c{base};
    if (pass != kBackward) {
      pick_tile(L, must_a || must_w, pass);
      if (L.pad_a) L.a = c.take((size_t)m * L.kp * 2);
      if (L.pad_w) L.w = c.take((size_t)cols() * L.kp * 2);
      L.per = round_up(cdiv(L.pad_a ? L.kp : k, L.splits), 64);
      L.splits = (int)cdiv(k, L.per);
      if (L.splits > 1) L.parts = reinterpret_cast<float*>(c.take((size_t)L.splits * m * round_up(tile_cols(), 16) * 4));
    } else {
      L.pad_a = must_a;
      L.pad_w = must_w;
      // dW's product reads A k x n: in the shards where they are whole k-tiles,
      // else in one piece
      L.groups = N > 1 && !L.pad_a && m_s % 64 == 0;
      if (L.pad_a || (N > 1 && !L.groups)) L.a = c.take((size_t)m * L.kp * 2);
      if (L.pad_w) L.w = c.take((size_t)cols() * L.kp * 2);
      L.d = c.take((size_t)m * ld_d() * 2);
      L.dt = c.take((size_t)cols() * ld_dt() * 2);
      L.d_rows = cdiv(m, 128) * cdiv(n, agmm::kDCols) >= 2 * cu_count ? 128 : 32;
      L.b_sums = reinterpret_cast<float*>(c.take((size_t)cdiv(m, L.d_rows) * cols() * 4));
      // One launch computes both products; each sum may be cut into ranges.
      // Tile and ranges are those that take the least: the workgroups' time
      // spread over the CUs and half of one for the last round, but no less than
      // the longest of them; and the ranges' sums, written and read at 4 TB/s,
      // with a launch more.
      double best = -1;
      int64_t want_a = 1, want_w = 1;
      for (int t : {256, 128}) {
        if (tile_key > 64 && t != (tile_key == 224 ? 256 : tile_key)) continue;
        const int64_t a_tiles = cdiv(m, t) * cdiv(k, t), w_tiles = cdiv(cols(), t) * cdiv(k, t);
        const double slots = cu_count * (t == 128 ? 2 : 1);
        const auto one = [&](int64_t sum) { return t == 256 ? 10.0 + 1.4 * (double)cdiv(sum, 64) : 5.0 + 0.92 * (double)cdiv(sum, 64); };
        for (int64_t ra = 1; ra == 1 || (ra <= 64 && a_tiles * ra <= 4 * cu_count && cols() / ra >= 256); ra *= 2)
          for (int64_t rw = 1; rw == 1 || (rw <= 64 && w_tiles * rw <= 4 * cu_count && m / rw >= 256); rw *= 2) {
            const double a_us = one(cdiv(cols(), ra)), w_us = one(cdiv(m, rw));
            const double sums = (ra > 1 ? (double)(ra * m) : 0.0) + (rw > 1 ? (double)(rw * cols()) : 0.0);
            const double us = std::max({((double)(a_tiles * ra) * a_us + (double)(w_tiles * rw) * w_us) / slots + w_us / 2, a_us, w_us}) +
                              sums * (double)k * 8 / 4e6 + (sums > 0 ? 3.0 : 0.0);
            if (best < 0 || us < best) best = us, L.tile_grads = t, want_a = ra, want_w = rw;
          }
      }
      L.a_per = round_up(cdiv(cols(), want_a), 64);
      L.a_ranges = (int)cdiv(cols(), L.a_per);
      L.w_per = round_up(cdiv(m, want_w), 64);
      L.w_ranges = (int)cdiv(m, L.w_per);
      if (L.a_ranges > 1) L.a_sums = reinterpret_cast<float*>(c.take((size_t)L.a_ranges * m * round_up(k, 4) * 4));
      if (L.w_ranges > 1) L.w_sums = reinterpret_cast<float*>(c.take((size_t)L.w_ranges * cols() * round_up(k, 4) * 4));
    }
    L.bytes = c.at;
    return L;
  }

  int apply() {
    size_t bytes = 0;
    for (int pass = 0; pass < passes(); ++pass) bytes = std::max(bytes, layout((Pass)pass, nullptr).bytes);
    const int rc = reserve(bytes);
    if (rc != AGMM_OK) return rc;
    for (int pass = 0; pass < passes(); ++pass) layouts[pass] = layout((Pass)pass, ws);
    return AGMM_OK;
  }

  agmm::TileOrder tiles_of(int64_t rows, int64_t columns, int tile_rows, int tile_columns) const {
    agmm::TileOrder o{};
    o.num_rb = (int32_t)cdiv(rows, tile_rows);
    o.num_cb = (int32_t)cdiv(columns, tile_columns);
    o.group_m = group_rows(o.num_rb, o.num_cb);
    o.xcd_remap = 1;
    return o;
  }

  static agmm::RowMap dense(const void* a, int64_t rows, int64_t ld) {
    agmm::RowMap r{};
    r.a_group[0] = a;
    r.a_ld = ld;
    r.rows_per_group = (int32_t)rows;
    r.num_groups = 1;
    return r;
  }

  // The copies of A (shards not NULL) and W that the layout has.
  agmm::FeedCopies copies(const Layout& L, const void* const* shards, const void* W) const {
    const auto copy = [&](const void* const* groups, int count, int64_t rows, int64_t ld, void* out) {
      agmm::PadRows c{};
      for (int g = 0; g < count; ++g) c.group[g] = groups[g];
      c.num_groups = count;
      c.rows = rows;
      c.cols = k;
      c.ld = ld;
      c.chunks = L.kp / 8;
      c.out = out;
      return c;
    };
    agmm::FeedCopies c{};
    if (L.a && shards) c.a = copy(shards, N, m_s, ld_a(), L.a);
    if (L.w && W) c.w = copy(&W, 1, cols(), ld_w(), L.w);
    return c;
  }

  agmm::KeptRows kept_rows(const void* values, const void* scales) const {
    return {const_cast<void*>(values), static_cast<uint8_t*>(const_cast<void*>(scales)), wide()};
  }

  int forward(const void* const* shards, const void* W, const void* bias, const void* residual, void* Y,
              void* saved, void* saved_scales, hipStream_t s) {
    const Layout& L = layouts[forward_pass(saved, saved_scales)];
    if (L.a || L.w) {
      const hipError_t err = agmm::launch_feed_copies(copies(L, shards, W), s);
      if (err != hipSuccess) return hip_err(err, "operand copy launch");
    }
    agmm::FeedProblem p{};
    if (L.a) {
      p.gemm.rows = dense(L.a, m, L.kp);
    } else {
      for (int g = 0; g < N; ++g) p.gemm.rows.a_group[g] = shards[g];
      p.gemm.rows.a_ld = ld_a();
      p.gemm.rows.rows_per_group = (int32_t)m_s;
      p.gemm.rows.num_groups = N;
      p.gemm.rows.c_group_rows = m_s;
    }
    if (L.tile == 64) {
      p.gemm.order.num_rb = (int32_t)cdiv(m, 16 * L.fm);
      p.gemm.order.num_cb = (int32_t)cdiv(n, L.yc);
    } else {
      p.gemm.order = tiles_of(m, tile_cols(), L.tile == 224 ? 256 : L.tile, L.tile);
    }
    p.gemm.m = (int32_t)m;
    p.gemm.n = (int32_t)tile_cols();
    p.gemm.k = (int32_t)(L.w ? L.kp : k);
    p.gemm.b = L.w ? L.w : W;
    p.gemm.ldb = L.w ? L.kp : ld_w();
    p.gemm.splits = L.splits;
    p.gemm.k_per_split = (int32_t)L.per;
    p.gemm.partials = L.parts;
    p.n = (int32_t)n;
    p.gated = parts == 2;
    p.act = activation_of(act);
    p.bias = bias;
    p.residual = residual;
    p.ldr = ldr ? ldr : n;
    p.y = Y;
    p.ldy = ldy ? ldy : n;
    p.kept = kept_rows(saved, saved_scales);
    const hipError_t err = L.tile == 64 ? agmm::launch_feed_few(p, L.fm, L.yc, dtype, s) : agmm::launch_feed_tiles(p, L.tile, dtype, s);
    return err == hipSuccess ? AGMM_OK : hip_err(err, "feed-forward launch");
  }

  int backward(const void* const* shards, const void* W, const void* saved, const void* saved_scales, const void* dY, void* dA,
               void* dW, void* dbias, hipStream_t s) {
    const Layout& L = layouts[kBackward];
    agmm::FeedDProblem e{};
    e.block = L.d_rows;
    e.m = m;
    e.n = (int32_t)n;
    e.gated = parts == 2;
    e.act = activation_of(act);
    e.kept = kept_rows(saved, saved_scales);
    e.dy = dY;
    e.lddy = lddy ? lddy : n;
    e.d = dA ? L.d : nullptr;
    e.ldd = ld_d();
    e.dt = dW ? L.dt : nullptr;
    e.ldt = ld_dt();
    e.sums = dbias ? L.b_sums : nullptr;
    hipError_t err = agmm::launch_feed_d(e, copies(L, dW ? shards : nullptr, dA ? W : nullptr), dtype, s);
    if (err != hipSuccess) return hip_err(err, "feed-forward gradient launch");
    agmm::FeedGrads g{};
    agmm::GemmProblem &ga = g.a, &gw = g.w;
    ga.rows = dense(L.d, m, e.ldd);
    ga.order = tiles_of(m, k, L.tile_grads, L.tile_grads);
    ga.m = (int32_t)m;
    ga.n = (int32_t)k;
    ga.k = (int32_t)cols();
    ga.b = L.w ? L.w : W;
    ga.ldb = L.w ? L.kp : ld_w();
    ga.splits = L.a_ranges;
    ga.k_per_split = (int32_t)L.a_per;
    ga.partials = L.a_sums;
    ga.c = dA;
    ga.ldc = ldda ? ldda : k;
    gw.rows = dense(L.dt, cols(), ld_dt());
    gw.order = tiles_of(cols(), k, L.tile_grads, L.tile_grads);
    gw.m = (int32_t)cols();
    gw.n = (int32_t)k;
    gw.k = (int32_t)m;
    gw.b = L.a ? L.a : shards ? shards[0] : nullptr;
    gw.ldb = L.a ? L.kp : ld_a();
    gw.splits = L.w_ranges;
    gw.k_per_split = (int32_t)L.w_per;
    gw.partials = L.w_sums;
    gw.c = dW;
    gw.ldc = lddw ? lddw : k;
    if (L.groups)
      for (int r = 0; r < N && shards; ++r) g.w_group[r] = shards[r];
    g.w_rows = L.groups ? (int32_t)m_s : 0;
    if (!dA) ga.m = 0;
    if (!dW) gw.m = 0;
    if (dbias) g.bias = {L.b_sums, cdiv(m, L.d_rows), cols(), dbias};
    err = agmm::launch_feed_grads(g, L.tile_grads, dtype, s);
    if (err != hipSuccess) return hip_err(err, "gradient products launch");
    const auto ranges = [&](const agmm::GemmProblem& g) { return agmm::SumRanges{g.partials, g.splits, g.m, g.n, g.c, g.ldc}; };
    const agmm::SumRanges sa = ranges(ga), sw = ranges(gw);
    const bool more_a = dA && L.a_ranges > 1, more_w = dW && L.w_ranges > 1;
    if (more_a || more_w) {
      err = agmm::launch_sum_ranges(more_a ? &sa : nullptr, more_w ? &sw : nullptr, dtype, s);
      if (err != hipSuccess) return hip_err(err, "gradient sums launch");
    }
    return AGMM_OK;
  }
};

namespace {

// Rows and columns: a launch of the column sums stays below 2^22 workgroups of
// 1024 threads.
constexpr int64_t kNormRows = int64_t(1) << 28;
constexpr int64_t kNormCols = int64_t(1) << 26;
constexpr int64_t kNormElems = int64_t(1) << 37;

int validate_norm(int64_t rows, int64_t cols, int dtype, int wtype) {
  if (rows < 1 || cols < 1)
    return set_err(AGMM_ERR_INVALID_ARG, "sizes must be >= 1 (rows=%lld, cols=%lld)", (long long)rows, (long long)cols);
  if (dtype != AGMM_BF16 && dtype != AGMM_FP16 && dtype != AGMM_FP32) return set_err(AGMM_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (wtype != AGMM_BF16 && wtype != AGMM_FP16 && wtype != AGMM_FP32)
    return set_err(AGMM_ERR_INVALID_ARG, "unknown weight dtype %d", wtype);
  if (wtype != dtype && wtype != AGMM_FP32)
    return set_err(AGMM_ERR_UNSUPPORTED, "weights have the rows' dtype %d or fp32 (got %d)", dtype, wtype);
  if (rows >= kNormRows || cols >= kNormCols || rows * cols >= kNormElems)
    return set_err(AGMM_ERR_UNSUPPORTED, "matrix too large (rows=%lld, cols=%lld)", (long long)rows, (long long)cols);
  return ok();
}

}  // namespace

struct agmm_norm_plan : PlanBase {
  int64_t rows = 0, cols = 0;
  int dtype = 0, wtype = 0, groups = 0;
  int64_t ldx = 0, ldy = 0, lddy = 0, lddx = 0;   // 0: dense
  uintptr_t elem() const { return dtype == AGMM_FP32 ? 4 : 2; }
  uintptr_t weight_elem() const { return wtype == AGMM_FP32 ? 4 : 2; }
  agmm::NormProblem problem(const void* x, const void* weight) const {
    agmm::NormProblem p{};
    p.rows = rows;
    p.cols = cols;
    p.dtype = dtype;
    p.wtype = wtype;
    p.cus = cu_count;
    p.x = x;
    p.ldx = ldx ? ldx : cols;
    p.weight = weight;
    p.groups = groups;
    return p;
  }
};

extern "C" {

int agmm_ff_plan_validate(int num_shards, int64_t m_per_shard, int64_t k, int64_t n_local, int dtype, int activation, int gated) {
  return validate_ff(num_shards, m_per_shard, k, n_local, dtype, activation, gated);
}

agmm_ff_plan_t agmm_ff_plan_create(int num_shards, int64_t m_per_shard, int64_t k, int64_t n_local, int dtype, int activation,
                                   int gated, int with_gradient) {
  if (validate_ff(num_shards, m_per_shard, k, n_local, dtype, activation, gated) != AGMM_OK) return nullptr;
  agmm_ff_plan* p = new (std::nothrow) agmm_ff_plan();
  if (!p) {
    set_err(AGMM_ERR_OOM, "out of host memory");
    return nullptr;
  }
  p->N = num_shards;
  p->m_s = m_per_shard;
  p->k = k;
  p->n = n_local;
  p->m = num_shards * m_per_shard;
  p->dtype = dtype;
  p->act = activation;
  p->parts = 1 + gated;
  p->with_gradient = with_gradient != 0;
  if (p->init() != AGMM_OK || p->apply() != AGMM_OK) {
    const int st = agmm::g_status;
    const std::string msg = agmm::g_msg;
    delete p;
    set_err(st, "%s", msg.c_str());
    return nullptr;
  }
  ok();
  return p;
}

int agmm_ff_plan_set_int(agmm_ff_plan_t p, const char* key, int64_t v) {
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "plan is NULL");
  if (!key) return set_err(AGMM_ERR_INVALID_ARG, "key is NULL");
  std::lock_guard<std::mutex> lk(p->mu);
  if (p->captured)
    return set_err(AGMM_ERR_UNSUPPORTED,
                   "the plan has been captured into a graph; its settings are fixed (create a new plan)");
  const std::string k(key);
  const auto bad = [&]() {
    return set_err(AGMM_ERR_INVALID_ARG, "value %lld out of range for key '%s'", (long long)v, key);
  };
  int64_t* field = nullptr;
  if (k == "lda" || k == "ldw" || k == "ldda" || k == "lddw") {
    if (v != 0 && (v < p->k || v >= kDimLimit)) return bad();
    field = k == "lda" ? &p->lda : k == "ldw" ? &p->ldw : k == "ldda" ? &p->ldda : &p->lddw;
  } else if (k == "ldr" || k == "ldy" || k == "lddy") {
    if (v != 0 && (v < p->n || v >= kDimLimit)) return bad();
    field = k == "ldr" ? &p->ldr : k == "ldy" ? &p->ldy : &p->lddy;
  } else if (k == "tile") {
    if (v != -1 && v != 64 && v != 128 && v != 224 && v != 256) return bad();
    if (v == 64 && !p->few_fits()) return set_err(AGMM_ERR_UNSUPPORTED, "too many workgroups for tile 64");
    field = &p->tile_key;
  } else {
    return set_err(AGMM_ERR_INVALID_ARG, "unknown key '%s'", key);
  }
  const int64_t old = *field;
  *field = v;
  if (p->apply() != AGMM_OK) {   // the plan keeps its settings and workspace
    *field = old;
    return agmm::g_status;
  }
  return ok();
}

int agmm_ff_plan_get_int(agmm_ff_plan_t p, const char* key, int64_t* value) {
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "plan is NULL");
  if (!key || !value) return set_err(AGMM_ERR_INVALID_ARG, "key or value is NULL");
  std::lock_guard<std::mutex> lk(p->mu);
  const std::string k(key);
  if (k == "lda") *value = p->ld_a();
  else if (k == "ldw") *value = p->ld_w();
  else if (k == "ldda") *value = p->ldda ? p->ldda : p->k;
  else if (k == "lddw") *value = p->lddw ? p->lddw : p->k;
  else if (k == "ldr") *value = p->ldr ? p->ldr : p->n;
  else if (k == "ldy") *value = p->ldy ? p->ldy : p->n;
  else if (k == "lddy") *value = p->lddy ? p->lddy : p->n;
  else if (k == "saved_cols") *value = p->wide();
  else if (k == "tile") *value = p->layouts[agmm_ff_plan::kForward].tile;
  else if (k == "captured") *value = p->captured;
  else return set_err(AGMM_ERR_INVALID_ARG, "unknown key '%s'", key);
  return ok();
}

size_t agmm_ff_plan_workspace_bytes(agmm_ff_plan_t p) { return p ? p->ws_bytes : 0; }

// An output at the address of an input, or of another output (a partial overlap
// is the caller's to avoid).
static int check_apart(const void* out, const char* name, std::initializer_list<const void*> others, const void* const* shards = nullptr,
                       int N = 0) {
  if (!out) return AGMM_OK;
  bool same = std::find(others.begin(), others.end(), out) != others.end();
  for (int r = 0; r < N && shards; ++r) same = same || shards[r] == out;
  return same ? set_err(AGMM_ERR_INVALID_ARG, "%s overlaps an operand of the call", name) : AGMM_OK;
}

int agmm_ff_forward(agmm_ff_plan_t p, const void* const* shard_ptrs, const void* W, const void* bias, const void* residual, void* Y,
                    void* saved, void* saved_scales, void* stream) {
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "plan is NULL");
  if (!shard_ptrs) return set_err(AGMM_ERR_INVALID_ARG, "shard_ptrs is NULL");
  int rc = AGMM_OK;
  for (int r = 0; r < p->N && rc == AGMM_OK; ++r) rc = check_ptr(shard_ptrs[r], "shard_ptrs", r, 16);
  if (rc == AGMM_OK) rc = check_ptr(W, "W", -1, 16);
  if (rc == AGMM_OK && bias) rc = check_ptr(bias, "bias", -1, 2);
  if (rc == AGMM_OK && residual) rc = check_ptr(residual, "residual", -1, 2);
  if (rc == AGMM_OK) rc = check_ptr(Y, "Y", -1, 2);
  if (rc == AGMM_OK && saved) rc = check_ptr(saved, "saved", -1, 16);
  if (rc != AGMM_OK) return rc;
  if (residual && p->parts == 2) return set_err(AGMM_ERR_UNSUPPORTED, "a gated product takes no residual");
  if (saved_scales && !saved) return set_err(AGMM_ERR_INVALID_ARG, "saved_scales without saved");
  rc = check_apart(Y, "Y", {W, bias, saved, saved_scales}, shard_ptrs, p->N);
  if (rc == AGMM_OK) rc = check_apart(saved, "saved", {W, bias, residual, saved_scales}, shard_ptrs, p->N);
  if (rc == AGMM_OK) rc = check_apart(saved_scales, "saved_scales", {W, bias, residual}, shard_ptrs, p->N);
  if (rc != AGMM_OK) return rc;
  std::lock_guard<std::mutex> lk(p->mu);
  if (residual == Y && (p->ldr ? p->ldr : p->n) != (p->ldy ? p->ldy : p->n))
    return set_err(AGMM_ERR_INVALID_ARG, "Y over residual needs equal strides");
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool ordered = p->layouts[agmm_ff_plan::forward_pass(saved, saved_scales)].bytes > 0;
  return p->run(s, ordered, [&] { return p->forward(shard_ptrs, W, bias, residual, Y, saved, saved_scales, s); });
}

// Whether the plan's way back needs kept pre-activations.
static int check_saved(agmm_ff_plan_t p, const void* saved, const void* saved_scales) {
  if (!saved && saved_scales) return set_err(AGMM_ERR_INVALID_ARG, "saved_scales without saved");
  if (saved) return check_ptr(saved, "saved", -1, 16);
  if (p->parts == 2 || p->act != AGMM_ACT_NONE) return set_err(AGMM_ERR_INVALID_ARG, "saved is NULL");
  return AGMM_OK;
}

int agmm_ff_backward(agmm_ff_plan_t p, const void* const* shard_ptrs, const void* W, const void* saved, const void* saved_scales,
                     const void* dY, void* dA, void* dW, void* dbias, void* stream) {
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "plan is NULL");
  if (!p->with_gradient) return set_err(AGMM_ERR_UNSUPPORTED, "the plan was created without the gradient's workspace");
  if (!dA && !dW && !dbias) return set_err(AGMM_ERR_INVALID_ARG, "dA, dW and dbias are all NULL");
  int rc = AGMM_OK;
  if (dW) {
    if (!shard_ptrs) return set_err(AGMM_ERR_INVALID_ARG, "shard_ptrs is NULL");
    for (int r = 0; r < p->N && rc == AGMM_OK; ++r) rc = check_ptr(shard_ptrs[r], "shard_ptrs", r, 16);
  }
  if (rc == AGMM_OK && dA) rc = check_ptr(W, "W", -1, 16);
  if (rc == AGMM_OK) rc = check_saved(p, saved, saved_scales);
  if (rc == AGMM_OK) rc = check_ptr(dY, "dY", -1, 2);
  if (rc == AGMM_OK && dA) rc = check_ptr(dA, "dA", -1, 2);
  if (rc == AGMM_OK && dW) rc = check_ptr(dW, "dW", -1, 2);
  if (rc == AGMM_OK && dbias) rc = check_ptr(dbias, "dbias", -1, 2);
  if (rc == AGMM_OK) rc = check_apart(dA, "dA", {W, saved, saved_scales, dY, dW, dbias}, shard_ptrs, p->N);
  if (rc == AGMM_OK) rc = check_apart(dW, "dW", {W, saved, saved_scales, dY, dbias}, shard_ptrs, p->N);
  if (rc == AGMM_OK) rc = check_apart(dbias, "dbias", {W, saved, saved_scales, dY}, shard_ptrs, p->N);
  if (rc != AGMM_OK) return rc;
  std::lock_guard<std::mutex> lk(p->mu);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return p->run(s, true, [&] { return p->backward(shard_ptrs, W, saved, saved_scales, dY, dA, dW, dbias, s); });
}

int agmm_ff_recompute(agmm_ff_plan_t p, const void* saved, const void* saved_scales, void* Y, void* stream) {
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "plan is NULL");
  int rc = check_ptr(saved, "saved", -1, 16);
  if (rc == AGMM_OK) rc = check_ptr(Y, "Y", -1, 2);
  if (rc == AGMM_OK) rc = check_apart(Y, "Y", {saved, saved_scales});
  if (rc != AGMM_OK) return rc;
  std::lock_guard<std::mutex> lk(p->mu);
  hipStream_t s = static_cast<hipStream_t>(stream);
  agmm::FeedAgainProblem a{};
  a.m = p->m;
  a.n = (int32_t)p->n;
  a.gated = p->parts == 2;
  a.act = activation_of(p->act);
  a.kept = p->kept_rows(saved, saved_scales);
  a.y = Y;
  a.ldy = p->ldy ? p->ldy : p->n;
  return p->run(s, false, [&]() -> int {
    const hipError_t err = agmm::launch_feed_again(a, p->dtype, s);
    return err == hipSuccess ? AGMM_OK : hip_err(err, "recompute launch");
  });
}

void agmm_ff_plan_destroy(agmm_ff_plan_t p) { delete p; }

int agmm_norm_plan_validate(int64_t rows, int64_t cols, int dtype, int weight_dtype) {
  return validate_norm(rows, cols, dtype, weight_dtype);
}

agmm_norm_plan_t agmm_norm_plan_create(int64_t rows, int64_t cols, int dtype, int weight_dtype) {
  if (validate_norm(rows, cols, dtype, weight_dtype) != AGMM_OK) return nullptr;
  agmm_norm_plan* p = new (std::nothrow) agmm_norm_plan();
  if (!p) {
    set_err(AGMM_ERR_OOM, "out of host memory");
    return nullptr;
  }
  p->rows = rows;
  p->cols = cols;
  p->dtype = dtype;
  p->wtype = weight_dtype;
  int rc = p->init();
  if (rc == AGMM_OK) {
    p->groups = agmm::norm_groups(rows, cols, dtype, p->cu_count);
    if (!agmm::norm_direct(cols, dtype, p->groups)) rc = p->reserve((size_t)p->groups * 2 * cols * sizeof(float));
  }
  if (rc != AGMM_OK) {
    const int st = agmm::g_status;
    const std::string msg = agmm::g_msg;
    delete p;
    set_err(st, "%s", msg.c_str());
    return nullptr;
  }
  ok();
  return p;
}

int agmm_norm_plan_set_int(agmm_norm_plan_t p, const char* key, int64_t v) {
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "plan is NULL");
  if (!key) return set_err(AGMM_ERR_INVALID_ARG, "key is NULL");
  std::lock_guard<std::mutex> lk(p->mu);
  if (p->captured)
    return set_err(AGMM_ERR_UNSUPPORTED,
                   "the plan has been captured into a graph; its settings are fixed (create a new plan)");
  const std::string k(key);
  int64_t* field = k == "ldx" ? &p->ldx : k == "ldy" ? &p->ldy : k == "lddy" ? &p->lddy : k == "lddx" ? &p->lddx : nullptr;
  if (!field) return set_err(AGMM_ERR_INVALID_ARG, "unknown key '%s'", key);
  if (v != 0 && (v < p->cols || v >= kDimLimit))
    return set_err(AGMM_ERR_INVALID_ARG, "value %lld out of range for key '%s'", (long long)v, key);
  *field = v;
  return ok();
}

int agmm_norm_plan_get_int(agmm_norm_plan_t p, const char* key, int64_t* value) {
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "plan is NULL");
  if (!key || !value) return set_err(AGMM_ERR_INVALID_ARG, "key or value is NULL");
  std::lock_guard<std::mutex> lk(p->mu);
  const std::string k(key);
  if (k == "ldx") *value = p->ldx ? p->ldx : p->cols;
  else if (k == "ldy") *value = p->ldy ? p->ldy : p->cols;
  else if (k == "lddy") *value = p->lddy ? p->lddy : p->cols;
  else if (k == "lddx") *value = p->lddx ? p->lddx : p->cols;
  else if (k == "captured") *value = p->captured;
  else return set_err(AGMM_ERR_INVALID_ARG, "unknown key '%s'", key);
  return ok();
}

size_t agmm_norm_plan_workspace_bytes(agmm_norm_plan_t p) { return p ? p->ws_bytes : 0; }

int agmm_norm_forward(agmm_norm_plan_t p, const void* x, const void* weight, const void* bias, float eps, void* y, float* mean,
                      float* rstd, void* stream) {
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "plan is NULL");
  int rc = check_ptr(x, "x", -1, p->elem());
  if (rc == AGMM_OK && weight) rc = check_ptr(weight, "weight", -1, p->weight_elem());
  if (rc == AGMM_OK && bias) rc = check_ptr(bias, "bias", -1, p->weight_elem());
  if (rc == AGMM_OK) rc = check_ptr(y, "y", -1, p->elem());
  if (rc == AGMM_OK && mean) rc = check_ptr(mean, "mean", -1, 4);
  if (rc == AGMM_OK && rstd) rc = check_ptr(rstd, "rstd", -1, 4);
  if (rc == AGMM_OK) rc = check_apart(y, "y", {weight, bias, mean, rstd});
  if (rc == AGMM_OK) rc = check_apart(mean, "mean", {x, weight, bias, rstd});
  if (rc == AGMM_OK) rc = check_apart(rstd, "rstd", {x, weight, bias});
  if (rc != AGMM_OK) return rc;
  if (!(eps >= 0.0f) || std::isinf(eps)) return set_err(AGMM_ERR_INVALID_ARG, "eps must be a finite number >= 0 (got %g)", (double)eps);
  std::lock_guard<std::mutex> lk(p->mu);
  hipStream_t s = static_cast<hipStream_t>(stream);
  agmm::NormProblem n = p->problem(x, weight);
  if (y == x && n.ldx != (p->ldy ? p->ldy : p->cols)) return set_err(AGMM_ERR_INVALID_ARG, "y over x needs equal strides");
  n.bias = bias;
  n.eps = eps;
  n.y = y;
  n.ldy = p->ldy ? p->ldy : p->cols;
  n.mean = mean;
  n.rstd = rstd;
  return p->run(s, false, [&]() -> int {
    const hipError_t err = agmm::launch_norm_forward(n, s);
    return err == hipSuccess ? AGMM_OK : hip_err(err, "norm launch");
  });
}

int agmm_norm_backward(agmm_norm_plan_t p, const void* x, const void* dy, const void* weight, const float* mean, const float* rstd,
                       void* dx, void* dweight, void* dbias, void* stream) {
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "plan is NULL");
  if (!dx && !dweight && !dbias) return set_err(AGMM_ERR_INVALID_ARG, "dx, dweight and dbias are all NULL");
  int rc = check_ptr(x, "x", -1, p->elem());
  if (rc == AGMM_OK) rc = check_ptr(dy, "dy", -1, p->elem());
  if (rc == AGMM_OK && weight) rc = check_ptr(weight, "weight", -1, p->weight_elem());
  if (rc == AGMM_OK) rc = check_ptr(mean, "mean", -1, 4);
  if (rc == AGMM_OK) rc = check_ptr(rstd, "rstd", -1, 4);
  if (rc == AGMM_OK && dx) rc = check_ptr(dx, "dx", -1, p->elem());
  if (rc == AGMM_OK && dweight) rc = check_ptr(dweight, "dweight", -1, p->weight_elem());
  if (rc == AGMM_OK && dbias) rc = check_ptr(dbias, "dbias", -1, p->weight_elem());
  if (rc == AGMM_OK) rc = check_apart(dx, "dx", {x, weight, mean, rstd});
  if (rc == AGMM_OK) rc = check_apart(dweight, "dweight", {x, dy, weight, mean, rstd, dx, dbias});
  if (rc == AGMM_OK) rc = check_apart(dbias, "dbias", {x, dy, weight, mean, rstd, dx});
  if (rc != AGMM_OK) return rc;
  std::lock_guard<std::mutex> lk(p->mu);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool direct = agmm::norm_direct(p->cols, p->dtype, p->groups), sums = !direct && (dweight || dbias);
  agmm::NormProblem n = p->problem(x, weight);
  n.dy = dy;
  n.lddy = p->lddy ? p->lddy : p->cols;
  n.mean = const_cast<float*>(mean);
  n.rstd = const_cast<float*>(rstd);
  n.dx = dx;
  n.lddx = p->lddx ? p->lddx : p->cols;
  if (dx == dy && n.lddx != n.lddy) return set_err(AGMM_ERR_INVALID_ARG, "dx over dy needs equal strides");
  n.sums = sums ? reinterpret_cast<float*>(p->ws) : nullptr;
  n.dweight = direct ? dweight : nullptr;
  n.dbias = direct ? dbias : nullptr;
  return p->run(s, sums, [&]() -> int {
    hipError_t err = agmm::launch_norm_backward(n, s);
    if (err != hipSuccess) return hip_err(err, "norm gradient launch");
    if (!sums) return AGMM_OK;
    agmm::SumColumns c{};
    c.sums = n.sums;
    c.groups = p->groups;
    c.cols = 2 * p->cols;
    c.first = p->cols;
    c.out = dweight;
    c.out2 = dbias;
    c.dtype = p->wtype;
    err = agmm::launch_sum_columns(c, s);
    return err == hipSuccess ? AGMM_OK : hip_err(err, "norm weight gradient launch");
  });
}

void agmm_norm_plan_destroy(agmm_norm_plan_t p) { delete p; }

}  // extern "C"
