// C ABI of the operators around the all-gather matmul (host side): the
// block-scaled 8-bit quantiser and product, and the vocabulary loss.
//
// Their plans are used as the all-gather matmul's are: a plan validates its
// problem, owns a workspace when a call needs one, and orders its calls
// (CallOrder), so that calls on different streams or threads never share the
// workspace at one time.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <mutex>
#include <new>
#include <string>

#include "agmm.h"
#include "agmm_host.h"
#include "ops_kernels.h"

namespace {

using agmm::hip_err;
using agmm::ok;
using agmm::set_err;

// Rows and columns of a quantised matrix, and their product: every launch
// then stays below 2^24 workgroups of 256 threads.
constexpr int64_t kQuantDim = int64_t(1) << 28;
constexpr int64_t kQuantElems = int64_t(1) << 37;

int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

using agmm::kDimLimit;

// Shard counts and sizes every plan here accepts (the all-gather matmul's
// rules).
int check_sizes(int N, int64_t m_s, int64_t k, int64_t n) {
  const int rc = agmm::check_counts(N, m_s, k, n);
  return rc == AGMM_OK ? agmm::check_limits(N, m_s, k, n) : rc;
}

// What every plan here owns: its device, a workspace, and the order of its
// calls.
struct PlanBase {
  int device = 0;
  int cu_count = 256;
  char* ws = nullptr;
  size_t ws_bytes = 0;
  agmm::CallOrder order;
  bool captured = false;
  std::mutex mu;

  int init() {
    hipError_t err = hipGetDevice(&device);
    if (err != hipSuccess) return hip_err(err, "hipGetDevice");
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device) == hipSuccess && cus > 0)
      cu_count = cus;
    return order.create(device);
  }

  // Replace the workspace by one of at least `bytes` (kept when it is large
  // enough).  On failure the plan keeps the one it has.
  int reserve(size_t bytes) {
    if (bytes <= ws_bytes) return AGMM_OK;
    // test hook: AGMM_TEST_FAIL_ALLOC=<n> makes every workspace allocation of
    // more than n bytes fail (n = 0 or 1: all of them)
    if (const char* hook = std::getenv("AGMM_TEST_FAIL_ALLOC")) {
      const long long limit = std::atoll(hook);
      if (limit <= 1 || (long long)bytes > limit)
        return set_err(AGMM_ERR_OOM, "workspace allocation of %zu bytes failed (forced by test hook)", bytes);
    }
    void* q = nullptr;
    const hipError_t err = hipMalloc(&q, bytes);
    if (err != hipSuccess) {
      (void)hipGetLastError();
      return set_err(AGMM_ERR_OOM, "workspace allocation of %zu bytes failed: %s", bytes, hipGetErrorString(err));
    }
    const int rc = order.idle();   // the previous call may still use the old one
    if (rc != AGMM_OK) {
      hipFree(q);
      return rc;
    }
    if (ws) hipFree(ws);
    ws = static_cast<char*>(q);
    ws_bytes = bytes;
    return AGMM_OK;
  }

  // A call that enqueues work.  One that uses no workspace needs no ordering.
  template <class F>
  int run(hipStream_t s, bool ordered, F&& body) {
    agmm::Call c;
    int rc = agmm::CallOrder::look(s, c);
    if (rc == AGMM_OK && c.capturing) captured = true;
    if (rc == AGMM_OK && ordered) rc = order.enter(c);
    if (rc != AGMM_OK) return rc;
    rc = body();
    if (!ordered) return rc == AGMM_OK ? ok() : rc;
    if (rc != AGMM_OK) {
      // whatever was enqueued before the failure still counts
      const int st = agmm::g_status;
      const std::string msg = agmm::g_msg;
      order.leave(c);
      return set_err(st, "%s", msg.c_str());
    }
    rc = order.leave(c);
    return rc == AGMM_OK ? ok() : rc;
  }

  ~PlanBase() {
    (void)order.idle();
    (void)hipGetLastError();
    if (ws) hipFree(ws);
    order.destroy();
  }
};

// The shard and other pointers of a call: none NULL, all aligned.
int check_ptr(const void* p, const char* name, int index, uintptr_t to) {
  char label[64];
  if (index >= 0) snprintf(label, sizeof label, "%s[%d]", name, index);
  else snprintf(label, sizeof label, "%s", name);
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "%s is NULL", label);
  if (!aligned(p, to)) return set_err(AGMM_ERR_UNSUPPORTED, "%s is not %d-byte aligned", label, (int)to);
  return AGMM_OK;
}

// Row blocks of `rows` x `cols` tiles walked together: the grouping whose
// first XCD range touches the fewest row and column blocks (tiles of one XCD
// share its L2).
int group_rows(int64_t nrb, int64_t ncb) {
  const int64_t per = cdiv(nrb * ncb, 8);
  int best = 4;
  int64_t best_cost = INT64_MAX;
  for (int g : {4, 8, 2, 16, 1}) {
    int64_t t = 0, rows = 0, cols = 0;
    for (int64_t grp = 0; t < per; ++grp) {
      const int64_t rh = std::min<int64_t>(nrb - grp * g, g), take = std::min(rh * ncb, per - t);
      rows += std::min(take, rh);
      cols = std::max(cols, cdiv(take, rh));
      t += take;
    }
    if (rows + cols < best_cost) best_cost = rows + cols, best = g;
  }
  return best;
}

// Rows and columns of a scaled product's C: with m * n below 2^36 the 128 x 128
// tiles then stay below the launch limit.
constexpr int64_t kScaledDim = int64_t(1) << 27;
constexpr int64_t kMaxGrid = int64_t(1) << 23;

int validate_scaled(int N, int64_t m_s, int64_t k, int64_t n, int a_format, int b_block_rows, int c_dtype) {
  const int rc = check_sizes(N, m_s, k, n);
  if (rc != AGMM_OK) return rc;
  if (a_format != AGMM_E4M3 && a_format != AGMM_E5M2)
    return set_err(AGMM_ERR_INVALID_ARG, "unknown 8-bit format %d", a_format);
  if (b_block_rows != 1 && b_block_rows != agmm::kScaleBlock)
    return set_err(AGMM_ERR_INVALID_ARG, "b_block_rows must be 1 or %d (got %d)", agmm::kScaleBlock, b_block_rows);
  if (c_dtype != AGMM_BF16 && c_dtype != AGMM_FP16 && c_dtype != AGMM_FP32)
    return set_err(AGMM_ERR_INVALID_ARG, "unknown dtype %d", c_dtype);
  if (N * m_s >= kScaledDim || n >= kScaledDim || N * m_s * n >= (int64_t(1) << 36))
    return set_err(AGMM_ERR_UNSUPPORTED, "problem too large (m=%lld, n_local=%lld)", (long long)(N * m_s), (long long)n);
  return ok();
}

}  // namespace

struct agmm_scaled_plan : PlanBase {
  int N = 0;
  int64_t m_s = 0, k = 0, n = 0, m = 0, k16 = 0;
  int a_format = 0, b_block_rows = 0, c_dtype = 0;
  int64_t lda = 0, ldb = 0, ldc = 0;   // 0: dense
  int tile_key = -1, splits_key = 0;
  bool exact = false;
  int tile = 0, splits = 1, kb_per_split = 0, group_m = 1;
  bool deep = false;

  // Sums of 128 by bf16 MFMAs, whose products and sums are those of fp32.  The
  // 8-bit ones, twice as fast, cut each product to 2^-13 of the largest beside
  // it (scaled.hip).  They are a choice for speed, taken where C is 16 bits and
  // k long: on normally distributed operands the cut is 2^-15 of a block's sum
  // of sizes (rms), where the operands' own rounding to 8 bits moves every
  // product by up to 2^-3 of itself; but a block with one large product among
  // many small ones may lose up to 2^-10 of its sum of sizes, and one whose
  // large product cancels may be wrong in all its digits.  "exact_sums" is for
  // callers who need the other.
  bool wide() const { return exact || c_dtype == AGMM_FP32 || k < 1024; }

  int64_t kb() const { return cdiv(k, agmm::kScaleBlock); }

  // Cycles a launch of a tile with `sp` k ranges takes, from measurements on
  // MI355X (8-bit operands, cycles of about 2.1 GHz):
  //  * a CU streams its operands at about 26 bytes per cycle from one
  //    workgroup, 38 from two; every workgroup reads (rows + columns) * 128
  //    bytes per k block, which is what bounds all but the bf16-MFMA form of
  //    the 128 x 128 tile and the 256 x 256 tile (MFMA);
  //  * setup, first loads and epilogue: 8 thousand cycles for the skinny tiles,
  //    12 for 128 x 128, 20 for 256 x 256;
  //  * a second launch that adds k ranges: 6 thousand, and 8 bytes per partial
  //    sum at about 1900 bytes per cycle.
  // E.g. (us, measured): 192 x 2048 x 2048: 32 x 32 tiles 9.3, 64 x 64 10.5,
  // 128 x 128 15.2; 512 x 4096 -> 2048: 128 x 128 with 4 ranges 18.8, one 22.7,
  // 256 x 256 26.8; 4096 x 4096 -> 4096: 256 x 256 60, 128 x 128 73; 8 x 4096 ->
  // 1792: 16 x 16 tiles 5.1, 16 x 32 7.3.
  double cycles(int t, int64_t sp) const {
    const int64_t rows = agmm::scaled_tile_rows(t), cols = agmm::scaled_tile_cols(t);
    const int64_t wgs = cdiv(m, rows) * cdiv(n, cols) * sp, blocks = cdiv(kb(), sp);
    double base, step;
    int64_t rounds = cdiv(wgs, cu_count);
    if (t == agmm::kScaled256) {
      base = 20e3;
      step = 2300;
    } else if (t == agmm::kScaled128) {
      base = 12e3;
      rounds = cdiv(wgs, 2 * (int64_t)cu_count);
      step = wgs <= cu_count ? (wide() ? 2100 : 1300) : wide() ? 3700 : 1700;
    } else {
      base = 8e3;
      step = (double)(rows + cols) * 128 / 26;
    }
    return base + rounds * blocks * step + (sp > 1 ? 6e3 + (double)sp * m * n * 8 / 1900 : 0);
  }

  // Tile and k ranges for a pair of keys; host only.
  void derive(int tile_k, int splits_k, int& t, int& sp, int& per) const {
    // the tiles of each value of the key "tile"
    static const int of_key[4][2] = {{agmm::kScaled256, agmm::kScaled256},
                                     {agmm::kScaled128, agmm::kScaled128},
                                     {agmm::kScaledSkinny16, agmm::kScaledSkinny16n},
                                     {agmm::kScaledSkinny32, agmm::kScaledSkinny64}};
    double best = -1;
    t = agmm::kScaled128;
    int64_t want = 1;
    for (int key = 0; key < 4; ++key) {
      if (tile_k >= 0 ? key != tile_k : key == 0 && wide()) continue;
      for (int c : of_key[key]) {
        const int64_t tiles = cdiv(m, agmm::scaled_tile_rows(c)) * cdiv(n, agmm::scaled_tile_cols(c));
        for (int64_t w : {1, 2, 3, 4, 6, 8, 12, 16}) {
          if (splits_k > 0) w = splits_k;
          w = std::max<int64_t>(1, std::min(w, kb()));
          if (tile_k < 0 && tiles * w >= kMaxGrid) continue;
          const double cost = cycles(c, w);
          if (best < 0 || cost < best) best = cost, t = c, want = w;
        }
      }
    }
    per = (int)cdiv(kb(), want);
    sp = (int)cdiv(kb(), per);
  }

  // Row length of the partial sums: whole 16-byte vectors.
  int64_t part_ld() const { return round_up(n, 4); }

  size_t need(int sp) const { return sp > 1 ? (size_t)sp * m * part_ld() * sizeof(float) : 0; }

  int apply(int tile_k, int splits_k, bool exact_sums) {
    if (exact_sums && tile_k == agmm::kScaled256)
      return set_err(AGMM_ERR_UNSUPPORTED, "tile 0 sums on the 8-bit matrix instruction: not with exact_sums");
    const bool was = exact;
    exact = exact_sums;   // wide() goes by it
    const int rc = apply_tiles(tile_k, splits_k);
    if (rc != AGMM_OK) exact = was;
    return rc;
  }

  int apply_tiles(int tile_k, int splits_k) {
    int t, sp, per;
    derive(tile_k, splits_k, t, sp, per);
    if (cdiv(m, agmm::scaled_tile_rows(t)) * cdiv(n, agmm::scaled_tile_cols(t)) * sp >= kMaxGrid)
      return set_err(AGMM_ERR_UNSUPPORTED, "too many workgroups for tile %d with %d k ranges", t, sp);
    const int rc = reserve(need(sp));
    if (rc != AGMM_OK) return rc;
    tile_key = tile_k;
    splits_key = splits_k;
    tile = t;
    splits = sp;
    kb_per_split = per;
    deep = t == agmm::kScaled128 && cdiv(m, 128) * cdiv(n, 128) * sp <= cu_count;
    group_m = group_rows(cdiv(m, agmm::scaled_tile_rows(t)), cdiv(n, agmm::scaled_tile_cols(t)));
    return ok();
  }
};

namespace {

int validate_loss(int N, int64_t m_s, int64_t k, int64_t n, int dtype, int64_t start, int64_t total) {
  const int rc = check_sizes(N, m_s, k, n);
  if (rc != AGMM_OK) return rc;
  if (dtype == AGMM_FP32)
    return set_err(AGMM_ERR_UNSUPPORTED, "the vocabulary loss takes bf16 or fp16 operands");
  if (dtype != AGMM_BF16 && dtype != AGMM_FP16) return set_err(AGMM_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (start < 0 || total < 1 || total >= agmm::kElemLimit || start > total - n)
    return set_err(AGMM_ERR_INVALID_ARG, "%lld columns from %lld on do not lie in a vocabulary of %lld", (long long)n,
                   (long long)start, (long long)total);
  if (N * m_s >= (int64_t(1) << 27) || n >= (int64_t(1) << 27))
    return set_err(AGMM_ERR_UNSUPPORTED, "problem too large (m=%lld, n_local=%lld)", (long long)(N * m_s), (long long)n);
  return ok();
}

// A workspace cut into 256-byte aligned pieces.  With base NULL it only adds
// up sizes.
struct Cut {
  char* base;
  size_t at = 0;
  char* take(size_t bytes) {
    char* p = base ? base + at : nullptr;
    at += (bytes + 255) & ~size_t(255);
    return p;
  }
};

}  // namespace

struct agmm_loss_plan : PlanBase {
  int N = 0;
  int64_t m_s = 0, k = 0, n = 0, m = 0;
  int dtype = 0;
  int64_t start = 0, total = 0, ignore = -100;
  bool with_gradient = true;
  int64_t lda = 0, ldw = 0, ldda = 0, lddw = 0;   // 0: dense
  int64_t piece_key = 0;                          // columns per piece; 0: automatic
  int64_t tile_key = -1;                          // 64 (few rows), 128, 256; -1: automatic

  // What a call of a pass uses, derived from the settings.
  struct Layout {
    bool pad_a = false, pad_w = false;   // rows that are not whole 16-byte vectors: zero-padded copies
    int64_t kp = 0;                      // k rounded up to 8
    int64_t piece = 0;                   // columns of the vocabulary per piece
    int tile = 256, tile_grads = 256;    // tile 64: the few-row form, in
    int fm = 0, fn = 0;                  // blocks of 16 fm x 16 fn
    int ranges = 1;                      // k ranges of the dA product
    int64_t per_range = 0;
    // a, w: gathered or padded copies of A and of a piece of W
    char *a = nullptr, *w = nullptr, *d = nullptr, *dt = nullptr;
    float *stats = nullptr, *running = nullptr, *rows = nullptr, *scale_all = nullptr, *sums = nullptr;
    size_t bytes = 0;
  };

  int64_t ld_a() const { return lda ? lda : k; }
  int64_t ld_w() const { return ldw ? ldw : k; }
  int64_t m8() const { return round_up(m, 8); }

  // Microseconds of one workgroup, measured on MI355X over sums of 300 to 4096:
  // 20 and 2.1 per 64 of its sum for the 256 x 256 tile (one to a CU), 5 and
  // 1.25 for the 128 x 128 one (two to a CU; 0.7 where it has the CU alone).
  static double workgroup_us(int tile, int64_t sum) {
    return tile == 256 ? 20.0 + 2.1 * (double)cdiv(sum, 64) : 5.0 + 1.25 * (double)cdiv(sum, 64);
  }

  // Form of the products with W: the one that takes the least.  1000 x 700 over
  // 30000 columns twice: 111 us by 128, 143 by 256; 8192 x 4096 over 131072: 7.4
  // ms by 128, 6.2 by 256.  `copied`: the tiles need a copy of W first, which
  // the few-row form does not.
  void pick_tile(Layout& L, bool copied) const {
    const double big = (double)cdiv(cdiv(m, 256) * cdiv(n, 256), cu_count) * workgroup_us(256, k);
    const int64_t tiles = cdiv(m, 128) * cdiv(n, 128), rest = tiles % (2 * cu_count);
    const double small = (double)(tiles / (2 * cu_count)) * workgroup_us(128, k) +
                         (rest == 0 ? 0.0 : rest > cu_count ? workgroup_us(128, k) : 5.0 + 0.7 * (double)cdiv(k, 64));
    const double bytes = (double)n * (double)k * 2;
    L.tile = tile_key > 0 ? (int)tile_key : big <= small ? 256 : 128;
    if (tile_key > 0 && tile_key != 64) return;
    L.fm = m <= 16 ? 1 : 4;
    L.fn = cdiv(n, 64) * cdiv(m, 16 * L.fm) >= 2 * cu_count ? 4 : 1;
    const int64_t wgs = cdiv(m, 16 * L.fm) * cdiv(n, 16 * L.fn);
    // its operands' way into the CUs at 10 MB/us together (6 in its largest
    // blocks, which leave room for few waves), 1.7 times as long for odd strides
    // in place, or W from HBM.  Measured (us), with the copy where one is
    // needed: 16 x 3000 over 3000 columns 7, 34 by 128; 24 x 3121 over 5391 30,
    // 50; 8 x 3001 over 20000 36, 70; 64 x 3000 over 60000 114, 84.
    const double rate = (L.fm * L.fn == 16 ? 6e6 : 10e6) / (copied && (ld_a() % 2 != 0 || ld_w() % 2 != 0) ? 1.7 : 1.0);
    const double few = 5.0 + std::max((double)wgs * 32 * (L.fm + L.fn) * (double)k / rate, bytes / 4.8e6);
    if (tile_key == 64 || (few < std::min(big, small) + (copied ? 2.0 + 2 * bytes / 5e6 : 0.0) && wgs < kMaxGrid))
      L.tile = 64;
  }

  // Columns of one pair of statistics.
  static int64_t stat_cols(const Layout& L) { return L.tile == 64 ? 16 * L.fn : L.tile / 2; }

  Layout layout(bool grad, char* base) const {
    Layout L;
    L.kp = round_up(k, 8);
    L.pad_a = k % 8 != 0 || ld_a() % 8 != 0;
    L.pad_w = k % 8 != 0 || ld_w() % 8 != 0;
    // Piece: the gradient keeps d twice (16 bits) for a piece, the forward
    // pass 8 bytes per row and 64 columns; 512 MiB of either by default, which
    // at 8192 rows is 16384 columns, long enough for the three products.
    const int64_t budget = int64_t(512) << 20;
    int64_t piece = piece_key;
    if (!piece) piece = grad ? budget / (4 * m8()) : budget / (m * 8) * 64;
    if (!piece_key && L.pad_w) piece = std::min(piece, budget / (2 * L.kp));
    if (!piece_key && grad) {   // and no more than a launch of the gradient products holds by its smaller tile
      const int64_t a_tiles = std::max<int64_t>(cdiv(m, 128) * cdiv(k, 128), 4 * cu_count);
      piece = std::min(piece, (agmm::kLossGrid - 1 - a_tiles) / cdiv(k, 128) * 128);
    }
    piece = std::max<int64_t>(256, piece / 256 * 256);
    L.piece = std::min(piece, n);
    pick_tile(L, !grad && L.pad_w);
    if (!grad && L.tile == 64) L.pad_a = L.pad_w = false;   // read in place
    Cut c{base};
    if (L.pad_w) L.w = c.take((size_t)L.piece * L.kp * 2);
    if (!grad) {
      if (L.pad_a) L.a = c.take((size_t)m * L.kp * 2);
      L.stats = reinterpret_cast<float*>(c.take((size_t)(cdiv(L.piece, stat_cols(L)) + 1) * m * 8));
      L.running = reinterpret_cast<float*>(c.take((size_t)m * 8));
    } else {
      if (L.pad_a || N > 1) L.a = c.take((size_t)m * L.kp * 2);   // dW's product reads it k x n, in one piece
      L.rows = reinterpret_cast<float*>(c.take((size_t)m * 16));
      L.scale_all = reinterpret_cast<float*>(c.take(4));
      L.d = c.take((size_t)m * round_up(L.piece, 8) * 2);
      L.dt = c.take((size_t)L.piece * m8() * 2);
      // One launch computes both products; dA's sum (the piece's columns) is
      // cut into ranges.  Tile and ranges are those that take the least: the
      // workgroups' time spread over the CUs and half of one for the last
      // round, but no less than the longest of them; and the ranges' sums,
      // written and read at 4 TB/s.  1500 x 300 over 8000 columns takes 33 us
      // by 128, 68 by 256; 800 x 4000 over 50000 takes 921 and 955.
      double best = -1;
      int64_t want = 1;
      for (int t : {256, 128}) {
        if (tile_key > 64 && t != tile_key) continue;
        const int64_t a_tiles = cdiv(m, t) * cdiv(k, t), w_tiles = cdiv(L.piece, t) * cdiv(k, t);
        const double slots = cu_count * (t == 128 ? 2 : 1), w_us = workgroup_us(t, m);
        for (int64_t r = 1; r == 1 || (r <= 64 && a_tiles * r <= 4 * cu_count && L.piece / r >= 256); r *= 2) {
          const double a_us = workgroup_us(t, cdiv(L.piece, r));
          const double us = std::max({((double)(a_tiles * r) * a_us + (double)w_tiles * w_us) / slots + w_us / 2, a_us, w_us}) +
                            (double)(r * m) * (double)k * 8 / 4e6;
          if (best < 0 || us < best) best = us, L.tile_grads = t, want = r;
        }
      }
      L.per_range = round_up(cdiv(L.piece, want), 64);
      L.ranges = (int)cdiv(L.piece, L.per_range);
      L.sums = reinterpret_cast<float*>(c.take((size_t)L.ranges * m * round_up(k, 4) * 4));
    }
    L.bytes = c.at;
    return L;
  }

  // Whether the launches over a piece stay within kLossGrid: automatic pieces
  // do, one that the caller set may not.
  bool fits(const Layout& L, bool grad) const {
    const int64_t rows = L.tile == 64 ? 16 * L.fm : L.tile, cols = L.tile == 64 ? 16 * L.fn : L.tile, t = L.tile_grads;
    return cdiv(m, rows) * cdiv(L.piece, cols) < agmm::kLossGrid &&
           (!grad || cdiv(k, t) * (cdiv(m, t) * L.ranges + cdiv(L.piece, t)) < agmm::kLossGrid);
  }

  int apply() {
    size_t bytes = 0;
    for (bool grad : {false, true}) {
      if (grad && !with_gradient) continue;
      const Layout L = layout(grad, nullptr);
      if (!fits(L, grad))
        return set_err(AGMM_ERR_UNSUPPORTED, "too many workgroups for pieces of %lld columns by tile %d", (long long)L.piece,
                       L.tile);
      bytes = std::max(bytes, L.bytes);
    }
    return reserve(bytes);
  }

  agmm::TileOrder tiles_of(int64_t rows, int64_t cols, int tile) const {
    agmm::TileOrder o{};
    o.num_rb = (int32_t)cdiv(rows, tile);
    o.num_cb = (int32_t)cdiv(cols, tile);
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

  // `count` groups of `rows` rows of k elements, `ld` apart, as rows of whole
  // 16-byte vectors at `out`.
  agmm::PadRows copy_of(const Layout& L, const void* const* groups, int count, int64_t rows, int64_t ld, void* out) const {
    agmm::PadRows c{};
    for (int g = 0; g < count; ++g) c.group[g] = groups[g];
    c.num_groups = count;
    c.rows = rows;
    c.cols = k;
    c.ld = ld;
    c.chunks = L.kp / 8;
    c.out = out;
    return c;
  }

  // Rows [v0, v0 + vn) of W as whole 16-byte vectors: in place, or copied.
  int piece_w(const Layout& L, const void* W, int64_t v0, int64_t vn, hipStream_t s, const void** w, int64_t* ld) const {
    const void* src = static_cast<const char*>(W) + v0 * ld_w() * 2;
    *w = src;
    *ld = ld_w();
    if (!L.pad_w) return AGMM_OK;
    const agmm::PadRows c = copy_of(L, &src, 1, vn, ld_w(), L.w);
    *w = L.w;
    *ld = L.kp;
    const hipError_t err = agmm::launch_loss_prepare(nullptr, &c, dtype, s);
    return err == hipSuccess ? AGMM_OK : hip_err(err, "weight copy launch");
  }

  agmm::RowMap rows_of_a(const Layout& L, const void* const* shards) const {
    if (L.a) return dense(L.a, m, L.kp);
    agmm::RowMap r{};
    for (int g = 0; g < N; ++g) r.a_group[g] = shards[g];
    r.a_ld = ld_a();
    r.rows_per_group = (int32_t)m_s;
    r.num_groups = N;
    r.c_group_rows = m_s;
    return r;
  }

  agmm::LossProblem logits(const Layout& L, const agmm::RowMap& rows, const void* w, int64_t ldb, int64_t v0,
                           int64_t vn, const int64_t* labels) const {
    agmm::LossProblem p{};
    p.gemm.rows = rows;
    if (L.tile == 64) {
      p.gemm.order.num_rb = (int32_t)cdiv(m, 16 * L.fm);
      p.gemm.order.num_cb = (int32_t)cdiv(vn, 16 * L.fn);
    } else {
      p.gemm.order = tiles_of(m, vn, L.tile);
    }
    p.gemm.m = (int32_t)m;
    p.gemm.n = (int32_t)vn;
    p.gemm.k = (int32_t)(L.tile == 64 ? k : L.kp);
    p.gemm.b = w;
    p.gemm.ldb = ldb;
    p.gemm.splits = 1;
    p.gemm.k_per_split = (int32_t)L.kp;
    p.tile = L.tile;
    p.labels = labels;
    p.label0 = start + v0;
    return p;
  }

  hipError_t launch_logits(const Layout& L, const agmm::LossProblem& p, bool grad, hipStream_t s) const {
    return L.tile == 64 ? agmm::launch_loss_few(p, L.fm, L.fn, dtype, grad, s) : agmm::launch_loss_logits(p, dtype, grad, s);
  }

  int forward(const void* const* shards, const void* W, const int64_t* labels, float* loss, float* lse, float* target,
              hipStream_t s) {
    const Layout L = layout(false, ws);
    int rc = AGMM_OK;
    if (L.a) {
      const agmm::PadRows c = copy_of(L, shards, N, m_s, ld_a(), L.a);
      const hipError_t err = agmm::launch_loss_prepare(nullptr, &c, dtype, s);
      if (err != hipSuccess) return hip_err(err, "row copy launch");
    }
    const agmm::RowMap rows = rows_of_a(L, shards);
    for (int64_t v0 = 0; v0 < n && rc == AGMM_OK; v0 += L.piece) {
      const int64_t vn = std::min(L.piece, n - v0);
      const void* w;
      int64_t ldb;
      rc = piece_w(L, W, v0, vn, s, &w, &ldb);
      if (rc != AGMM_OK) break;
      agmm::LossProblem p = logits(L, rows, w, ldb, v0, vn, labels);
      p.stats = L.stats;
      p.target = target;
      hipError_t err = launch_logits(L, p, false, s);
      if (err != hipSuccess) return hip_err(err, "loss logits launch");
      agmm::LossCombine c{};
      c.stats = L.stats;
      c.parts = (L.tile == 64 ? 1 : 2) * p.gemm.order.num_cb;
      c.m = m;
      c.running = L.running;
      c.first = v0 == 0;
      c.last = v0 + vn == n;
      c.labels = labels;
      c.start = start;
      c.n = n;
      c.total = total;
      c.ignore = ignore;
      c.loss = loss;
      c.lse = lse;
      c.target = target;
      err = agmm::launch_loss_combine(c, s);
      if (err != hipSuccess) return hip_err(err, "loss combine launch");
    }
    return rc;
  }

  int backward(const void* const* shards, const void* W, const int64_t* labels, const float* lse,
               const float* grad_loss, const float* grad_lse, void* dA, void* dW, hipStream_t s) {
    const Layout L = layout(true, ws);
    int rc;
    const agmm::RowMap rows = rows_of_a(L, shards);
    agmm::LossRows lr{};
    lr.m = m;
    lr.labels = labels;
    lr.total = total;
    lr.ignore = ignore;
    lr.lse = lse;
    lr.grad_loss = grad_loss;
    lr.grad_lse = grad_lse;
    lr.rows = L.rows;
    lr.scale_all = L.scale_all;
    agmm::PadRows copy{};
    if (L.a) copy = copy_of(L, shards, N, m_s, ld_a(), L.a);
    hipError_t err = agmm::launch_loss_prepare(&lr, L.a ? &copy : nullptr, dtype, s);
    if (err != hipSuccess) return hip_err(err, "loss rows launch");
    for (int64_t v0 = 0; v0 < n; v0 += L.piece) {
      const int64_t vn = std::min(L.piece, n - v0);
      const void* w;
      int64_t ldb;
      rc = piece_w(L, W, v0, vn, s, &w, &ldb);
      if (rc != AGMM_OK) return rc;
      agmm::LossProblem p = logits(L, rows, w, ldb, v0, vn, labels);
      p.rows = L.rows;
      p.scale_all = L.scale_all;
      p.d = dA ? L.d : nullptr;
      p.ldd = round_up(vn, 8);
      p.dt = dW ? L.dt : nullptr;
      p.ldt = m8();
      err = launch_logits(L, p, true, s);
      if (err != hipSuccess) return hip_err(err, "loss gradient launch");
      agmm::GemmProblem ga{}, gw{};
      ga.rows = dense(L.d, m, round_up(vn, 8));
      ga.order = tiles_of(m, k, L.tile_grads);
      ga.m = (int32_t)m;
      ga.n = (int32_t)k;
      ga.k = (int32_t)vn;
      ga.b = w;
      ga.ldb = ldb;
      // the last piece may have fewer ranges: the rest keep their sums
      ga.k_per_split = (int32_t)L.per_range;
      ga.splits = (int32_t)cdiv(vn, L.per_range);
      ga.partials = L.sums;
      gw.rows = dense(L.dt, vn, m8());
      gw.order = tiles_of(vn, k, L.tile_grads);
      gw.m = (int32_t)vn;
      gw.n = (int32_t)k;
      gw.k = (int32_t)m;
      gw.b = L.a ? L.a : shards[0];
      gw.ldb = L.a ? L.kp : ld_a();
      gw.splits = 1;
      gw.k_per_split = (int32_t)round_up(m, 64);
      gw.ldc = lddw ? lddw : k;
      gw.c = static_cast<char*>(dW) + v0 * gw.ldc * 2;
      err = agmm::launch_loss_grads(dA ? &ga : nullptr, v0 > 0, dW ? &gw : nullptr, L.scale_all, L.tile_grads, dtype, s);
      if (err != hipSuccess) return hip_err(err, "gradient products launch");
    }
    if (dA) {
      agmm::LossFinish f{};
      f.sums = L.sums;
      f.ranges = L.ranges;
      f.m = m;
      f.k = (int32_t)k;
      f.rows = L.rows;
      f.da = dA;
      f.ldda = ldda ? ldda : k;
      err = agmm::launch_loss_da_finish(f, dtype, s);
      if (err != hipSuccess) return hip_err(err, "dA cast launch");
    }
    return AGMM_OK;
  }
};

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
  if (ldx >= kQuantElems || ldq >= kQuantElems || ldqt >= kQuantElems)
    return set_err(AGMM_ERR_UNSUPPORTED, "row length too large (ldx=%lld, ldq=%lld, ldqt=%lld)", (long long)ldx,
                   (long long)ldq, (long long)ldqt);
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

int agmm_scaled_plan_validate(int num_shards, int64_t m_per_shard, int64_t k, int64_t n_local, int a_format,
                              int b_block_rows, int c_dtype) {
  return validate_scaled(num_shards, m_per_shard, k, n_local, a_format, b_block_rows, c_dtype);
}

agmm_scaled_plan_t agmm_scaled_plan_create(int num_shards, int64_t m_per_shard, int64_t k, int64_t n_local,
                                           int a_format, int b_block_rows, int c_dtype) {
  if (validate_scaled(num_shards, m_per_shard, k, n_local, a_format, b_block_rows, c_dtype) != AGMM_OK)
    return nullptr;
  agmm_scaled_plan* p = new (std::nothrow) agmm_scaled_plan();
  if (!p) {
    set_err(AGMM_ERR_OOM, "out of host memory");
    return nullptr;
  }
  p->N = num_shards;
  p->m_s = m_per_shard;
  p->k = k;
  p->k16 = round_up(k, 16);
  p->n = n_local;
  p->m = num_shards * m_per_shard;
  p->a_format = a_format;
  p->b_block_rows = b_block_rows;
  p->c_dtype = c_dtype;
  if (p->init() != AGMM_OK || p->apply(-1, 0, false) != AGMM_OK) {
    const int st = agmm::g_status;
    const std::string msg = agmm::g_msg;
    delete p;
    set_err(st, "%s", msg.c_str());
    return nullptr;
  }
  return p;
}

int agmm_scaled_plan_set_int(agmm_scaled_plan_t p, const char* key, int64_t v) {
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
  if (k == "tile") {
    if (v < -1 || v > 3) return bad();
    return p->apply((int)v, p->splits_key, p->exact);
  }
  if (k == "splits") {
    if (v < 0 || v > 4096) return bad();
    return p->apply(p->tile_key, (int)v, p->exact);
  }
  if (k == "exact_sums") {
    if (v != 0 && v != 1) return bad();
    return p->apply(p->tile_key, p->splits_key, v == 1);
  }
  if (k == "lda" || k == "ldb" || k == "ldc") {
    const int64_t row = k == "ldc" ? p->n : p->k16;
    if (v != 0 && (v < row || v >= kDimLimit || (k != "ldc" && v % 16 != 0))) return bad();
    (k == "lda" ? p->lda : k == "ldb" ? p->ldb : p->ldc) = v;
    return ok();
  }
  return set_err(AGMM_ERR_INVALID_ARG, "unknown key '%s'", key);
}

int agmm_scaled_plan_get_int(agmm_scaled_plan_t p, const char* key, int64_t* value) {
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "plan is NULL");
  if (!key || !value) return set_err(AGMM_ERR_INVALID_ARG, "key or value is NULL");
  std::lock_guard<std::mutex> lk(p->mu);
  const std::string k(key);
  if (k == "tile") *value = p->tile == agmm::kScaledSkinny16n ? 2 : p->tile == agmm::kScaledSkinny64 ? 3 : p->tile;
  else if (k == "splits") *value = p->splits;
  else if (k == "exact_sums") *value = p->exact;
  else if (k == "lda") *value = p->lda ? p->lda : p->k16;
  else if (k == "ldb") *value = p->ldb ? p->ldb : p->k16;
  else if (k == "ldc") *value = p->ldc ? p->ldc : p->n;
  else if (k == "captured") *value = p->captured;
  else return set_err(AGMM_ERR_INVALID_ARG, "unknown key '%s'", key);
  return ok();
}

size_t agmm_scaled_plan_workspace_bytes(agmm_scaled_plan_t p) { return p ? p->ws_bytes : 0; }

int agmm_scaled_run(agmm_scaled_plan_t p, const void* const* shard_ptrs, const float* const* scale_ptrs,
                    const void* B, const float* B_scales, void* C, void* stream) {
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "plan is NULL");
  if (!shard_ptrs || !scale_ptrs) return set_err(AGMM_ERR_INVALID_ARG, "shard_ptrs or scale_ptrs is NULL");
  int rc = AGMM_OK;
  for (int r = 0; r < p->N && rc == AGMM_OK; ++r) {
    rc = check_ptr(shard_ptrs[r], "shard_ptrs", r, 16);
    if (rc == AGMM_OK) rc = check_ptr(scale_ptrs[r], "scale_ptrs", r, 4);
  }
  if (rc == AGMM_OK) rc = check_ptr(B, "B", -1, 16);
  if (rc == AGMM_OK) rc = check_ptr(B_scales, "B_scales", -1, 4);
  if (rc == AGMM_OK) rc = check_ptr(C, "C", -1, 16);
  if (rc != AGMM_OK) return rc;
  std::lock_guard<std::mutex> lk(p->mu);
  agmm::ScaledProblem g{};
  for (int r = 0; r < p->N; ++r) {
    g.a_group[r] = shard_ptrs[r];
    g.a_scale[r] = scale_ptrs[r];
  }
  g.a_ld = p->lda ? p->lda : p->k16;
  g.rows_per_group = (int32_t)p->m_s;
  g.num_groups = p->N;
  g.m = (int32_t)p->m;
  g.n = (int32_t)p->n;
  g.k16 = (int32_t)p->k16;
  g.kb = (int32_t)p->kb();
  g.b = B;
  g.ldb = p->ldb ? p->ldb : p->k16;
  g.b_scale = B_scales;
  g.nb = (int32_t)cdiv(p->n, p->b_block_rows);
  g.b_block_rows = p->b_block_rows;
  g.a_format = p->a_format;
  g.c = C;
  g.ldc = p->ldc ? p->ldc : p->n;
  g.c_dtype = p->c_dtype;
  g.wide = p->wide();
  g.deep = p->deep;
  g.order.num_rb = (int32_t)cdiv(p->m, agmm::scaled_tile_rows(p->tile));
  g.order.num_cb = (int32_t)cdiv(p->n, agmm::scaled_tile_cols(p->tile));
  g.order.group_m = p->group_m;
  g.order.xcd_remap = 1;
  g.splits = p->splits;
  g.kb_per_split = p->kb_per_split;
  g.partials = reinterpret_cast<float*>(p->ws);
  g.part_ld = p->part_ld();
  hipStream_t s = static_cast<hipStream_t>(stream);
  return p->run(s, p->splits > 1, [&]() -> int {
    const hipError_t err = agmm::launch_scaled(g, p->tile, s);
    return err == hipSuccess ? AGMM_OK : hip_err(err, "scaled product launch");
  });
}

void agmm_scaled_plan_destroy(agmm_scaled_plan_t p) { delete p; }

int agmm_loss_plan_validate(int num_shards, int64_t m_per_shard, int64_t k, int64_t n_local, int dtype,
                            int64_t vocab_start, int64_t vocab_size) {
  return validate_loss(num_shards, m_per_shard, k, n_local, dtype, vocab_start, vocab_size);
}

agmm_loss_plan_t agmm_loss_plan_create(int num_shards, int64_t m_per_shard, int64_t k, int64_t n_local, int dtype,
                                       int64_t vocab_start, int64_t vocab_size, int with_gradient) {
  if (validate_loss(num_shards, m_per_shard, k, n_local, dtype, vocab_start, vocab_size) != AGMM_OK) return nullptr;
  agmm_loss_plan* p = new (std::nothrow) agmm_loss_plan();
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
  p->start = vocab_start;
  p->total = vocab_size;
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

int agmm_loss_plan_set_int(agmm_loss_plan_t p, const char* key, int64_t v) {
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
  } else if (k == "piece") {
    if (v < 0 || v >= kDimLimit) return bad();
    field = &p->piece_key;
  } else if (k == "tile") {
    if (v != -1 && v != 64 && v != 128 && v != 256) return bad();
    if (v == 64 && cdiv(p->m, 64) * cdiv(p->n, 64) >= kMaxGrid)
      return set_err(AGMM_ERR_UNSUPPORTED, "too many workgroups for tile 64");
    field = &p->tile_key;
  } else if (k == "ignore_index") {
    p->ignore = v;
    return ok();
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

int agmm_loss_plan_get_int(agmm_loss_plan_t p, const char* key, int64_t* value) {
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "plan is NULL");
  if (!key || !value) return set_err(AGMM_ERR_INVALID_ARG, "key or value is NULL");
  std::lock_guard<std::mutex> lk(p->mu);
  const std::string k(key);
  if (k == "lda") *value = p->ld_a();
  else if (k == "ldw") *value = p->ld_w();
  else if (k == "ldda") *value = p->ldda ? p->ldda : p->k;
  else if (k == "lddw") *value = p->lddw ? p->lddw : p->k;
  else if (k == "piece") *value = p->layout(p->with_gradient, nullptr).piece;
  else if (k == "tile") *value = p->layout(false, nullptr).tile;
  else if (k == "ignore_index") *value = p->ignore;
  else if (k == "captured") *value = p->captured;
  else return set_err(AGMM_ERR_INVALID_ARG, "unknown key '%s'", key);
  return ok();
}

size_t agmm_loss_plan_workspace_bytes(agmm_loss_plan_t p) { return p ? p->ws_bytes : 0; }

int agmm_loss_forward(agmm_loss_plan_t p, const void* const* shard_ptrs, const void* W, const int64_t* labels,
                      float* loss, float* lse, float* target, void* stream) {
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "plan is NULL");
  if (!shard_ptrs) return set_err(AGMM_ERR_INVALID_ARG, "shard_ptrs is NULL");
  int rc = AGMM_OK;
  for (int r = 0; r < p->N && rc == AGMM_OK; ++r) rc = check_ptr(shard_ptrs[r], "shard_ptrs", r, 16);
  if (rc == AGMM_OK) rc = check_ptr(W, "W", -1, 16);
  if (rc == AGMM_OK) rc = check_ptr(labels, "labels", -1, 8);
  if (rc == AGMM_OK) rc = check_ptr(loss, "loss", -1, 4);
  if (rc == AGMM_OK) rc = check_ptr(lse, "lse", -1, 4);
  if (rc == AGMM_OK) rc = check_ptr(target, "target", -1, 4);
  if (rc != AGMM_OK) return rc;
  std::lock_guard<std::mutex> lk(p->mu);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return p->run(s, true, [&] { return p->forward(shard_ptrs, W, labels, loss, lse, target, s); });
}

int agmm_loss_backward(agmm_loss_plan_t p, const void* const* shard_ptrs, const void* W, const int64_t* labels,
                       const float* lse, const float* grad_loss, const float* grad_lse, void* dA, void* dW,
                       void* stream) {
  if (!p) return set_err(AGMM_ERR_INVALID_ARG, "plan is NULL");
  if (!p->with_gradient) return set_err(AGMM_ERR_UNSUPPORTED, "the plan was created without the gradient's workspace");
  if (!shard_ptrs) return set_err(AGMM_ERR_INVALID_ARG, "shard_ptrs is NULL");
  if (!dA && !dW) return set_err(AGMM_ERR_INVALID_ARG, "dA and dW are both NULL");
  int rc = AGMM_OK;
  for (int r = 0; r < p->N && rc == AGMM_OK; ++r) rc = check_ptr(shard_ptrs[r], "shard_ptrs", r, 16);
  if (rc == AGMM_OK) rc = check_ptr(W, "W", -1, 16);
  if (rc == AGMM_OK) rc = check_ptr(labels, "labels", -1, 8);
  if (rc == AGMM_OK) rc = check_ptr(lse, "lse", -1, 4);
  if (rc == AGMM_OK) rc = check_ptr(grad_loss, "grad_loss", -1, 4);
  if (rc == AGMM_OK && grad_lse) rc = check_ptr(grad_lse, "grad_lse", -1, 4);
  if (rc == AGMM_OK && dA) rc = check_ptr(dA, "dA", -1, 16);
  if (rc == AGMM_OK && dW) rc = check_ptr(dW, "dW", -1, 16);
  if (rc != AGMM_OK) return rc;
  std::lock_guard<std::mutex> lk(p->mu);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return p->run(s, true, [&] { return p->backward(shard_ptrs, W, labels, lse, grad_loss, grad_lse, dA, dW, s); });
}

void agmm_loss_plan_destroy(agmm_loss_plan_t p) { delete p; }

}  // extern "C"
