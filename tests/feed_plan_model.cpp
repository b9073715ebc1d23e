// The feed-forward block's and layer norm's host source on a model of the
// runtime (no GPU): what a call launches, and what it refuses.  agmm_feed.cpp is
// part of this file, so that a plan's own time model can be asked.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <set>
#include <string>
#include <vector>

struct ihipStream_t {};
struct ihipEvent_t {};

#include "agmm_feed.cpp"

const char* hipGetErrorString(hipError_t) { return "model error"; }
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipGetDevice(int* device) { return *device = 0, hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* value, hipDeviceAttribute_t, int) { return *value = 256, hipSuccess; }
hipError_t hipMalloc(void** p, size_t) {
  *p = std::aligned_alloc(256, 256);   // never read
  return *p ? hipSuccess : hipErrorOutOfMemory;
}
hipError_t hipFree(void* p) { return std::free(p), hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipStreamWaitEvent(hipStream_t, hipEvent_t, unsigned) { return hipSuccess; }
hipError_t hipStreamGetCaptureInfo(hipStream_t, hipStreamCaptureStatus* status, unsigned long long* id) {
  return *status = hipStreamCaptureStatusNone, *id = 0, hipSuccess;
}
hipError_t hipEventCreateWithFlags(hipEvent_t* e, unsigned) { return *e = new ihipEvent_t, hipSuccess; }
hipError_t hipEventDestroy(hipEvent_t e) { return delete e, hipSuccess; }
hipError_t hipEventRecord(hipEvent_t, hipStream_t) { return hipSuccess; }
hipError_t hipEventSynchronize(hipEvent_t) { return hipSuccess; }

namespace {

// What the call launched.
struct Launched {
  int count = 0, tile = 0, splits = 0;
  bool copied = false;
} launched;

int failures = 0;

void expect(bool is, const std::string& what) {
  if (is) return;
  if (++failures <= 20) std::printf("FAILED: %s\n", what.c_str());
}

}  // namespace

namespace agmm {
hipError_t launch_feed_tiles(const FeedProblem& p, int tile, int, hipStream_t) {
  launched.tile = tile;
  launched.splits = p.gemm.splits;
  return ++launched.count, hipSuccess;
}
hipError_t launch_feed_few(const FeedProblem& p, int, int, int, hipStream_t) {
  launched.tile = 64;
  launched.splits = p.gemm.splits;
  return ++launched.count, hipSuccess;
}
hipError_t launch_feed_copies(const FeedCopies&, hipStream_t) { return launched.copied = true, ++launched.count, hipSuccess; }
hipError_t launch_feed_d(const FeedDProblem&, const FeedCopies&, int, hipStream_t) { return ++launched.count, hipSuccess; }
hipError_t launch_feed_again(const FeedAgainProblem&, int, hipStream_t) { return ++launched.count, hipSuccess; }
hipError_t launch_feed_grads(FeedGrads, int, int, hipStream_t) { return ++launched.count, hipSuccess; }
hipError_t launch_sum_ranges(const SumRanges*, const SumRanges*, int, hipStream_t) { return ++launched.count, hipSuccess; }
hipError_t launch_sum_columns(const SumColumns&, hipStream_t) { return ++launched.count, hipSuccess; }
hipError_t launch_norm_forward(const NormProblem&, hipStream_t) { return ++launched.count, hipSuccess; }
hipError_t launch_norm_backward(const NormProblem&, hipStream_t) { return ++launched.count, hipSuccess; }
bool norm_direct(int64_t, int, int groups) { return groups == 1; }
int norm_groups(int64_t rows, int64_t, int, int) { return rows <= 4 ? 1 : 4; }
}  // namespace agmm

namespace {

// Addresses that nothing reads: 256 bytes apart, aligned to 256.
alignas(256) char memory[16384];
char* at(int i) { return memory + 256 * i; }

Launched forward(agmm_ff_plan_t p, int N, int keep) {
  const void* shards[agmm::kMaxGroups];
  for (int r = 0; r < N; ++r) shards[r] = at(r % 8);
  launched = Launched{};
  const int rc = agmm_ff_forward(p, shards, at(8), nullptr, nullptr, at(9), keep ? at(10) : nullptr, keep == 8 ? at(11) : nullptr, nullptr);
  expect(rc == AGMM_OK, "forward: " + agmm::g_msg);
  return launched;
}

// A call runs a form that it can use, the cheapest one by the plan's time model.
void forms() {
  std::mt19937 rng(1);
  const auto size = [&](double lo, double hi) {
    return (int64_t)std::exp(std::uniform_real_distribution<double>(std::log(lo), std::log(hi))(rng));
  };
  int by[257] = {};
  for (int i = 0; i < 4000; ++i) {
    const bool large = i % 2 == 0;
    const int64_t m_s = i == 0 ? 300 : size(large ? 1024 : 1, large ? 16384 : 4096), k = i == 0 ? 7008 : size(large ? 512 : 64, 8192) / 8 * 8,
                  n = i == 0 ? 6636 : size(large ? 512 : 16, 8192);
    const int N = 1, gated = i == 0 || i % 3 != 0;
    const int keep = i == 0 ? 8 : (i / 3 % 3) * 8;
    agmm_ff_plan_t p = agmm_ff_plan_create(N, m_s, k, n, AGMM_BF16, AGMM_ACT_SILU, gated, 0);
    const std::string what = std::to_string(m_s) + " x " + std::to_string(k) + " -> " + std::to_string(1 + gated) + " x " + std::to_string(n) +
                             ", " + std::to_string(keep) + " bits kept";
    expect(p, what + ": " + agmm::g_msg);
    if (!p) continue;
    const Launched l = forward(p, N, keep);
    expect(l.tile == 64 || l.tile == 128 || l.tile == 224 || l.tile == 256, what + ": no product");
    const bool no_224 = gated && keep == 8;
    expect(!(no_224 && l.tile == 224), what + ": tiles of 224 cut the blocks of 32 columns");
    ++by[l.tile];
    // every form of tiles that the call could have run
    const int64_t nc = p->tile_cols();
    const bool lines = p->ld_a() % 64 == 0 && p->ld_w() % 64 == 0;
    const auto price = [&](int t, bool copied, int splits) {
      const int64_t tiles = agmm::cdiv(m_s, t == 224 ? 256 : t) * agmm::cdiv(nc, t) * splits;
      return p->tiles_us(t, tiles, agmm::cdiv(k, splits), lines || copied) + (copied ? p->copy_us() : 0.0) + (splits > 1 ? p->join_us(splits, 4.0) : 0.0);
    };
    if (l.tile != 64) {
      for (int t : {128, 224, 256})
        for (bool copied : {false, true})
          expect((t == 224 && no_224) || price(l.tile, l.copied, l.tile == 128 ? l.splits : 1) <= price(t, copied, 1) * 1.02,
                 what + ": " + std::to_string(t) + " would take less than " + std::to_string(l.tile));
    }
    for (int t : {64, 128, 224, 256}) {        // a form that is asked for
      if (agmm_ff_plan_set_int(p, "tile", t) != AGMM_OK) continue;
      const int ran = forward(p, N, keep).tile;
      expect(ran == (t == 224 && no_224 ? 256 : t), what + ": tile " + std::to_string(t) + " ran " + std::to_string(ran));
    }
    agmm_ff_plan_destroy(p);
  }
  std::printf("64: %d, 128: %d, 224: %d, 256: %d\n", by[64], by[128], by[224], by[256]);
  expect(by[64] > 100 && by[128] > 100 && by[224] > 100 && by[256] > 100, "every form is chosen");
}

// Two operands of a call at one address: refused where either is an output, with
// nothing launched, but for the pairs that may be in place.
struct Operand {
  std::string name;
  void** where;
  bool output;
};
template <class F>
void pairs(const std::string& entry, const std::vector<Operand>& operands, const std::set<std::string>& in_place, F&& call) {
  launched = Launched{};
  expect(call() == AGMM_OK && launched.count > 0, entry + ": " + agmm::g_msg);
  for (const Operand& out : operands) {
    if (!out.output) continue;
    for (const Operand& other : operands) {
      if (&out == &other) continue;
      void* const kept = *out.where;
      *out.where = *other.where;
      launched = Launched{};
      const int rc = call();
      const std::string what = entry + ": " + out.name + " at " + other.name;
      if (in_place.count(out.name + " " + other.name)) {
        expect(rc == AGMM_OK && launched.count > 0, what + ": " + agmm::g_msg);
      } else {
        expect(rc == AGMM_ERR_INVALID_ARG && agmm::g_msg.find("overlaps") != std::string::npos, what + " is not refused");
        expect(launched.count == 0, what + ": launched");
      }
      *out.where = kept;
    }
  }
}

void overlaps() {
  for (int gated : {0, 1})
    for (int scaled : {0, 1}) {
      void *A[3] = {at(0), at(1), at(2)}, *W = at(3), *b = at(4), *r = gated ? nullptr : at(5), *y = at(6), *v = at(7), *s = scaled ? at(8) : nullptr;
      void *dy = at(9), *da = at(10), *dw = at(11), *db = at(12);
      agmm_ff_plan_t p = agmm_ff_plan_create(3, 4, 64, 64, AGMM_BF16, AGMM_ACT_SILU, gated, 1);
      std::vector<Operand> all = {{"shard 0", &A[0], false}, {"shard 2", &A[2], false}, {"W", &W, false}, {"bias", &b, false},
                                  {"Y", &y, true}, {"saved", &v, true}};
      if (!gated) all.push_back({"residual", &r, false});
      if (scaled) all.push_back({"saved_scales", &s, true});
      pairs("forward", all, {"Y residual"}, [&] { return agmm_ff_forward(p, A, W, b, r, y, v, s, nullptr); });
      all = {{"shard 0", &A[0], false}, {"shard 2", &A[2], false}, {"W", &W, false}, {"saved", &v, false}, {"dY", &dy, false},
             {"dA", &da, true}, {"dW", &dw, true}, {"dbias", &db, true}};
      if (scaled) all.push_back({"saved_scales", &s, false});
      pairs("backward", all, {}, [&] { return agmm_ff_backward(p, A, W, v, s, dy, da, dw, db, nullptr); });
      all = {{"saved", &v, false}, {"Y", &y, true}};
      if (scaled) all.push_back({"saved_scales", &s, false});
      pairs("recompute", all, {}, [&] { return agmm_ff_recompute(p, v, s, y, nullptr); });
      agmm_ff_plan_destroy(p);
    }
  for (int64_t rows : {2, 100}) {               // the weights' gradients in one launch, and in two
    void *x = at(0), *dy = at(1), *w = at(2), *b = at(3), *y = at(4), *mean = at(5), *rstd = at(6), *dx = at(7), *dw = at(8), *db = at(9);
    agmm_norm_plan_t p = agmm_norm_plan_create(rows, 64, AGMM_FP32, AGMM_FP32);
    const auto f = [](void*& q) { return static_cast<float*>(q); };
    pairs("norm", {{"x", &x, false}, {"weight", &w, false}, {"bias", &b, false}, {"y", &y, true}, {"mean", &mean, true}, {"rstd", &rstd, true}},
          {"y x"}, [&] { return agmm_norm_forward(p, x, w, b, 1e-5f, y, f(mean), f(rstd), nullptr); });
    pairs("norm backward", {{"x", &x, false}, {"dy", &dy, false}, {"weight", &w, false}, {"mean", &mean, false}, {"rstd", &rstd, false},
                            {"dx", &dx, true}, {"dweight", &dw, true}, {"dbias", &db, true}},
          {"dx dy"}, [&] { return agmm_norm_backward(p, x, dy, w, f(mean), f(rstd), dx, dw, db, nullptr); });
    agmm_norm_plan_destroy(p);
  }
}

}  // namespace

int main(int argc, char** argv) {
  const std::string part = argc > 1 ? argv[1] : "forms";
  if (part == "forms") forms();
  else if (part == "overlaps") overlaps();
  else expect(false, "unknown part");
  if (!failures) std::printf("all as expected\n");
  return failures ? 1 : 0;
}
