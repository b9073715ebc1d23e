// Order of a plan's calls, on a model of streams and events (no GPU): the host
// sources are compiled against tests/hip_model, every launch is an operation,
// and the checks ask whether one call's operations come after another's.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <set>
#include <string>
#include <vector>

#include "agmm.h"
#include "agmm_kernels.h"
#include "ops_kernels.h"

struct ihipStream_t {
  std::set<int> before;              // what the next operation comes after
  unsigned long long capture = 0;    // the graph capture it is part of
};
struct ihipEvent_t {
  std::set<int> before;
  bool recorded = false;
  unsigned long long capture = 0;
};

namespace {

struct Op {
  std::set<int> before;
};
std::vector<Op> ops;
std::set<int> finished;              // what the host has waited for
std::set<int> freed_early;           // operations not waited for when memory was freed
std::vector<ihipStream_t*> internal; // streams the library made
ihipStream_t default_stream, per_thread[2];
int thread_now = 0;

ihipStream_t& at(hipStream_t s) {
  if (!s) return default_stream;
  return s == hipStreamPerThread ? per_thread[thread_now] : *s;
}

hipError_t enqueue(hipStream_t s) {
  ihipStream_t& t = at(s);
  ops.push_back({t.before});
  t.before.insert((int)ops.size() - 1);
  return hipSuccess;
}

}  // namespace

const char* hipGetErrorString(hipError_t) { return "model error"; }
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipGetDevice(int* device) { return *device = 0, hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* value, hipDeviceAttribute_t, int) { return *value = 256, hipSuccess; }
hipError_t hipMalloc(void** p, size_t bytes) {
  *p = std::aligned_alloc(256, 256 + (bytes < 4096 ? (bytes + 255) / 256 * 256 : 4096));   // never read
  return *p ? hipSuccess : hipErrorOutOfMemory;
}
hipError_t hipFree(void* p) {
  for (int i = 0; i < (int)ops.size(); ++i)
    if (!finished.count(i)) freed_early.insert(i);
  std::free(p);
  return hipSuccess;
}
hipError_t hipMemcpy(void*, const void*, size_t, hipMemcpyKind) { return hipSuccess; }
hipError_t hipMemcpyAsync(void*, const void*, size_t, hipMemcpyKind, hipStream_t s) { return enqueue(s); }
hipError_t hipStreamCreateWithFlags(hipStream_t* s, unsigned) {
  internal.push_back(*s = new ihipStream_t);
  return hipSuccess;
}
hipError_t hipStreamDestroy(hipStream_t s) {
  internal.erase(std::remove(internal.begin(), internal.end(), s), internal.end());
  delete s;
  return hipSuccess;
}
hipError_t hipStreamSynchronize(hipStream_t s) {
  finished.insert(at(s).before.begin(), at(s).before.end());
  return hipSuccess;
}
hipError_t hipStreamWaitEvent(hipStream_t s, hipEvent_t e, unsigned) {
  ihipStream_t& t = at(s);
  if (!e->recorded) return hipSuccess;
  // an event may not be waited for across the boundary of a capture, except
  // that it brings a stream into the capture it was recorded in
  if (t.capture && t.capture != e->capture) return hipErrorStreamCaptureIsolation;
  if (!t.capture && e->capture) t.capture = e->capture, t.before.clear();
  t.before.insert(e->before.begin(), e->before.end());
  return hipSuccess;
}
hipError_t hipStreamIsCapturing(hipStream_t s, hipStreamCaptureStatus* status) {
  return *status = at(s).capture ? hipStreamCaptureStatusActive : hipStreamCaptureStatusNone, hipSuccess;
}
hipError_t hipStreamGetCaptureInfo(hipStream_t s, hipStreamCaptureStatus* status, unsigned long long* id) {
  *id = at(s).capture;
  return hipStreamIsCapturing(s, status);
}
hipError_t hipEventCreate(hipEvent_t* e) { return *e = new ihipEvent_t, hipSuccess; }
hipError_t hipEventCreateWithFlags(hipEvent_t* e, unsigned) { return hipEventCreate(e); }
hipError_t hipEventDestroy(hipEvent_t e) { return delete e, hipSuccess; }
hipError_t hipEventRecord(hipEvent_t e, hipStream_t s) {
  *e = ihipEvent_t{at(s).before, true, at(s).capture};
  return hipSuccess;
}
hipError_t hipEventSynchronize(hipEvent_t e) {
  if (e->capture) return hipErrorCapturedEvent;
  finished.insert(e->before.begin(), e->before.end());
  return hipSuccess;
}
hipError_t hipEventElapsedTime(float* ms, hipEvent_t, hipEvent_t) { return *ms = 1.0f, hipSuccess; }

namespace agmm {
int tile_bm(int) { return 128; }
int tile_bn(int) { return 128; }
int tile_bk(int) { return 64; }
int tile_occ(int) { return 1; }
hipError_t launch_gemm_mfma(const GemmProblem&, int, int, bool, hipStream_t s) { return enqueue(s); }
hipError_t launch_skinny_fullk(const GemmProblem&, int, int, hipStream_t s) { return enqueue(s); }
hipError_t launch_splitk_reduce(const GemmProblem&, int, hipStream_t s) { return enqueue(s); }
hipError_t launch_gemm_f32(const GemmProblem&, bool, hipStream_t s) { return enqueue(s); }
hipError_t launch_gather(const GatherProblem&, int, hipStream_t s) { return enqueue(s); }
hipError_t launch_pad_copy(const PadCopyProblem&, hipStream_t s) { return enqueue(s); }
hipError_t launch_transpose16(const void*, int64_t, int64_t, int64_t, void*, hipStream_t s) { return enqueue(s); }
hipError_t noalloc_scratch(void**) { return hipErrorInvalidSymbol; }
hipError_t launch_quantize(const QuantProblem&, hipStream_t s) { return enqueue(s); }
hipError_t launch_scaled(const ScaledProblem&, int, hipStream_t s) { return enqueue(s); }
// (the loss's products: with the limit on the workgroups of a launch)
constexpr int64_t kGrid = int64_t(1) << 24;
int64_t tiles(const GemmProblem& p) { return (int64_t)p.order.num_rb * p.order.num_cb; }
hipError_t launch_loss_logits(const LossProblem& p, int, bool, hipStream_t s) {
  return tiles(p.gemm) < kGrid ? enqueue(s) : hipErrorInvalidValue;
}
hipError_t launch_loss_few(const LossProblem& p, int, int, int, bool, hipStream_t s) {
  return tiles(p.gemm) < kGrid ? enqueue(s) : hipErrorInvalidValue;
}
hipError_t launch_loss_combine(const LossCombine&, hipStream_t s) { return enqueue(s); }
hipError_t launch_loss_prepare(const LossRows*, const PadRows*, int, hipStream_t s) { return enqueue(s); }
hipError_t launch_loss_grads(const GemmProblem* a, bool, const GemmProblem* w, const float*, int, int, hipStream_t s) {
  return (a ? tiles(*a) * a->splits : 0) + (w ? tiles(*w) : 0) < kGrid ? enqueue(s) : hipErrorInvalidValue;
}
hipError_t launch_loss_da_finish(const LossFinish&, int, hipStream_t s) { return enqueue(s); }
}  // namespace agmm

namespace {

alignas(256) char memory[4096];
int failures = 0;

void expect(bool is, const std::string& what) {
  if (is) return;
  std::printf("FAILED: %s\n", what.c_str());
  ++failures;
}

// A plan of one of the kinds, and its calls.
struct Plan {
  std::string name;
  std::function<int(hipStream_t)> run;
  std::function<void()> destroy;

  // the operations of a call
  std::vector<int> call(hipStream_t s) const {
    const int first = (int)ops.size();
    expect(run(s) == AGMM_OK, name + ": " + agmm_last_error());
    std::vector<int> mine;
    for (int i = first; i < (int)ops.size(); ++i) mine.push_back(i);
    expect(!mine.empty(), name + ": a call without work");
    return mine;
  }
};

// The end of a capture: streams that joined it are ordinary ones again.
void end_capture() {
  for (ihipStream_t* s : internal)
    if (s->capture) *s = ihipStream_t{};
}

bool after(const std::vector<int>& later, const std::vector<int>& earlier) {
  for (int b : later)
    for (int a : earlier)
      if (!ops[b].before.count(a)) return false;
  return true;
}

const void* shard_list[2] = {memory, memory};
const float* scale_list[2] = {reinterpret_cast<float*>(memory), reinterpret_cast<float*>(memory)};

Plan make(int kind) {
  void* m = memory;
  float* f = reinterpret_cast<float*>(memory);
  int64_t* l = reinterpret_cast<int64_t*>(memory);
  if (kind == 0) {
    agmm_scaled_plan_t p = agmm_scaled_plan_create(2, 8, 4096, 64, AGMM_E4M3, 128, AGMM_BF16);
    expect(p && agmm_scaled_plan_set_int(p, "splits", 4) == AGMM_OK, "scaled plan");
    return {"scaled product in k ranges", [=](hipStream_t s) { return agmm_scaled_run(p, shard_list, scale_list, m, f, m, s); },
            [=] { agmm_scaled_plan_destroy(p); }};
  }
  if (kind <= 2) {
    agmm_loss_plan_t p = agmm_loss_plan_create(2, 8, 64, 512, AGMM_FP16, 0, 512, 1);
    expect(p, "loss plan");
    if (kind == 1)
      return {"loss", [=](hipStream_t s) { return agmm_loss_forward(p, shard_list, m, l, f, f, f, s); }, [=] { agmm_loss_plan_destroy(p); }};
    return {"loss gradient", [=](hipStream_t s) { return agmm_loss_backward(p, shard_list, m, l, f, f, f, m, m, s); },
            [=] { agmm_loss_plan_destroy(p); }};
  }
  agmm_plan_t p = agmm_plan_create(2, 64, 4096, 128, AGMM_BF16, 1);
  expect(p, "matmul plan");
  const int v = kind == 3 ? AGMM_VARIANT_UNFUSED : AGMM_VARIANT_STAGED;
  expect(agmm_plan_set_int(p, "variant", v) == AGMM_OK, agmm_last_error());
  return {kind == 3 ? "matmul, unfused" : "matmul, staged", [=](hipStream_t s) { return agmm_run(p, shard_list, m, m, s); },
          [=] { agmm_plan_destroy(p); }};
}

void check(int kind) {
  ihipStream_t s[4], c1, c2, d1;
  Plan p = make(kind);
  const auto says = [&](const char* what) { return p.name + ": " + what; };

  const std::vector<int> e1 = p.call(&s[0]);
  const std::vector<int> e2 = p.call(&s[1]);
  expect(after(e2, e1), says("two streams"));

  // a call captured into a graph between two eager ones
  c1.capture = 7;
  const std::vector<int> g1 = p.call(&c1);
  end_capture();
  const std::vector<int> e3 = p.call(&s[2]);
  expect(after(e3, e2), says("eager, captured, eager"));

  if (kind != 4) {   // (a graph holds at most one staged call)
    // an eager call between two of one capture
    c2.capture = 7;
    const std::vector<int> g2 = p.call(&c2);
    expect(after(g2, g1), says("captured, eager, captured in the same graph"));
    // and a call of another graph
    d1.capture = 8;
    p.call(&d1);
    ihipStream_t c3;
    c3.capture = 7;
    expect(after(p.call(&c3), g2), says("two graphs by turns"));
  }

  // the default stream, before and after others
  const std::vector<int> e4 = p.call(nullptr);
  expect(after(e4, e3), says("the default stream after another"));
  std::vector<int> e5 = p.call(&s[3]);
  expect(after(e5, e4), says("another stream after the default one"));

  // handles that do not name one stream: a thread's own default stream, and a
  // handle that a new stream got after the old one's end
  const std::vector<int> t0 = p.call(hipStreamPerThread);
  thread_now = 1;
  const std::vector<int> t1 = p.call(hipStreamPerThread);
  thread_now = 0;
  expect(after(t1, t0), says("the default streams of two threads"));
  const std::vector<int> old = p.call(&s[0]);
  s[0] = ihipStream_t{};
  e5 = p.call(&s[0]);
  expect(after(e5, old), says("a stream with the handle of one that ended"));

  // a plan's end waits for its last eager call, also where one was captured after it
  d1 = ihipStream_t{};
  d1.capture = 9;
  p.call(&d1);
  end_capture();
  freed_early.clear();
  p.destroy();
  for (int o : e5) expect(!freed_early.count(o), says("freed while an eager call may run"));
}

// Pieces and tiles of the loss that a launch cannot hold are refused when they
// are set; what was accepted runs.
void check_pieces(int64_t m, int64_t k, int64_t n, int64_t tile, int64_t piece, bool gradient, bool accepted) {
  const std::string what = "piece of " + std::to_string(piece) + " by tile " + std::to_string(tile) + (gradient ? ", gradient" : "");
  agmm_loss_plan_t p = agmm_loss_plan_create(1, m, k, n, AGMM_BF16, 0, n, gradient);
  expect(p && agmm_loss_plan_set_int(p, "tile", tile) == AGMM_OK, what + ": tile");
  int64_t before = 0, after = 0;
  agmm_loss_plan_get_int(p, "piece", &before);
  const int rc = agmm_loss_plan_set_int(p, "piece", piece);
  expect(rc == (accepted ? AGMM_OK : AGMM_ERR_UNSUPPORTED), what + ": status " + std::to_string(rc));
  agmm_loss_plan_get_int(p, "piece", &after);
  expect(accepted || after == before, what + ": the plan keeps its piece");
  float* f = reinterpret_cast<float*>(memory);
  int64_t* l = reinterpret_cast<int64_t*>(memory);
  ihipStream_t s;
  int run = agmm_loss_forward(p, shard_list, memory, l, f, f, f, &s);
  if (run == AGMM_OK && gradient) run = agmm_loss_backward(p, shard_list, memory, l, f, f, f, memory, memory, &s);
  expect(run == AGMM_OK, what + ": " + agmm_last_error());
  agmm_loss_plan_destroy(p);
}

}  // namespace

int main(int argc, char** argv) {
  if (argc > 1) {
    check_pieces(int64_t(1) << 19, 8, int64_t(1) << 20, 128, int64_t(1) << 20, false, false);   // 2^25 tiles
    check_pieces(int64_t(1) << 19, 8, int64_t(1) << 20, 256, int64_t(1) << 20, false, true);    // 2^23
    check_pieces(int64_t(1) << 19, 8, int64_t(1) << 20, 128, int64_t(1) << 18, false, true);
    check_pieces(8, int64_t(1) << 16, int64_t(1) << 23, 128, int64_t(1) << 23, true, false);    // dW: 2^25 tiles
    check_pieces(8, int64_t(1) << 16, int64_t(1) << 23, 128, int64_t(1) << 20, true, true);
    check_pieces(16, 64, (int64_t(1) << 27) - 1, 64, (int64_t(1) << 30) - 1, false, true);
  } else {
    for (int kind = 0; kind < 5; ++kind) check(kind);
  }
  if (!failures) std::printf("all in order\n");
  return failures != 0;
}
