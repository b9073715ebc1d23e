// Status and plan bookkeeping shared by the host sources of the C ABI
// (agmm_api.cpp, agmm_ops.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <string>
#include <vector>

#include "agmm.h"
#include "agmm_kernels.h"

namespace agmm {

// Status and message of this thread's most recent call into the library.
inline thread_local int g_status = AGMM_OK;
inline thread_local std::string g_msg;

inline int set_err(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_status = status;
  g_msg = buf;
  return status;
}

inline int ok() {
  g_status = AGMM_OK;
  g_msg.clear();
  return AGMM_OK;
}

inline int hip_err(hipError_t e, const char* what) {
  return set_err(AGMM_ERR_HIP, "%s failed: %s", what, hipGetErrorString(e));
}

// Limits of a plan's sizes: m = num_shards * m_per_shard, k and n, and the
// elements of any matrix between them.
constexpr int64_t kDimLimit = int64_t(1) << 30;
constexpr int64_t kElemLimit = int64_t(1) << 40;

inline int check_counts(int N, int64_t m_s, int64_t k, int64_t n) {
  if (N < 1) return set_err(AGMM_ERR_INVALID_ARG, "num_shards must be >= 1 (got %d)", N);
  if (N > kMaxGroups)
    return set_err(AGMM_ERR_UNSUPPORTED, "num_shards %d exceeds the supported maximum %d", N, kMaxGroups);
  if (m_s < 1 || k < 1 || n < 1)
    return set_err(AGMM_ERR_INVALID_ARG, "sizes must be >= 1 (m_per_shard=%lld, k=%lld, n_local=%lld)",
                   (long long)m_s, (long long)k, (long long)n);
  return AGMM_OK;
}

inline int check_limits(int N, int64_t m_s, int64_t k, int64_t n) {
  // m_s first: N * m_s must not overflow
  const int64_t m = m_s < kDimLimit ? N * m_s : m_s;
  if (m >= kDimLimit || k >= kDimLimit || n >= kDimLimit || m * k >= kElemLimit || k * n >= kElemLimit ||
      m * n >= kElemLimit)
    return set_err(AGMM_ERR_UNSUPPORTED, "problem too large (m=%lld, k=%lld, n=%lld)", (long long)m, (long long)k,
                   (long long)n);
  return AGMM_OK;
}

// One call's view of the caller's stream.
struct Call {
  hipStream_t s = nullptr;
  bool capturing = false;
  unsigned long long capture_id = 0;
};

// The order of a plan's calls: a call's stream waits for the plan's previous
// call before any work of its own, so that no two calls use the workspace at
// one time.  The eager calls and the calls of each graph capture are chains of
// their own, each with its event: an event recorded on one side of a capture
// boundary must not be waited for on the other, a captured call's work happens
// at each replay (the caller's streams order replays), and a call of one chain
// between two of another must not make the second forget the first.
class CallOrder {
 public:
  int create(int device) {
    device_ = device;
    return make(&eager_.event);
  }

  // After the last use; create() may have failed or not been called.
  void destroy() {
    if (eager_.event) hipEventDestroy(eager_.event);
    for (const Chain& c : captured_) hipEventDestroy(c.event);
    eager_ = Chain{};
    captured_.clear();
  }

  // Find out whether `s` is being captured into a graph (the default stream
  // cannot be).
  static int look(hipStream_t s, Call& c) {
    c = Call{};
    c.s = s;
    if (!s) return AGMM_OK;
    hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
    unsigned long long id = 0;
    const hipError_t err = hipStreamGetCaptureInfo(s, &st, &id);
    if (err != hipSuccess) return hip_err(err, "hipStreamGetCaptureInfo");
    if (st == hipStreamCaptureStatusInvalidated)
      return set_err(AGMM_ERR_HIP, "the stream's graph capture has been invalidated");
    c.capturing = st == hipStreamCaptureStatusActive;
    c.capture_id = c.capturing ? id : 0;
    return AGMM_OK;
  }

  // Order a call after its chain's previous one.
  int enter(const Call& c) {
    const Chain* chain = find(c);
    if (!chain || !chain->begun || same_stream(*chain, c)) return AGMM_OK;
    if (!chain->stream) {
      const int rc = on_device([](CallOrder* o) { return hipEventRecord(o->eager_.event, nullptr); }, "hipEventRecord(done)");
      if (rc != AGMM_OK) return rc;
    }
    const hipError_t err = hipStreamWaitEvent(c.s, chain->event, 0);
    return err == hipSuccess ? AGMM_OK : hip_err(err, "hipStreamWaitEvent(done)");
  }

  // End a call: everything it enqueued is on, or has joined, its stream.  The
  // default stream needs no event per call: it never ends, so what orders a
  // later call after it is recorded, or waited for, when that time comes.
  int leave(const Call& c) {
    Chain* chain = find(c);
    if (!chain) {
      Chain made;
      made.capture = c.capture_id;
      const int rc = make(&made.event);
      if (rc != AGMM_OK) return rc;
      captured_.push_back(made);
      chain = &captured_.back();
    }
    if (c.s) {
      const hipError_t err = hipEventRecord(chain->event, c.s);
      if (err != hipSuccess) return hip_err(err, "hipEventRecord(done)");
    }
    chain->begun = true;
    chain->stream = c.s;
    return AGMM_OK;
  }

  // Wait on the host for the plan's last eager call.
  int idle() {
    if (!eager_.begun) return AGMM_OK;
    if (!eager_.stream)
      return on_device([](CallOrder*) { return hipStreamSynchronize(nullptr); }, "hipStreamSynchronize");
    const hipError_t err = hipEventSynchronize(eager_.event);
    return err == hipSuccess ? AGMM_OK : hip_err(err, "hipEventSynchronize(done)");
  }

 private:
  struct Chain {
    hipEvent_t event = nullptr;        // end of its last call (a call on the default stream: not recorded yet)
    hipStream_t stream = nullptr;      // that call's stream
    bool begun = false;
    unsigned long long capture = 0;
  };

  // Whether the chain's last call is on the call's very stream, which orders the
  // two by itself.  Equal handles do not say so: a stream's handle is given to
  // another after its end, while its work may still run, and
  // hipStreamPerThread is a stream of each host thread.  The default stream
  // does not end, nor does a stream during its capture.
  static bool same_stream(const Chain& chain, const Call& c) {
    return chain.stream == c.s && (c.capturing ? c.s != hipStreamPerThread : !c.s);
  }

  // The chain a call belongs to, or NULL for the first call of a capture.
  Chain* find(const Call& c) {
    if (!c.capturing) return &eager_;
    for (Chain& k : captured_)
      if (k.capture == c.capture_id) return &k;
    return nullptr;
  }

  static int make(hipEvent_t* e) {
    const hipError_t err = hipEventCreateWithFlags(e, hipEventDisableTiming);
    return err == hipSuccess ? AGMM_OK : hip_err(err, "hipEventCreate");
  }

  // The default stream is the current device's: make that the plan's.
  int on_device(hipError_t (*f)(CallOrder*), const char* what) {
    int dev = device_;
    hipError_t err = hipGetDevice(&dev);
    if (err == hipSuccess && dev != device_) err = hipSetDevice(device_);
    if (err == hipSuccess) err = f(this);
    if (dev != device_) (void)hipSetDevice(dev);
    return err == hipSuccess ? AGMM_OK : hip_err(err, what);
  }

  int device_ = 0;
  Chain eager_;
  std::vector<Chain> captured_;        // one for every graph a call was captured into
};

}  // namespace agmm
