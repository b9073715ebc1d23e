// What the operators' plans share (agmm_ops.cpp, agmm_feed.cpp): size rules,
// the workspace, and the order of a plan's calls.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <mutex>
#include <string>

#include "agmm_host.h"

namespace agmm {

inline int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Shard counts and sizes every plan here accepts (the all-gather matmul's
// rules).
inline int check_sizes(int N, int64_t m_s, int64_t k, int64_t n) {
  const int rc = check_counts(N, m_s, k, n);
  return rc == AGMM_OK ? check_limits(N, m_s, k, n) : rc;
}

// What every plan here owns: its device, a workspace, and the order of its
// calls.
struct PlanBase {
  int device = 0;
  int cu_count = 256;
  char* ws = nullptr;
  size_t ws_bytes = 0;
  CallOrder order;
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
    Call c;
    int rc = CallOrder::look(s, c);
    if (rc == AGMM_OK && c.capturing) captured = true;
    if (rc == AGMM_OK && ordered) rc = order.enter(c);
    if (rc != AGMM_OK) return rc;
    rc = body();
    if (!ordered) return rc == AGMM_OK ? ok() : rc;
    if (rc != AGMM_OK) {
      // whatever was enqueued before the failure still counts
      const int st = g_status;
      const std::string msg = g_msg;
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
inline int check_ptr(const void* p, const char* name, int index, uintptr_t to) {
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
inline int group_rows(int64_t nrb, int64_t ncb) {
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

}  // namespace agmm
