// What the loss's row copy refuses, called in the built library (no GPU: a call
// that is accepted ends with another error; hipErrorInvalidValue is 1 in the model's
// header, with which this is compiled, as in the runtime's).
#include <hip/hip_runtime.h>

#include <cstdio>
#include <initializer_list>

#include "ops_kernels.h"

int main() {
  int failures = 0;
  const auto refused = [&](int64_t cols, int64_t chunks, int64_t groups = 1, int64_t rows = 4) {
    agmm::PadRows c{};
    c.num_groups = groups;
    c.rows = rows;
    c.cols = c.ld = cols;
    c.chunks = chunks;
    const hipError_t err = agmm::launch_loss_prepare(nullptr, &c, agmm::kDtypeBf16, nullptr);
    if (err == hipErrorInvalidValue) return;
    std::printf("FAILED: %lld columns in %lld pieces of 8 (%lld x %lld rows): %d\n", (long long)cols, (long long)chunks, (long long)groups,
                (long long)rows, (int)err);
    ++failures;
  };
  for (int64_t cols : {1, 7, 8, 9, 100, 2124}) {
    const int64_t chunks = (cols + 7) / 8;
    refused(cols, chunks + 1);                 // pieces without a column
    refused(cols, chunks + 8);
    refused(cols, chunks - 1);                 // columns without a piece
  }
  refused(100, 13, 0);
  refused(100, 13, agmm::kMaxGroups + 1);
  refused(100, 13, 1, 0);
  if (!failures) std::printf("all as expected\n");
  return failures ? 1 : 0;
}
