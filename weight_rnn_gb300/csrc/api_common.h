// api_common.h -- what the translation units of the C ABI share: the thread's
// last error, the failure hook, the scratch pool and pointer checks.  Defined
// in api.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace delta {
namespace api {

constexpr int kMaxDevices = 64;

// true (and one injection used up) when this call is to fail on purpose
bool take_injection();

// record the message and return the status
int fail(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int cuda_fail(cudaError_t err, const char *what);

// the library's memory pool on the current device
cudaError_t scratch_pool(cudaMemPool_t *out);

inline bool aligned16(const void *p) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};
inline Range range(const void *p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + (uintptr_t)bytes};
}
inline bool overlap(Range a, Range b) {
  return a.lo != 0 && b.lo != 0 && a.hi > a.lo && b.hi > b.lo && a.lo < b.hi && b.lo < a.hi;
}

}  // namespace api
}  // namespace delta
