// block_common.h -- what the translation units of the block operators' C ABI
// share: type and overlap checks, and the scratch of one call.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/delta.h"
#include "api_common.h"

namespace delta {
namespace api {

constexpr int64_t kMaxElems = int64_t(1) << 40;  // products of sizes stay far inside 64 bits

inline int64_t esize(delta_dtype dt) { return dt == DELTA_BF16 ? 2 : 4; }

inline int check_dtype(delta_dtype dt) {
  return dt == DELTA_F32 || dt == DELTA_BF16 ? DELTA_OK : fail(DELTA_ERR_INVALID, "unknown dtype %d", (int)dt);
}

inline bool aligned_to(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)n == 0; }

// no output may overlap an input or another output; where one may be updated
// in place the caller leaves that pair out
struct Span {
  const char *name;
  Range r;
};
template <int NO, int NI>
int check_overlap(const Span (&outs)[NO], const Span (&ins)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlap(outs[i].r, ins[j].r))
        return fail(DELTA_ERR_INVALID, "%s overlaps %s", outs[i].name, ins[j].name);
    for (int j = i + 1; j < NO; ++j)
      if (overlap(outs[i].r, outs[j].r))
        return fail(DELTA_ERR_INVALID, "%s overlaps %s", outs[i].name, outs[j].name);
  }
  return DELTA_OK;
}

inline int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Stream-ordered scratch of one call, cut into 256-byte pieces.
struct Scratch {
  void *base = nullptr;
  int64_t used = 0, size = 0;
  cudaStream_t s;
  explicit Scratch(cudaStream_t st) : s(st) {}
  void want(int64_t bytes) { size += up(bytes, 256); }
  cudaError_t take() {
    if (size == 0) return cudaSuccess;
    cudaMemPool_t pool;
    const cudaError_t e = scratch_pool(&pool);
    return e != cudaSuccess ? e : cudaMallocFromPoolAsync(&base, (size_t)size, pool, s);
  }
  void *cut(int64_t bytes) {
    void *p = static_cast<unsigned char *>(base) + used;
    used += up(bytes, 256);
    return p;
  }
  cudaError_t release() { return base ? cudaFreeAsync(base, s) : cudaSuccess; }
};

}  // namespace api
}  // namespace delta
