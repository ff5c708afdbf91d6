// chain.cuh -- kernels that follow one another on a stream: a kernel launched as
// a dependent may start while the one before it ends, sets itself up, and waits
// with chain_wait() for that kernel's end and memory before it reads or writes
// any.  Every thread of it waits, so that its own end implies the end of all
// before it.  A call's first kernel is a dependent too, but where the call goes
// on to the tensor-core product: that takes tensor memory while it waits, and a
// caller's kernel before it may have yet to take some.
// A gap between two kernels shrinks from about 2.5 us to 1.
#pragma once

#include <cuda_runtime.h>

namespace delta {

__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel's CTAs may take the places that this one leaves free: for a
// next kernel of the same call.  A call's last kernel leaves it out, since CTAs
// that come one by one crowd on the SMs that are free first.
__device__ __forceinline__ void chain_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t chain_launch(void (*kern)(P...), dim3 grid, dim3 block, int smem, int cluster, bool dependent,
                         cudaStream_t s, A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  int n = 0;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = (unsigned)cluster;
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  if (dependent) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = (unsigned)n;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

}  // namespace delta
