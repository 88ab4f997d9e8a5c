// Launching a kernel so that it may start while the one before it in the
// stream ends (programmatic dependent launch), and the device's side of it.
//
// A kernel launched by launch_after() calls let_next_start() at once and
// after_prior() before it touches global memory: until then it may only set up
// shared memory.  after_prior() returns when everything before the launch is
// complete and visible.  Pointers handed to it come back as new values, so no
// load through them can be moved above the wait.  What they point at changes
// while the kernel is already resident, so it is read by ordinary loads, never
// by the read-only ones (__ldg, ld.global.nc), which hold for data that stays
// as it is from the kernel's first instruction to its last.
#pragma once

#include <cuda_runtime.h>

namespace kvz {

template <class... K, class... A>
cudaError_t launch_after(void (*kernel)(K...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, int cluster,
                         A&&... args) {
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, K(args)...);
}

__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <class... P>
__device__ __forceinline__ void after_prior(P*&... ptr) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  ((void)([&] { asm volatile("" : "+l"(ptr)::"memory"); }()), ...);
}

}  // namespace kvz
