// A kernel that follows another in a stream and may start before it ends: its
// CTAs come up, and do what needs nothing of the kernel before, while that one
// drains.  The scan's kernels do without let_next_start(): CTAs that come up as
// single slots fall free crowd on the first SMs (the backward pass's carry
// kernel and, B1 L512 E2048 N16, its main kernel: 53 us against 46; B2 L4096
// E1024 N32: 385 against 381).
#pragma once
#include <cuda_runtime.h>

#include <utility>

namespace linattn {

// In the kernel before: the next one may be brought up once every CTA has got
// here (or ended).
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// In the kernel behind: everything that the kernel before has written is there
// after this (nothing to wait for in an ordinary launch).
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One split of an SM's memory between shared memory and L1 (the most shared
// memory) for the kernels of a chain: a kernel that wants another split than
// the one before waits for an empty SM, 6 us (forward pass of B2 L4096 E2048,
// fp32 and 16 states: 160 us against 151; bf16 and 8 states: 110 against 106).
template <typename K>
cudaError_t most_shared(K *kernel) {
  return cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                              cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
}

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid_x, unsigned grid_y, unsigned threads,
                             size_t smem, cudaStream_t s, A &&...args) {
  cudaLaunchAttribute attr[1] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid_x, grid_y);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace linattn
