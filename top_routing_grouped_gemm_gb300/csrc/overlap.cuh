// Launches that are set up while the kernel before them in the stream ends.
//
// A kernel launched so begins with after_previous(), before it reads or writes memory of the caller's:
// there it waits until the kernel before it has ended and its writes are seen, so the stream's order
// holds as ever, for plain loads (what is read-only for a kernel's whole life is another matter: no
// __ldg and no restricted pointers here).  What is saved is the launch itself (0.4 us of a one-token
// step of 2.3 us in a graph; calls one after the other: 8192 x 4096 recurrence forward + backward
// 129 -> 124 us, norm + rotation's backward of 32768 x 32 x 128 185 -> 174 us).  No kernel lets the
// next one in before its own blocks end: those took the first places that came free, unevenly
// (124 -> 128 us).
#pragma once

#include <cuda_runtime.h>

namespace moe {

// (Without effect in an ordinary launch.)
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

inline cudaLaunchAttribute behind_previous() {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  return attr;
}

// A launch's own error, which is not left behind for a later call to find.
inline cudaError_t launched(cudaError_t err) {
  if (err != cudaSuccess) cudaGetLastError();
  return err;
}

template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, int threads, int smem,
                          cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr = behind_previous();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return launched(cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...));
}

}  // namespace moe
