// vdit_internal.h - what the library's translation units share on the host side.
#pragma once

#include <cuda_runtime.h>

namespace vdit {

// Launches `kernel` so that its CTAs may start while the kernel before it in the
// stream still runs (programmatic dependent launch), once that kernel has called
// let_next_start().  Saves about 1 us between kernels that take little more (the
// selection at 512 tokens: 30.1 to 27.8 us).  Every thread of `kernel` must call
// wait_for_previous() before it reads anything or returns, also where it has nothing
// to do: the kernel after it waits for it alone, and would else start while the one
// before still writes to memory that the caller has back by then.  The watchdog's
// flag is read after that wait too, so that the previous kernel's waits are in it.
// What the kernel before writes is not read-only for the lifetime of `kernel`: it is
// read by plain loads or __ldcg, never by __ldg or through a __restrict__ pointer
// (the compiler may take the non-coherent path there, and move the load ahead of
// the wait).
template <typename... P, typename... A>
bool launch_early(void (*kernel)(P...), dim3 grid, unsigned threads, cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess;
}

#ifdef __CUDACC__
// The kernel before this one has completed and its writes are visible.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel's CTAs may take what room there is.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

// Device address, on the current device, of the watchdog's flag word, or null
// if the runtime reports an error.  The flag is one device symbol of
// vdit_api.cu; kernels of other translation units take its address as an
// argument.
const unsigned int* watchdog_flag();

// 128-token blocks of a sequence.
inline int sparse_blocks(int L) { return (int)(((long long)L + 127) / 128); }

}  // namespace vdit
