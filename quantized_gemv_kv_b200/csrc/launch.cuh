// Launches that may be prepared while the previous kernel of the stream still
// runs (programmatic stream serialization).  A kernel launched this way calls
// wait_for_previous() before it touches memory, so the stream's order is the
// usual one; what overlaps is the launch itself (1.5 us of a call between
// kernels that follow one another).
#pragma once

#include <atomic>

#include "sf_internal.h"

namespace sfd {

// Until the kernels before this one have ended and their writes are visible.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel be prepared; it waits for this one's end all the same.
__device__ __forceinline__ void let_next_prepare() { asm volatile("griddepcontrol.launch_dependents;"); }

}  // namespace sfd

namespace sf {

// Lets a kernel have `bytes` of dynamic shared memory (and, where `wide`, clusters of sixteen blocks): told once per
// device.  A kernel's limit is one for the whole process, so the number must not depend on the call: another thread's
// could come between this one and the launch.  told: one variable per kernel, of devices that know.
template <class P>
sf_status allow_smem(void (*kernel)(P), size_t bytes, std::atomic<unsigned long long>& told, bool wide = false) {
  int dev = 0;
  SF_CHECK_CUDA(cudaGetDevice(&dev));
  const unsigned long long bit = 1ull << (dev & 63);
  if ((told.load(std::memory_order_relaxed) & bit) != 0) return SF_OK;
  SF_CHECK_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)));
  if (wide) SF_CHECK_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
  if (dev < 64) told.fetch_or(bit, std::memory_order_relaxed);
  return SF_OK;
}

// cluster: blocks per thread-block cluster (1: none).
template <class P>
sf_status launch(const char* what, void (*kernel)(P), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s,
                 const P& params) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, params);
  if (e != cudaSuccess) {
    cudaGetLastError();  // not left for a later call to find
    return cuda_fail(e, what);
  }
  return SF_OK;
}

}  // namespace sf
