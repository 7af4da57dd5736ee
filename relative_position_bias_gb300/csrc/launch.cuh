// Host-side launchers of the kernel templates; each padded width WP is
// instantiated in its own translation unit so the build compiles in parallel.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"

namespace dera {

// Sets up a kernel once per device: its dynamic shared memory, and, where its warps split their registers,
// that it compiled to the count the split was computed for (with fewer the split would wait for ever, so
// the launch is refused).
template <class K>
inline cudaError_t prepare_kernel(K kernel, int smem, int launch_regs, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  if (launch_regs > 0) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < launch_regs) return cudaErrorInvalidKernelImage;
  }
  if (dev < 64) done.fetch_or(bit, std::memory_order_release);
  return cudaSuccess;
}

struct AttnMaps {
  CUtensorMap q, k, v, th, tw;
};

template <int WP>
cudaError_t launch_attention(const AttnMaps& maps, const AttnArgs& args, int ctas, bool fused, int head_dim,
                             cudaStream_t stream);

cudaError_t launch_project(const CUtensorMap& q, const CUtensorMap& th, const CUtensorMap& tw,
                           const ProjArgs& args, int in_fmt, int head_dim, int max_ctas, cudaStream_t stream);

cudaError_t launch_wait_selftest(int* status, long long budget, cudaStream_t stream);

struct BwdMaps {
  CUtensorMap q, dout, k, v, th, tw;
};

// The backward's attention kernels and its table reduction for head_dim 64, in
// stream order; the compact rel_h, rel_w in args must already be written.
cudaError_t launch_backward(const BwdMaps& maps, const BwdArgs& args, int WP, cudaStream_t stream);

}  // namespace dera
