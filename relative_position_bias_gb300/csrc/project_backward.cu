// Launch of the projection's backward (project_backward.cuh).
#include "project_backward.cuh"

#include <atomic>

namespace dera {

template <bool BF16>
static cudaError_t launch_pb_t(const PbArgs& a, int ctas, cudaStream_t s) {
  auto kernel = relpos_pb_kernel<BF16>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PbSmem<BF16>::kAlloc);
  if (e != cudaSuccess) return e;
  // The register split needs the launch pool it was computed for; a build that compiled to fewer
  // registers is refused rather than launched into a wait that never ends.
  static std::atomic<int> fits{0};   // 0 unknown, 1 fits, -1 refused
  if (fits.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    fits.store(fa.numRegs >= kPbLaunchRegs ? 1 : -1, std::memory_order_relaxed);
  }
  if (fits.load(std::memory_order_relaxed) < 0) return cudaErrorInvalidKernelImage;
  kernel<<<dim3(ctas, a.D / 64), kPbThreads, PbSmem<BF16>::kAlloc, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int total = (2 * a.H - 1 + 2 * a.W - 1) * a.D;
  relpos_pb_tables_kernel<<<total / 32, 256, 0, s>>>(a, ctas);
  return cudaGetLastError();
}

cudaError_t launch_project_backward(const PbArgs& a, int ctas, bool bf16, cudaStream_t s) {
  return bf16 ? launch_pb_t<true>(a, ctas, s) : launch_pb_t<false>(a, ctas, s);
}

}  // namespace dera
