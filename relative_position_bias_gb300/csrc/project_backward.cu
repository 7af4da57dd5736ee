// Launch of the projection's backward (project_backward.cuh).
#include "launch.cuh"
#include "project_backward.cuh"

namespace dera {

template <bool BF16>
static cudaError_t launch_pb_t(const PbArgs& a, int ctas, cudaStream_t s) {
  auto kernel = relpos_pb_kernel<BF16>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = prepare_kernel(kernel, PbSmem<BF16>::kAlloc, kPbLaunchRegs, done);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(ctas, a.D / 64), kPbThreads, PbSmem<BF16>::kAlloc, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int total = (2 * a.H - 1 + 2 * a.W - 1) * a.D;
  return launch_early(relpos_pb_tables_kernel, dim3(total / 32), dim3(256), 0, s, a, ctas);
}

cudaError_t launch_project_backward(const PbArgs& a, int ctas, bool bf16, cudaStream_t s) {
  return bf16 ? launch_pb_t<true>(a, ctas, s) : launch_pb_t<false>(a, ctas, s);
}

}  // namespace dera
