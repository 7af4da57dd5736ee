#include "linear_inst.cuh"

namespace dera {
int few_clusters(int size) {
  static std::atomic<int> known[64][3];   // 1 + the number, by device and size
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 0;
  std::atomic<int>& n = known[dev][size == 2 ? 0 : (size == 4 ? 1 : 2)];
  if (n.load() > 0) return n.load() - 1;
  // all of them have one CTA an SM, by their shared memory
  auto kernel = linear_few_kernel<kLinForward, 32, true>;
  static_assert(2 * LinSmem<32>::kAlloc > 228 * 1024 && 2 * LinSmem<64>::kAlloc > 228 * 1024);
  static std::atomic<unsigned long long> done{0};
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg;
  cluster_launch(&cfg, &attr, size, LinSmem<32>::kAlloc);
  cfg.gridDim = dim3(size);
  int most = 0;
  if (prepare_kernel(kernel, LinSmem<32>::kAlloc, 0, done) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&most, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  n.store(most + 1);
  return most;
}

cudaError_t launch_linear_forward(const LinMaps& m, const LinArgs& a, const LinPlan& p, cudaStream_t s) {
  return launch_lin_all<kLinForward>(m, a, p, s);
}
}  // namespace dera
