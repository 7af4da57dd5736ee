// Launch of the kernels in linear.cuh for one kind of product.
#pragma once
#include "launch.cuh"
#include "linear.cuh"
#include "linear_pair.cuh"

namespace dera {

static void cluster_launch(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int size, int smem) {
  *attr = {};
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = size;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  *cfg = {};
  cfg->blockDim = dim3(kLinThreads);
  cfg->dynamicSmemBytes = smem;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}

template <int KIND, int BN, bool BF16>
static cudaError_t launch_lin_few(const LinMaps& m, const LinArgs& a, cudaStream_t s) {
  auto kernel = linear_few_kernel<KIND, BN, BF16>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = prepare_kernel(kernel, LinSmem<BN>::kAlloc, 0, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg;
  cluster_launch(&cfg, &attr, a.pieces, LinSmem<BN>::kAlloc);
  cfg.gridDim = dim3(a.m_tiles * a.pieces, a.n_tiles);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kernel, m.a, m.b, a);
}

template <int KIND, int BN, int EPI, bool FINE, bool BF16>
static cudaError_t launch_lin_pair(const LinMaps& m, const LinArgs& a, int pairs, bool beside, cudaStream_t s) {
  auto kernel = linear_pair_kernel<KIND, BN, EPI, FINE, BF16>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = prepare_kernel(kernel, PairSmem<KIND, BN, EPI>::kAlloc, 0, done);
  if (e != cudaSuccess) return e;
  if (beside) return launch_early(kernel, dim3(2 * pairs), dim3(pair_threads(EPI)), PairSmem<KIND, BN, EPI>::kAlloc, s, m, a);
  kernel<<<2 * pairs, pair_threads(EPI), PairSmem<KIND, BN, EPI>::kAlloc, s>>>(m, a);
  return cudaGetLastError();
}

// Tokens by features: the gradient of the weight has only pairs.
template <int KIND, bool BF16>
static cudaError_t launch_lin_kind(const LinMaps& m, const LinArgs& a, const LinPlan& p, cudaStream_t s) {
  if constexpr (KIND != kLinWeight) {
    if (p.turned) {
      if (p.bn == 32) return launch_lin_few<KIND, 32, BF16>(m, a, s);
      if (p.bn == 64) return launch_lin_few<KIND, 64, BF16>(m, a, s);
      return p.bn == 128 ? launch_lin_few<KIND, 128, BF16>(m, a, s) : launch_lin_few<KIND, 256, BF16>(m, a, s);
    }
    if (p.fine)
      return p.bn == 128 ? launch_lin_pair<KIND, 128, 8, true, BF16>(m, a, p.pairs, p.beside, s)
                         : launch_lin_pair<KIND, 256, 8, true, BF16>(m, a, p.pairs, p.beside, s);
    if (p.bn == 128) return launch_lin_pair<KIND, 128, 8, false, BF16>(m, a, p.pairs, p.beside, s);
  }
  if constexpr (KIND != kLinWeight)
    if (p.epi == 16) return launch_lin_pair<KIND, 256, 16, false, BF16>(m, a, p.pairs, p.beside, s);
  return launch_lin_pair<KIND, 256, 8, false, BF16>(m, a, p.pairs, p.beside, s);
}

template <int KIND>
static cudaError_t launch_lin_all(const LinMaps& m, const LinArgs& a, const LinPlan& p, cudaStream_t s) {
  return a.fmt == kBF16 ? launch_lin_kind<KIND, true>(m, a, p, s) : launch_lin_kind<KIND, false>(m, a, p, s);
}

}  // namespace dera
