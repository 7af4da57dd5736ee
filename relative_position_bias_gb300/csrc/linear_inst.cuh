// Launch of the kernels in linear.cuh for one kind of product.
#pragma once
#include "launch.cuh"
#include "linear.cuh"
#include "linear_pair.cuh"

namespace dera {

template <int KIND, int BN, bool TURNED, bool BF16>
static cudaError_t launch_lin(const LinMaps& m, const LinArgs& a, cudaStream_t s) {
  auto kernel = linear_kernel<KIND, BN, TURNED, BF16>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = prepare_kernel(kernel, LinSmem<BN>::kAlloc, 0, done);
  if (e != cudaSuccess) return e;
  kernel<<<a.batches * a.m_tiles * a.n_tiles, kLinThreads, LinSmem<BN>::kAlloc, s>>>(m.a, m.b, a);
  return cudaGetLastError();
}

template <int KIND, int BN, bool BF16>
static cudaError_t launch_lin_pair(const LinMaps& m, const LinArgs& a, int pairs, cudaStream_t s) {
  auto kernel = linear_pair_kernel<KIND, BN, BF16>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = prepare_kernel(kernel, PairSmem<KIND, BN>::kAlloc, 0, done);
  if (e != cudaSuccess) return e;
  kernel<<<2 * pairs, pair_threads(KIND), PairSmem<KIND, BN>::kAlloc, s>>>(m.a, m.b, a);
  return cudaGetLastError();
}

// Tokens by features: the gradient of the weight has only pairs.
template <int KIND, bool BF16>
static cudaError_t launch_lin_kind(const LinMaps& m, const LinArgs& a, const LinPlan& p, cudaStream_t s) {
  if (p.pairs > 0)
    return p.bn == 256 ? launch_lin_pair<KIND, 256, BF16>(m, a, p.pairs, s) : launch_lin_pair<KIND, 128, BF16>(m, a, p.pairs, s);
  if constexpr (KIND != kLinWeight) {
    if (!p.turned) return launch_lin<KIND, 128, false, BF16>(m, a, s);
    if (p.bn == 32) return launch_lin<KIND, 32, true, BF16>(m, a, s);
    return p.bn == 64 ? launch_lin<KIND, 64, true, BF16>(m, a, s) : launch_lin<KIND, 128, true, BF16>(m, a, s);
  }
  return cudaErrorInvalidValue;
}

template <int KIND>
static cudaError_t launch_lin_all(const LinMaps& m, const LinArgs& a, const LinPlan& p, cudaStream_t s) {
  return a.fmt == kBF16 ? launch_lin_kind<KIND, true>(m, a, p, s) : launch_lin_kind<KIND, false>(m, a, p, s);
}

}  // namespace dera
