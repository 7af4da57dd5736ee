// Launchers of the kernels in qk_norm_rope.cuh.
#include "qk_norm_rope.cuh"

#include <algorithm>

namespace dera {

namespace {

template <bool BF16, int D, bool NORM>
cudaError_t fwd(const QkArgs& a, int mode, dim3 grid, cudaStream_t s) {
  switch (mode) {
    case kRotNone: qk_norm_rope_kernel<BF16, D, kRotNone, NORM><<<grid, kQkThreads, 0, s>>>(a); break;
    case kRotHalf: qk_norm_rope_kernel<BF16, D, kRotHalf, NORM><<<grid, kQkThreads, 0, s>>>(a); break;
    default: qk_norm_rope_kernel<BF16, D, kRotPairs, NORM><<<grid, kQkThreads, 0, s>>>(a); break;
  }
  return cudaGetLastError();
}

template <bool BF16, int D, bool NORM, bool ZF32>
cudaError_t bwd(const QkArgs& a, int mode, dim3 grid, cudaStream_t s) {
  switch (mode) {
    case kRotNone: qk_norm_rope_bwd_kernel<BF16, D, kRotNone, NORM, ZF32><<<grid, kQkThreads, 0, s>>>(a); break;
    case kRotHalf: qk_norm_rope_bwd_kernel<BF16, D, kRotHalf, NORM, ZF32><<<grid, kQkThreads, 0, s>>>(a); break;
    default: qk_norm_rope_bwd_kernel<BF16, D, kRotPairs, NORM, ZF32><<<grid, kQkThreads, 0, s>>>(a); break;
  }
  return cudaGetLastError();
}

template <bool BF16, int D>
cudaError_t pick(const QkArgs& a, int mode, bool norm, bool backward, dim3 grid, cudaStream_t s) {
  if (!backward) return norm ? fwd<BF16, D, true>(a, mode, grid, s) : fwd<BF16, D, false>(a, mode, grid, s);
  if (a.z_fmt == kF32) return norm ? bwd<BF16, D, true, true>(a, mode, grid, s) : bwd<BF16, D, false, true>(a, mode, grid, s);
  return norm ? bwd<BF16, D, true, false>(a, mode, grid, s) : bwd<BF16, D, false, false>(a, mode, grid, s);
}

int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

}  // namespace

QkPlan qk_plan(long long tokens, const int (&heads)[3], int head_dim, bool backward, int sms) {
  QkPlan p;
  const int blocks = ceil_div(tokens, kQkThreads / (head_dim / 8));   // runs of tokens
  const int total = heads[0] + heads[1] + heads[2];
  // Heads per block: as many as leave eight blocks for every SM, at least one and, where it is more
  // than three, whole batches of the four rows that a thread loads at once.  Each block loads its
  // tokens' angles once, so more heads mean fewer of those loads.
  const long long want = 8ll * std::max(sms, 1);
  const long long most = std::max<long long>(1, static_cast<long long>(blocks) * total / want);
  p.per = static_cast<int>(most >= 16 ? 16 : (most >= 4 ? most / 4 * 4 : most));
  for (int i = 0; i < 3; ++i) p.groups[i] = ceil_div(heads[i], p.per);
  const int gy = p.groups[0] + p.groups[1] + p.groups[2];
  // backward: about `want` blocks, so that the partial weight gradients stay small, each with the same
  // number of runs
  p.grid_x = blocks;
  if (backward) p.grid_x = ceil_div(blocks, std::max<long long>(1, static_cast<long long>(blocks) * gy / want));
  p.part_rows_q = p.groups[0] * p.grid_x;
  p.part_rows_k = p.groups[1] * p.grid_x;
  return p;
}

cudaError_t launch_qk(QkArgs& a, const QkPlan& p, int head_dim, int mode, bool bf16, bool norm, bool backward,
                      float* dqw, float* dkw, cudaStream_t s) {
  a.per = p.per;
  for (int i = 0; i < 3; ++i) a.groups[i] = p.groups[i];
  const dim3 grid(p.grid_x, p.groups[0] + p.groups[1] + p.groups[2]);
  cudaError_t e;
  if (head_dim == 128)
    e = bf16 ? pick<true, 128>(a, mode, norm, backward, grid, s) : pick<false, 128>(a, mode, norm, backward, grid, s);
  else
    e = bf16 ? pick<true, 64>(a, mode, norm, backward, grid, s) : pick<false, 64>(a, mode, norm, backward, grid, s);
  if (e != cudaSuccess || !backward || !norm) return e;
  return launch_early(qk_weight_grad_kernel, dim3(head_dim / 32, 2), dim3(32, 32), 0, s,
                      static_cast<const float*>(a.parts), p.part_rows_q, p.part_rows_k, head_dim, dqw, dkw);
}

}  // namespace dera
