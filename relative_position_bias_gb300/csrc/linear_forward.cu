#include "linear_inst.cuh"

namespace dera {
cudaError_t launch_linear_forward(const LinMaps& m, const LinArgs& a, const LinPlan& p, cudaStream_t s) {
  return launch_lin_all<kLinForward>(m, a, p, s);
}
}  // namespace dera
