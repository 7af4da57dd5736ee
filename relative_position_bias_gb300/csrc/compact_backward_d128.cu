#include "compact_backward_inst.cuh"

namespace dera {

cudaError_t launch_cb_d128(const CbMaps& m, const CbArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? launch_cb<true, 128>(m, a, s) : launch_cb<false, 128>(m, a, s);
}

}  // namespace dera
