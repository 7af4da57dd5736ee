// Launchers of the kernels in layer_norm.cuh, and the activations' backward.
#include "layer_norm.cuh"

#include <algorithm>

#include "activation.cuh"
#include "launch.cuh"

namespace dera {

namespace {

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

constexpr int kRingMost = 216 * 1024;   // dynamic shared memory of a block

// Bytes of the ring of a launch, and how many sets it holds: an SM's shared memory over its blocks.
int ring_bytes(LnArgs& a, const LnPlan& p, int row_bytes, bool vec) {
  if (!vec) return 0;
  const int set = p.threads / p.tpr * row_bytes;
  a.sets = std::max(1, std::min(8, (kRingMost / p.blocks - 2048) / set));
  return kLnRingHead + a.sets * set;
}
int size_of(int fmt) { return fmt == kF32 ? 4 : 2; }

template <class Kernel>
cudaError_t launch(Kernel kernel, const LnArgs& a, const LnPlan& p, int smem, std::atomic<unsigned long long>& done, cudaStream_t s) {
  const cudaError_t e = prepare_kernel(kernel, kRingMost, 0, done);
  if (e != cudaSuccess) return e;
  kernel<<<p.grid, p.threads, smem, s>>>(a);
  return cudaGetLastError();
}

template <int XF, int MAXT, int NV, bool VEC>
cudaError_t fwd(const LnArgs& a, const LnPlan& p, int smem, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  return launch(layer_norm_kernel<XF, MAXT, NV, VEC>, a, p, smem, done, s);
}
template <int XF, int ZF, int MAXT, int NV, bool VEC, int BLOCKS>
cudaError_t bwd(const LnArgs& a, const LnPlan& p, int smem, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  return launch(layer_norm_bwd_kernel<XF, ZF, MAXT, NV, VEC, BLOCKS>, a, p, smem, done, s);
}

template <int XF, int NV>
cudaError_t fwd_warp(LnArgs& a, int sms, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const int row = a.C * size_of(XF), params = a.w ? (a.b ? 8 : 4) * a.C : 0;
  a.sets = std::max(1, std::min(8, (kRingMost / ln_warp_blocks(NV) - 2048 - 640 - params) / 8 / row));
  LnPlan p;
  p.threads = 256;
  p.grid = static_cast<int>(std::min(ceil_div(a.rows, 8), static_cast<long long>(ln_warp_blocks(NV)) * std::max(sms, 1)));
  return launch(layer_norm_warp_kernel<XF, NV>, a, p, 640 + params + 8 * a.sets * row, done, s);
}

template <int XF, bool VEC>
cudaError_t fwd_of(LnArgs& a, const LnPlan& p, int sms, cudaStream_t s) {
  if constexpr (VEC) {   // whatever the number of rows: a row's bits do not depend on it
    if (a.C <= 256) return fwd_warp<XF, 1>(a, sms, s);
    if (a.C <= 512) return fwd_warp<XF, 2>(a, sms, s);
    if (a.C <= 768) return fwd_warp<XF, 3>(a, sms, s);
    if (a.C <= 1024) return fwd_warp<XF, 4>(a, sms, s);
    if (a.C <= 2048) return fwd_warp<XF, 8>(a, sms, s);
  }
  const int smem = ring_bytes(a, p, a.C * size_of(a.x_fmt), VEC);
  if (a.C > 8192) return fwd<XF, 1024, 2, VEC>(a, p, smem, s);
  if constexpr (VEC) return fwd<XF, 512, 2, VEC>(a, p, smem, s);
  else return a.C > 2048 ? fwd<XF, 1024, 1, VEC>(a, p, smem, s) : fwd<XF, 256, 1, VEC>(a, p, smem, s);
}

template <int XF, int ZF, bool VEC>
cudaError_t bwd_of(LnArgs& a, const LnPlan& p, cudaStream_t s) {
  const int G = p.threads / p.tpr;
  int smem = ring_bytes(a, p, a.C * (size_of(a.x_fmt) + size_of(a.y_fmt) + (a.dres ? size_of(a.dx_fmt) : 0)), VEC);
  if (a.parts && G > 1) smem = std::max(smem, kLnRingHead + 2 * G * a.C * 4);   // the sums
  if (a.C > 8192) return bwd<XF, ZF, 1024, 2, VEC, 1>(a, p, smem, s);
  if constexpr (VEC) {
    if (a.C > 4096) return bwd<XF, ZF, 512, 2, VEC, 1>(a, p, smem, s);
    if (a.C > 512) return bwd<XF, ZF, 256, 2, VEC, 2>(a, p, smem, s);
  } else if (a.C > 2048) {
    return bwd<XF, ZF, 1024, 1, VEC, 1>(a, p, smem, s);
  }
  return bwd<XF, ZF, 256, 1, VEC, 3>(a, p, smem, s);
}

}  // namespace

LnPlan ln_plan(long long rows, int C, bool backward, bool vec, int sms) {
  LnPlan p;
  // eight elements a thread twice over: half of the shuffles and addresses an element, where the registers allow it (32768 x
  // 1024, bf16, backward: 55 us instead of 58; rows read element by element 291 instead of 136, 108 since)
  const int nv = C > (!vec ? 8192 : (backward ? 512 : 2048)) ? 2 : 1;
  p.tpr = static_cast<int>(ceil_div(ceil_div(C, 8 * nv), 32)) * 32;
  const int G = std::max(1, 256 / p.tpr);
  p.threads = G * p.tpr;
  // blocks: a row set each until the SMs are full of threads
  p.blocks = std::max(1, (backward ? (nv == 2 ? 512 : 768) : 1024) / p.threads);
  p.grid = static_cast<int>(std::min(ceil_div(rows, G), static_cast<long long>(std::max(sms, 1)) * p.blocks));
  return p;
}

template <int XF>
static cudaError_t fwd_any(LnArgs& a, const LnPlan& p, bool vec, int sms, cudaStream_t s) {
  return vec ? fwd_of<XF, true>(a, p, sms, s) : fwd_of<XF, false>(a, p, sms, s);
}
template <int XF, int ZF>
static cudaError_t bwd_any(LnArgs& a, const LnPlan& p, bool vec, cudaStream_t s) {
  return vec ? bwd_of<XF, ZF, true>(a, p, s) : bwd_of<XF, ZF, false>(a, p, s);
}

cudaError_t launch_ln(LnArgs& a, const LnPlan& p, bool vec, int sms, cudaStream_t s) {
  a.tpr = p.tpr;
  if (a.x_fmt == kF32) return fwd_any<kF32>(a, p, vec, sms, s);
  return a.x_fmt == kBF16 ? fwd_any<kBF16>(a, p, vec, sms, s) : fwd_any<kF16>(a, p, vec, sms, s);
}

cudaError_t launch_ln_backward(LnArgs& a, const LnPlan& p, bool vec, float* dw, float* db, cudaStream_t s) {
  a.tpr = p.tpr;
  cudaError_t e;
  if (a.x_fmt == kF32)
    e = a.y_fmt == kF32 ? bwd_any<kF32, kF32>(a, p, vec, s) : (a.y_fmt == kBF16 ? bwd_any<kF32, kBF16>(a, p, vec, s)
                                                                            : bwd_any<kF32, kF16>(a, p, vec, s));
  else if (a.x_fmt == kBF16)
    e = a.y_fmt == kF32 ? bwd_any<kBF16, kF32>(a, p, vec, s) : bwd_any<kBF16, kBF16>(a, p, vec, s);
  else
    e = a.y_fmt == kF32 ? bwd_any<kF16, kF32>(a, p, vec, s) : bwd_any<kF16, kF16>(a, p, vec, s);
  if (e != cudaSuccess || !a.parts) return e;
  return launch_partial_rows(a.parts, p.grid, 2 * a.C, a.C, dw, db, s);
}

cudaError_t launch_partial_rows(const float* parts, int rows, int n, int n1, float* d1, float* d2, cudaStream_t s) {
  return launch_early(partial_rows_kernel, dim3((n + 31) / 32), dim3(32, 32), 0, s, parts, rows, n, n1, d1, d2);
}

// dpre = dy act'(pre): bound by memory; eight elements a thread, what is left at the end one each.  8 x 4096 x 2048, fp16 to fp32,
// 537 MB: 88 us, 6.1 TB/s.
template <int ACT>
__global__ void __launch_bounds__(256) act_backward_kernel(const ActArgs a) {
  const long long n8 = a.n & ~7ll, step = static_cast<long long>(gridDim.x) * 2048;
  for (long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * 8; i < n8; i += step) {
    float u[8], z[8];
    load8(a.pre, i, u, a.fmt);
    load8(a.dy, i, z, a.z_fmt);
    slope_all<ACT>(z, u);
    store8(a.dpre, i, z, a.out_fmt);
  }
  const long long i = n8 + threadIdx.x;
  if (blockIdx.x == 0 && i < a.n) {
    const float z = load_elem(a.dy, i, a.z_fmt) * act_slope<ACT>(pair_of(load_elem(a.pre, i, a.fmt))).x;
    if (a.out_fmt == kF32) static_cast<float*>(a.dpre)[i] = z;
    else static_cast<uint16_t*>(a.dpre)[i] = static_cast<uint16_t>(pack_in(z, 0.f, a.out_fmt));
  }
}

template <int ACT>
static cudaError_t act_backward(const ActArgs& a, int sms, cudaStream_t s) {
  const long long blocks = std::min(ceil_div(a.n, 2048), static_cast<long long>(std::max(sms, 1)) * 64);
  act_backward_kernel<ACT><<<static_cast<int>(blocks), 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_act_backward(const ActArgs& a, int sms, cudaStream_t s) {
  switch (a.act) {
    case kActRelu: return act_backward<kActRelu>(a, sms, s);
    case kActGelu: return act_backward<kActGelu>(a, sms, s);
    case kActGeluTanh: return act_backward<kActGeluTanh>(a, sms, s);
    case kActQuickGelu: return act_backward<kActQuickGelu>(a, sms, s);
    default: return act_backward<kActSilu>(a, sms, s);
  }
}

}  // namespace dera
