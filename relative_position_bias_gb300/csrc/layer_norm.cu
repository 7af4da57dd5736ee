// Launchers of the kernels in layer_norm.cuh, and the activations' backward.
#include "layer_norm.cuh"

#include <algorithm>

#include "activation.cuh"

namespace dera {

namespace {

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

template <int XF, bool VEC>
cudaError_t fwd(const LnArgs& a, const LnPlan& p, cudaStream_t s) {
  if (a.C > 8192) layer_norm_kernel<XF, 1024, 2, VEC, 1><<<p.grid, p.threads, 0, s>>>(a);
  else if (a.C > 2048) layer_norm_kernel<XF, 1024, 1, VEC, 2><<<p.grid, p.threads, 0, s>>>(a);
  else layer_norm_kernel<XF, 256, 1, VEC, 4><<<p.grid, p.threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <int XF, int ZF, bool VEC>
cudaError_t bwd(const LnArgs& a, const LnPlan& p, cudaStream_t s) {
  const int G = p.threads / p.tpr;
  const size_t smem = a.parts && G > 1 ? static_cast<size_t>(2) * G * 8 * p.tpr * sizeof(float) : 0;   // 16 KB
  if (a.C > 8192) layer_norm_bwd_kernel<XF, ZF, 1024, 2, VEC, 1><<<p.grid, p.threads, smem, s>>>(a);
  else if (a.C > 2048) layer_norm_bwd_kernel<XF, ZF, 1024, 1, VEC, 1><<<p.grid, p.threads, smem, s>>>(a);
  else layer_norm_bwd_kernel<XF, ZF, 256, 1, VEC, 2><<<p.grid, p.threads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

LnPlan ln_plan(long long rows, int C, bool backward, int sms) {
  LnPlan p;
  const int nv = C > 8192 ? 2 : 1;
  p.tpr = static_cast<int>(ceil_div(ceil_div(C, 8 * nv), 32)) * 32;
  const int G = std::max(1, 256 / p.tpr);
  p.threads = G * p.tpr;
  // blocks: a row set each until the SMs are full of threads
  const long long most = static_cast<long long>(std::max(sms, 1)) * std::max(1, (backward ? 1024 : 2048) / p.threads);
  p.grid = static_cast<int>(std::min(ceil_div(rows, G), most));
  return p;
}

cudaError_t launch_ln(LnArgs& a, const LnPlan& p, bool vec, cudaStream_t s) {
  a.tpr = p.tpr;
  if (!vec) return fwd<-1, false>(a, p, s);
  if (a.x_fmt == kF32) return fwd<kF32, true>(a, p, s);
  return a.x_fmt == kBF16 ? fwd<kBF16, true>(a, p, s) : fwd<kF16, true>(a, p, s);
}

cudaError_t launch_ln_backward(LnArgs& a, const LnPlan& p, bool vec, float* dw, float* db, cudaStream_t s) {
  a.tpr = p.tpr;
  cudaError_t e;
  if (!vec) e = bwd<-1, -1, false>(a, p, s);
  else if (a.x_fmt == kF32)
    e = a.y_fmt == kF32 ? bwd<kF32, kF32, true>(a, p, s) : (a.y_fmt == kBF16 ? bwd<kF32, kBF16, true>(a, p, s)
                                                                           : bwd<kF32, kF16, true>(a, p, s));
  else if (a.x_fmt == kBF16)
    e = a.y_fmt == kF32 ? bwd<kBF16, kF32, true>(a, p, s) : bwd<kBF16, kBF16, true>(a, p, s);
  else
    e = a.y_fmt == kF32 ? bwd<kF16, kF32, true>(a, p, s) : bwd<kF16, kF16, true>(a, p, s);
  if (e != cudaSuccess || !a.parts) return e;
  return launch_partial_rows(a.parts, p.grid, 2 * a.C, a.C, dw, db, s);
}

cudaError_t launch_partial_rows(const float* parts, int rows, int n, int n1, float* d1, float* d2, cudaStream_t s) {
  return launch_early(partial_rows_kernel, dim3((n + 31) / 32), dim3(32, 32), 0, s, parts, rows, n, n1, d1, d2);
}

// dpre = dy act'(pre): bound by memory; eight elements a thread where n and the addresses allow.
template <int ACT, bool VEC>
__global__ void __launch_bounds__(256) act_backward_kernel(const ActArgs a) {
  constexpr int E = VEC ? 8 : 1;
  const long long step = static_cast<long long>(gridDim.x) * 256 * E;
  for (long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * E; i < a.n; i += step) {
    if (VEC) {
      float u[8], z[8];
      load8(a.pre, i, u, a.fmt);
      load8(a.dy, i, z, a.z_fmt);
      slope_all<ACT>(z, u);
      store8(a.dpre, i, z, a.out_fmt);
    } else {
      const float z = load_elem(a.dy, i, a.z_fmt) * act_slope<ACT>(pair_of(load_elem(a.pre, i, a.fmt))).x;
      if (a.out_fmt == kF32) static_cast<float*>(a.dpre)[i] = z;
      else static_cast<uint16_t*>(a.dpre)[i] = static_cast<uint16_t>(pack_in(z, 0.f, a.out_fmt));
    }
  }
}

template <int ACT>
static cudaError_t act_backward(const ActArgs& a, int sms, cudaStream_t s) {
  const bool vec = a.n % 8 == 0;
  const long long blocks = std::min(ceil_div(a.n, vec ? 2048 : 256), static_cast<long long>(std::max(sms, 1)) * 16);
  if (vec) act_backward_kernel<ACT, true><<<static_cast<int>(blocks), 256, 0, s>>>(a);
  else act_backward_kernel<ACT, false><<<static_cast<int>(blocks), 256, 0, s>>>(a);
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
