// Launch of the compact-bias backward for one head dimension; included by one .cu for each, so that
// the build compiles them side by side.
#pragma once
#include "compact_backward.cuh"
#include "launch.cuh"

namespace dera {

template <int WP, bool BF16, int D>
static cudaError_t launch_cb_rows(const CbMaps& m, const CbArgs& a, unsigned grid, cudaStream_t s) {
  auto kernel = relpos_cb_rows_kernel<WP, BF16, D>;
  using SM = CbRowsSmem<WP, D>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = prepare_kernel(kernel, SM::kAlloc, 0, done);
  if (e != cudaSuccess) return e;
  kernel<<<grid, CbRowsDims<D>::kThreads, SM::kAlloc, s>>>(m.kg, m.vg, a);
  return cudaGetLastError();
}

template <bool BF16, int D>
static cudaError_t launch_cb_cols(const CbMaps& m, const CbArgs& a, unsigned grid, cudaStream_t s) {
  auto kernel = relpos_cb_cols_kernel<BF16, D>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = prepare_kernel(kernel, CbColsSmem<D>::kAlloc, kCbColsLaunchRegs, done);
  if (e != cudaSuccess) return e;
  return launch_early(kernel, dim3(grid), dim3(kCbColsThreads), CbColsSmem<D>::kAlloc, s, m.q64, m.dout64, m.k, m.v, a);
}

template <bool BF16, int D>
static cudaError_t launch_cb(const CbMaps& m, const CbArgs& a, cudaStream_t s) {
  const int units = a.BH * a.n_tiles;
  const CbSplit rs = {a.rows_full, a.rows_split}, cs = {a.cols_full, a.cols_split};
  // heads in y: at most 65535 a launch
  cudaError_t e = cudaSuccess;
  for (int b0 = 0; b0 < a.BH && e == cudaSuccess; b0 += 65535) {
    CbArgs p = a;
    const int nb = a.BH - b0 < 65535 ? a.BH - b0 : 65535;
    const size_t rows = static_cast<size_t>(b0) * a.N, blocks = static_cast<size_t>(b0) * a.n_blocks;
    const size_t bias = a.bias_fmt == kF32 ? 4 : 2, out = a.out_fmt == kF32 ? 4 : 2;
    p.rel_h = static_cast<const char*>(a.rel_h) + rows * a.H * bias;
    p.rel_w = static_cast<const char*>(a.rel_w) + rows * a.W * bias;
    p.lse = a.lse + rows;
    p.out = static_cast<const char*>(a.out) + rows * D * out;
    p.dout = static_cast<const char*>(a.dout) + rows * D * 2;
    p.hl = a.hl + blocks * a.H * kCbRow;
    p.rw = a.rw + blocks * a.W * kCbRow;
    p.nD = a.nD + blocks * 64;
    relpos_cb_prep_kernel<BF16, D><<<dim3(a.n_tiles, nb), kCbPrepThreads, 0, s>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  const unsigned rgrid = static_cast<unsigned>(rs.blocks(units)), cgrid = static_cast<unsigned>(cs.blocks(units));
  switch (cb_width(a.W)) {
    case 16: e = launch_cb_rows<16, BF16, D>(m, a, rgrid, s); break;
    case 32: e = launch_cb_rows<32, BF16, D>(m, a, rgrid, s); break;
    case 48: e = launch_cb_rows<48, BF16, D>(m, a, rgrid, s); break;
    default: e = launch_cb_rows<64, BF16, D>(m, a, rgrid, s); break;
  }
  if (e != cudaSuccess) return e;
  e = launch_cb_cols<BF16, D>(m, a, cgrid, s);
  const int joins = rs.tail(units) + cs.tail(units);
  if (e != cudaSuccess || joins == 0) return e;
  relpos_cb_join_kernel<D><<<dim3(joins, D / 4), kCbJoinThreads, 0, s>>>(a, rs.tail(units));
  return cudaGetLastError();
}

}  // namespace dera
