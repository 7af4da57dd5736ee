#include "linear_inst.cuh"

namespace dera {

// Partial sums of a matrix's columns: block i adds every gridDim.x-th run of 32 rows.  A warp reads 32 chunks of
// eight columns of one row at a time.
__global__ void __launch_bounds__(256) column_sums_kernel(const void* g, long long rows, int cols, int fmt, float* parts) {
  grid_launch_dependents();
  const int c = (blockIdx.y * 32 + (threadIdx.x & 31)) * 8, w = threadIdx.x >> 5;
  __shared__ float red[8][256];
  float s[8] = {};
  if (c < cols) {
    #pragma unroll 4
    for (long long r = static_cast<long long>(blockIdx.x) * 8 + w; r < rows; r += static_cast<long long>(gridDim.x) * 8) {
      float v[8];
      load8(g, static_cast<size_t>(r) * cols + c, v, fmt);
      #pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += v[e];
    }
  }
  #pragma unroll
  for (int e = 0; e < 8; ++e) red[w][(threadIdx.x & 31) * 8 + e] = s[e];
  __syncthreads();
  const int col = blockIdx.y * 256 + threadIdx.x;
  if (col >= cols) return;
  float v = 0.f;
  #pragma unroll
  for (int i = 0; i < 8; ++i) v += red[i][threadIdx.x];
  parts[static_cast<size_t>(blockIdx.x) * cols + col] = v;
}

cudaError_t launch_linear_weight(const LinMaps& m, const LinArgs& a, const LinPlan& p, cudaStream_t s) {
  return launch_lin_all<kLinWeight>(m, a, p, s);
}

// The pieces of a split contraction, added in order.
__global__ void __launch_bounds__(256) sum_pieces_kernel(const float* parts, int pieces, long long n, void* out, int out_fmt) {
  grid_wait_prerequisites();   // every piece is written
  const long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  float v[8], x[8];
  load8(parts, i, v, kF32);
  #pragma unroll 4
  for (int p = 1; p < pieces; ++p) {
    load8(parts, static_cast<size_t>(p) * n + i, x, kF32);
    #pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += x[e];
  }
  store8(out, i, v, out_fmt);
}

cudaError_t launch_sum_pieces(const float* parts, int pieces, long long n, void* out, int out_fmt, cudaStream_t s) {
  return launch_early(sum_pieces_kernel, dim3(static_cast<unsigned>((n + 2047) / 2048)), dim3(256), 0, s, parts, pieces, n,
                      out, out_fmt);
}

cudaError_t launch_column_sums(const void* g, long long rows, int cols, int fmt, float* parts, int blocks, cudaStream_t s) {
  column_sums_kernel<<<dim3(blocks, (cols + 255) / 256), 256, 0, s>>>(g, rows, cols, fmt, parts);
  return cudaGetLastError();
}
}  // namespace dera
