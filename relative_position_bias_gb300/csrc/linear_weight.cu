#include "linear_inst.cuh"

namespace dera {

// Partial sums of a matrix's columns: block i adds every gridDim.x-th run of 8 rows, a warp each, 32 chunks of eight columns at a time.
// Bound by memory: 32768 x 1024 bf16, 67 MB, 9.3 us with the join.
__global__ void __launch_bounds__(256) column_sums_kernel(const void* g, long long rows, int cols, int fmt, float* parts) {
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
  grid_wait_prerequisites();   // as in linear_pair.cuh
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

// Blocks of 256 threads: the first `dw_blocks` add the pieces of eight neighbouring elements a thread, in order; the others the partial
// rows of 32 columns of dy's sums, eight runs of rows a block, in a fixed order.
__global__ void __launch_bounds__(256) linear_join_kernel(const LinJoin j, int dw_blocks) {
  __shared__ float red[8][33];
  grid_wait_prerequisites();   // every piece and every partial row is written
  if (static_cast<int>(blockIdx.x) < dw_blocks) {
    const long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * 8;
    if (i >= j.n) return;
    float v[8], x[8];
    load8(j.parts, i, v, kF32);
    #pragma unroll 4
    for (int p = 1; p < j.pieces; ++p) {
      load8(j.parts, static_cast<size_t>(p) * j.n + i, x, kF32);
      #pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += x[e];
    }
    store8(j.dw, i, v, j.dw_fmt);
    return;
  }
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, c = (blockIdx.x - dw_blocks) * 32 + lane;
  float v = 0.f;
  if (c < j.out) {
    #pragma unroll 8
    for (int r = run; r < j.sum_rows; r += 8) v += j.sums[static_cast<size_t>(r) * j.out + c];
  }
  red[run][lane] = v;
  __syncthreads();
  if (run == 0 && c < j.out) {
    float s = 0.f;
    #pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][lane];
    j.db[c] = s;
  }
}

cudaError_t launch_linear_join(const LinJoin& j, cudaStream_t s) {
  const long long dw_blocks = j.dw ? (j.n + 2047) / 2048 : 0;
  const int db_blocks = j.db ? (j.out + 31) / 32 : 0;
  return launch_early(linear_join_kernel, dim3(static_cast<unsigned>(dw_blocks + db_blocks)), dim3(256), 0, s, j,
                      static_cast<int>(dw_blocks));
}

cudaError_t launch_column_sums(const void* g, long long rows, int cols, int fmt, float* parts, int blocks, bool beside, cudaStream_t s) {
  const dim3 grid(blocks, (cols + 255) / 256);
  if (beside) return launch_early(column_sums_kernel, grid, dim3(256), 0, s, g, rows, cols, fmt, parts);
  column_sums_kernel<<<grid, 256, 0, s>>>(g, rows, cols, fmt, parts);
  return cudaGetLastError();
}
}  // namespace dera
