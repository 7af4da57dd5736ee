// Launch arguments and launchers behind the entry points of dera_train.h.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>

#include "split.h"

namespace dera {

// A launch whose blocks may start before the kernel ahead of it in the stream is complete; it has to wait for
// that one itself (grid_wait_prerequisites).
template <class Kernel, class... Args>
cudaError_t launch_early(Kernel kernel, dim3 grid, dim3 threads, size_t smem, cudaStream_t s, const Args&... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int kQkThreads = 256;

struct HeadsPtr {
  char* data;
  long long sb, st, sh;   // strides in elements
};

struct QkArgs {
  HeadsPtr x[3];        // q, k, v in token order (forward: read; backward: q, k read)
  HeadsPtr dx[3];       // backward: dq, dk, dv in token order
  const void* z[3];     // backward: dq_out, dk_out, dv_out
  void* zo[3];          // forward: q_out, k_out, v_out
  const void* w[2];     // q_weight, k_weight
  const float* cos;
  const float* sin;
  const int* positions;
  float* parts;         // backward: [2][part_rows][D] partial weight gradients
  int heads[3];         // q, k, v heads (v: 0 if absent)
  int groups[3];        // blocks in y for each, each of `per` heads
  int per;
  int N, table_rows, half;   // half = rotary_dim / 2
  long long tokens;     // B * N
  float eps;
  int w_fmt, z_fmt, dx_fmt;
};

// Rotation: none, pairs (i, i + half), pairs (2i, 2i + 1).
enum : int { kRotNone = 0, kRotHalf = 1, kRotPairs = 2 };

// How qk_norm_rope's grid is cut for a size.
struct QkPlan {
  int per;             // heads per block
  int groups[3];       // blocks in y of q, k, v
  int grid_x;          // blocks over tokens
  int part_rows_q, part_rows_k;   // backward: partial rows of the weight gradients
};
QkPlan qk_plan(long long tokens, const int (&heads)[3], int head_dim, bool backward, int sms);
cudaError_t launch_qk(QkArgs& a, const QkPlan& p, int head_dim, int mode, bool bf16, bool norm, bool backward,
                      float* dqw, float* dkw, cudaStream_t s);

// Compact-bias backward (compact_backward.cuh).
// hl and rw are kept by blocks of 64 queries, a row of 64 floats for each grid row (column), so that
// what a step needs is one run of whole 256-byte rows.  The 16-byte chunks of row i are permuted by
// i % 8: threads that read the same queries of neighbouring rows then hit different banks.
constexpr int kCbRow = 64;
__host__ __device__ constexpr int cb_at(int row, int query) {
  return row * kCbRow + ((((query >> 2) ^ (row & 7))) << 2) + (query & 3);
}

struct CbArgs {
  const void* q;        // [BH, N, D]
  const void* k;
  const void* v;
  const void* rel_h;    // [BH, N, H] bias dtype
  const void* rel_w;    // [BH, N, W]
  const float* lse;     // [BH, N] base 2
  const void* out;      // [BH, N, D]
  const void* dout;     // [BH, N, D]
  float* hl;            // [BH][n_blocks][H][kCbRow] log2(e) rel_h - lse of 64 queries (-inf: P = 0)
  float* rw;            // [BH][n_blocks][W][kCbRow] log2(e) rel_w
  float* nD;            // [BH][64 n_blocks] -D
  void* dq;
  void* dk;
  void* dv;
  float* drel_h;
  float* drel_w;
  float* parts_rows;    // [piece][128 (D + W)] of the split units
  float* parts_cols;    // [piece][128 (2 D)]
  int* status;
  int BH, H, W, N;
  int n_tiles;          // ceil(N / 128)
  int n_blocks;         // 2 n_tiles: 64-query blocks
  int rows_full, rows_split, cols_full, cols_split;   // units that are whole, pieces of each other unit
  float scale, scale_log2;
  int out_fmt, grad_fmt, bias_fmt;
};

struct CbMaps {
  CUtensorMap q64, dout64;      // 64-row tiles (cols kernel)
  CUtensorMap kg, vg;           // by grid rows (rows kernel)
  CUtensorMap k, v;             // 128-row tiles (cols kernel)
};
cudaError_t launch_cb_d64(const CbMaps& maps, const CbArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_cb_d128(const CbMaps& maps, const CbArgs& a, bool bf16, cudaStream_t s);

// Backward of the projection (project_backward.cuh).
struct PbArgs {
  const void* q;         // [tokens, D]
  const void* th;        // [2H-1, D]
  const void* tw;        // [2W-1, D]
  const float* drel_h;   // [tokens, H]
  const float* drel_w;   // [tokens, W]
  const void* dq_in;     // [tokens, D] grad dtype, or null
  void* dq;
  float* parts;          // [CTA][(2H-1) + (2W-1)][D]
  float* dth;
  float* dtw;
  int* status;
  int H, W, N, D;
  long long tokens;      // BH * N
  long long n_tiles;     // ceil(tokens / 128)
  int grad_fmt;
};
cudaError_t launch_project_backward(const PbArgs& a, int ctas, bool bf16, cudaStream_t s);

}  // namespace dera
