// Launch arguments and launchers behind the entry points of dera_block.h.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "train.cuh"

namespace dera {

// ------------------------------------------------------------------------------------ layer norm
constexpr int kLnMaxCols = 16384;

struct LnArgs {
  const void* x;          // [rows, C], rows xs elements apart
  const void* w;          // [C] or null
  const void* b;
  void* y;                // [rows, C]
  float* mean;
  float* rstd;
  const void* dy;         // backward: [rows, C]
  const void* dres;       // [rows, C] in dx's type, or null
  const float* mean_in;
  const float* rstd_in;
  void* dx;               // [rows, C]
  float* parts;           // [blocks][2 C] partial dw, db, or null
  long long rows, xs;
  float eps;
  int C, tpr;             // tpr: threads a row
  int sets;               // sets of rows in the ring
  int* status;
  int x_fmt, w_fmt, y_fmt, dx_fmt;   // y_fmt: dy's too
};

// How a layer norm's rows are cut.
struct LnPlan {
  int threads, tpr, grid, blocks;   // blocks: of an SM
};
LnPlan ln_plan(long long rows, int C, bool backward, bool vec, int sms);
cudaError_t launch_ln(LnArgs& a, const LnPlan& p, bool vec, int sms, cudaStream_t s);
cudaError_t launch_ln_backward(LnArgs& a, const LnPlan& p, bool vec, float* dw, float* db, cudaStream_t s);
// d1[c], d2[c]: the first n1 and the other columns of `rows` partial rows of n, summed
cudaError_t launch_partial_rows(const float* parts, int rows, int n, int n1, float* d1, float* d2, cudaStream_t s);

// ------------------------------------------------------------------------------------ activations
struct ActArgs {
  const void* dy;
  const void* pre;
  void* dpre;
  long long n;
  int act, fmt, z_fmt, out_fmt;   // pre's, dy's and dpre's types
};
cudaError_t launch_act_backward(const ActArgs& a, int sms, cudaStream_t s);

// ---------------------------------------------------------------------------------------- linear
// A tensor of tokens by its strides: element (b, n, f) is at b sb + n sn + (f / d) sh + f % d (d = 0: one head).
struct LinView {
  long long sb, sn, sh;
  int d;
};

// D = A B^T over `steps` steps of 64, rows of A against rows of B, and what becomes of an element of D.
//   kLinForward   rows: tokens of x, columns: rows of W;           y = act(D + bias) + residual
//   kLinInput     rows: tokens of dy, columns: columns of W;       dx = D * slope(input_pre)
//   kLinWeight    rows: columns of dy, columns: features of x;     dW = D
// With `turned` the operands are swapped, rows of D are features and columns tokens.
enum : int { kLinForward = 0, kLinInput = 1, kLinWeight = 2 };

struct LinArgs {
  const void* bias;      // [features] or null
  const void* aux;       // residual (forward), input_pre (input gradient), or null
  void* pre;             // forward: D + bias before the activation, or null
  void* out;
  float* parts;          // a piece of a split contraction: [piece][rows][cols] fp32, or null
  int* status;
  LinView out_at, aux_at;
  int a_d, b_d;          // features a head of each operand as TMA sees it (0: one head)
  int rows, cols;        // of D: rows of one batch, and columns
  int batches, m_tiles, n_tiles;   // m_tiles: of one batch
  int steps, steps_batch;          // contraction steps of 64, and those of one batch where it runs over tokens
  int pieces;                      // kLinWeight, turned: pieces of the contraction
  int piece_steps;                 // kLinWeight: steps of a piece (the last may have fewer)
  int by_piece, by_n, by_m, by_b;  // how far a pair's next tile is, as digits of (batch, m, n, piece)
  int act, fmt, bias_fmt, aux_fmt, out_fmt;
};

constexpr int kLinChain = 8;   // steps of a chain of sums on the tensor core, where its cuts matter (linear_pair.cuh)

struct LinMaps {
  CUtensorMap a, b;
  CUtensorMap out, aux, pre;   // pairs, but for dW: boxes of 32 rows x 32 columns of what lies beside D
};

struct LinPlan {
  int bn;                // columns of a tile
  bool turned;
  int pairs;             // pairs of CTAs that share tiles of 256 rows (0: turned)
  int epi;               // epilogue warps of a CTA of a pair
  bool fine;             // long sums in chains (an fp32 output)
  int pieces, piece_steps;
  bool beside;           // kLinWeight: launched early, with the kernel before it on the stream, which is of the same call
};
// The end of a backward: dW from its pieces, and db from its partial rows (either may be absent).
struct LinJoin {
  const float* parts;    // [pieces][n]
  void* dw;
  long long n;           // a multiple of 8
  int pieces, dw_fmt;
  const float* sums;     // [sum_rows][out]
  float* db;
  int sum_rows, out;
};
cudaError_t launch_linear_join(const LinJoin& j, cudaStream_t s);
// Clusters of 2, 4 or 8 CTAs of linear_few_kernel that run at the same time on the current device, one CTA an SM.
int few_clusters(int size);
cudaError_t launch_linear_forward(const LinMaps& m, const LinArgs& a, const LinPlan& p, cudaStream_t s);
cudaError_t launch_linear_input(const LinMaps& m, const LinArgs& a, const LinPlan& p, cudaStream_t s);
cudaError_t launch_linear_weight(const LinMaps& m, const LinArgs& a, const LinPlan& p, cudaStream_t s);
// partial rows of g's column sums: [blocks][cols]
// beside: early, with the kernel before it on the stream, which is of the same call
cudaError_t launch_column_sums(const void* g, long long rows, int cols, int fmt, float* parts, int blocks, bool beside, cudaStream_t s);

}  // namespace dera
