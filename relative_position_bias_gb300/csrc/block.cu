// C entry points of dera_block.h: argument checks, how a product is cut, and launches.
#include "../../include/dera_block.h"

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "activation.cuh"
#include "block.cuh"
#include "host.cuh"

using namespace dera;

namespace {

constexpr int kMaxFeatures = 1 << 20;

int elem_size(dera_dtype t) { return t == DERA_F32 ? 4 : 2; }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// ------------------------------------------------------------------------------------ layer norm
dera_status check_ln(int rows, int cols) {
  return rows < 0 || cols < 1 || cols > kLnMaxCols ? DERA_ERR_SHAPE : DERA_OK;
}

// The types of a norm's rows: `other` goes with x's.
bool ln_types(dera_dtype x, dera_dtype other) {
  return is_float(x) && is_float(other) && (other == DERA_F32 || other == x || x == DERA_F32);
}
bool ln_weight_type(dera_dtype w, dera_dtype x, dera_dtype other) {
  return w == DERA_F32 || (is_float(w) && (w == x || w == other));
}

struct Ptr {
  const void* p;
  int align;   // of its elements
};
dera_status check_ptrs(std::initializer_list<Ptr> ptrs, int dev) {
  for (const Ptr& q : ptrs)
    if (q.p && !aligned(q.p, q.align)) return DERA_ERR_ALIGN;
  for (const Ptr& q : ptrs)
    if (q.p) DERA_TRY(check_ptr(q.p, dev));
  return DERA_OK;
}

size_t ln_workspace(int rows, int cols, int sms) {
  // by either plan: whether rows are whole 16-byte chunks is for the call to say
  const int grid = std::max(ln_plan(rows, cols, true, true, sms).grid, ln_plan(rows, cols, true, false, sms).grid);
  return align256(static_cast<size_t>(grid) * 2 * cols * sizeof(float));
}

// ---------------------------------------------------------------------------------------- linear
dera_status check_linear(int B, int N, int heads, int head_dim, int out) {
  if (B < 0 || N < 0 || heads < 1 || head_dim < 1 || out < 1) return DERA_ERR_SHAPE;
  const long long K = static_cast<long long>(heads) * head_dim;
  if (static_cast<long long>(B) * N > 0x7fffffffLL || K > kMaxFeatures || out > kMaxFeatures) return DERA_ERR_SHAPE;
  if (head_dim % 8 != 0 || out % 8 != 0 || (heads > 1 && head_dim % 64 != 0)) return DERA_ERR_SHAPE;
  return DERA_OK;
}

// take_heads, with strides that a TMA descriptor can hold.
dera_status take_tokens(const dera_heads* t, int B, int N, int heads, int d, bool distinct, HeadsPtr* out) {
  DERA_TRY(take_heads(t, B, N, heads, d, distinct, out));
  const long long st[3] = {out->sb, out->st, out->sh};
  const int n[3] = {B, N, heads};
  for (int i = 0; i < 3; ++i)
    if ((n[i] > 1 && st[i] == 0) || st[i] >= (1ll << 37)) return DERA_ERR_SHAPE;
  return DERA_OK;
}

// Contiguous rows of `f` features.
HeadsPtr rows_of(const void* p, int N, int f) {
  return {static_cast<char*>(const_cast<void*>(p)), static_cast<long long>(N) * f, f, 0};
}

// Whether the batches of a view follow one another as its tokens do.
bool merges(const HeadsPtr& t, int B, int N) { return B == 1 || N == 1 || t.sb == static_cast<long long>(N) * t.st; }

// Tokens of one product: [B, N], as one batch where every view allows it.
struct Tokens {
  int B, N;
  bool merged;
  Tokens(int B_, int N_, std::initializer_list<const HeadsPtr*> views) : B(B_), N(N_), merged(true) {
    for (const HeadsPtr* v : views) merged = merged && (!v->data || merges(*v, B_, N_));
    if (merged) {
      B = 1;
      N = B_ * N_;
    }
  }
  HeadsPtr of(HeadsPtr t, int N_) const {
    if (merged) {
      if (N_ == 1) t.st = t.sb;
      t.sb = 0;
    }
    return t;
  }
};

LinView view_of(const HeadsPtr& t, int heads, int d) {
  return {t.sb, t.st, heads > 1 ? t.sh : 0, heads > 1 ? d : 0};
}

// A view whose heads lie side by side is one of plain rows.
void join_heads(const HeadsPtr& t, int* heads, int* d) {
  if (*heads > 1 && t.sh == *d) {
    *d *= *heads;
    *heads = 1;
  }
}

int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

// Columns of a tile for `tokens` of them in a turned product.
int turned_columns(int tokens) { return tokens <= 32 ? 32 : (tokens <= 64 ? 64 : (tokens <= 128 ? 128 : 256)); }

// Cuts rows x cols of D into tiles; false if there are more than a grid holds.
bool cut(LinArgs* a, const LinPlan& p, int batches, int rows, int cols) {
  a->batches = batches;
  a->rows = rows;
  a->cols = cols;
  a->pieces = p.pieces;
  a->piece_steps = p.piece_steps;
  a->m_tiles = ceil_div(rows, p.turned ? 128 : 256);
  a->n_tiles = ceil_div(cols, p.bn);
  if (static_cast<double>(batches) * a->m_tiles * a->n_tiles * a->pieces >= 2147483647.0) return false;
  int far = p.pairs;
  a->by_piece = far % a->pieces;
  a->by_n = (far /= a->pieces) % a->n_tiles;
  a->by_m = (far /= a->n_tiles) % a->m_tiles;
  a->by_b = far / a->m_tiles;
  return true;
}

// How D of tokens (rows) by features is cut, `steps` steps long.  `long_epilogue`: one that outlasts a tile's products.
LinPlan token_plan(const Tokens& tok, int features, int steps, bool f32, bool long_epilogue, int sms) {
  LinPlan p = {};
  p.pieces = 1;
  p.piece_steps = steps;
  // Few tokens take linear_few_kernel: up to 128 always.  More, 256 to a tile, only where a contraction is long and the tiles so
  // few that each has a whole cluster of 8: the pairs' kernel has one CTA pair a tile and takes 5.3 us + 0.23 a step, this one
  // 12 + 0.27 for an eighth of the steps.  256 tokens x 4096 x 1024: 13.4 us against 19.6, 300 x 8192 x 512 15.7 against 33.9; but
  // 256 x 1024 x 1024 11.9 against 8.8 and, with a cluster of 4, 512 x 4096 x 1024 25.3 against 19.7.
  if (tok.merged && (tok.N <= 128 || steps >= 48)) {
    const int bn = turned_columns(tok.N);
    const long long tiles = static_cast<long long>(ceil_div(features, 128)) * ceil_div(tok.N, bn);
    // The largest cluster that leaves every CTA two steps or more and that all tiles can have at the same time.  A cluster lies
    // within a group of SMs that share their way to memory, so that 152 SMs hold 15 of 8, not 19: 256 x 4096 x 1920 (15 tiles)
    // takes 14.3 us, x 2048 in two rounds 25.4.
    int pieces = 8;
    while (pieces > 1 && (2 * pieces > steps || tiles > few_clusters(pieces))) pieces /= 2;
    if (tok.N <= 128 || pieces == 8) {
      p.turned = true;
      p.bn = bn;
      p.pieces = pieces;
      return p;
    }
  }
  const int pairs = std::max(1, sms / 2);
  const double m = static_cast<double>(tok.B) * ceil_div(tok.N, 256);
  const double wide = m * ceil_div(features, 256), narrow = m * ceil_div(features, 128);
  // Time in us by tiles of 256 x 256 and of 256 x 128, fitted to sizes between 196 x 768 x 768 and 9728 x 4096 x 2048: start, end and
  // first loads, and for every wave its steps, or its epilogue where that takes longer.  A narrow tile's step takes not half but
  // 0.85 of a wide one's (the loads of a step are 3/4).
  const double t_wide = 7 + std::ceil(wide / pairs) * std::max(0.27 * steps, 3.0);
  const double t_narrow = 5.3 + std::ceil(narrow / pairs) * std::max(0.23 * steps, 2.4);
  p.bn = t_wide <= t_narrow ? 256 : 128;
  p.fine = f32 && steps > kLinChain;
  p.epi = p.bn == 256 && long_epilogue && !p.fine ? 16 : 8;
  p.pairs = static_cast<int>(std::min<double>(pairs, p.bn == 256 ? wide : narrow));
  return p;
}

// How dW = [out, K] is cut: tiles and pieces of the contraction over `steps` steps.
struct WeightPlan {
  LinPlan p;
  size_t bytes;   // of the pieces
};
WeightPlan weight_plan(int out, int K, int steps, int sms) {
  const int pairs = std::max(1, sms / 2);
  const double tiles = static_cast<double>(ceil_div(out, 256)) * ceil_div(K, 256);
  double best = 0;
  int pieces = 1;
  for (int q = 1; q <= 64 && (q == 1 || 4 * q <= steps); ++q) {
    // in steps of 0.27 us: waves of pieces, each with 8 steps' time for its start and end; and the join, a kernel that reads what the pieces wrote
    double t = std::ceil(tiles * q / pairs) * (ceil_div(steps, q) + 8);
    if (q > 1) t += 8 + 8.0 * q * out * K / 6.8e12 / 0.27e-6;
    if (q == 1 || t < best) {
      best = t;
      pieces = q;
    }
  }
  WeightPlan w = {};
  w.p.piece_steps = ceil_div(steps, pieces);
  w.p.pieces = ceil_div(steps, w.p.piece_steps);
  w.p.bn = 256;
  w.p.pairs = static_cast<int>(std::min<double>(pairs, tiles * w.p.pieces));
  w.bytes = w.p.pieces > 1 ? align256(static_cast<size_t>(w.p.pieces) * out * K * sizeof(float)) : 0;
  return w;
}

// Columns of the epilogue's boxes (as the kernel takes them): 128 bytes of the output's type.
int box_columns(dera_dtype out) { return out == DERA_F32 ? 32 : 64; }

dera_status status_of(cudaError_t e) { return e == cudaSuccess ? DERA_OK : DERA_ERR_CUDA; }

// Partial rows of dy's column sums: four blocks an SM over all columns (256 a block), each with 32 rows or more.
int sum_blocks(long long rows, int out, int sms) {
  return static_cast<int>(std::min<long long>((rows + 31) / 32, std::max(1, 4 * sms / ceil_div(out, 256))));
}

// Workspace of the backward: the column sums' partial rows, then the pieces of dW.
size_t sums_bytes(long long rows, int out, int sms) {
  return align256(static_cast<size_t>(sum_blocks(rows, out, sms)) * out * sizeof(float));
}
size_t linear_backward_workspace(int B, int N, int K, int out, int sms) {
  // whether the batches merge or not
  const long long one = (static_cast<long long>(B) * N + 63) / 64, each = static_cast<long long>(B) * ceil_div(N, 64);
  const long long most = 0x7fffffff;
  return sums_bytes(static_cast<long long>(B) * N, out, sms) + std::max(weight_plan(out, K, static_cast<int>(std::min(one, most)), sms).bytes,
                                         weight_plan(out, K, static_cast<int>(std::min(each, most)), sms).bytes);
}

}  // namespace

extern "C" {

dera_status dera_layer_norm(const void* x, const void* weight, const void* bias, void* y, float* mean, float* rstd,
                            int rows, int cols, long long x_stride, float eps, dera_dtype in_dtype,
                            dera_dtype weight_dtype, dera_dtype out_dtype, void* stream) {
  DERA_TRY(check_ln(rows, cols));
  if ((rows > 1 && x_stride < cols) || !(eps >= 0.f) || std::isinf(eps)) return DERA_ERR_SHAPE;
  if (!ln_types(in_dtype, out_dtype) || (weight && !ln_weight_type(weight_dtype, in_dtype, out_dtype)))
    return DERA_ERR_DTYPE;
  if (rows == 0) return DERA_OK;
  if (!x || !y || !mean || !rstd || (bias && !weight)) return DERA_ERR_NULL;
  int dev = 0;
  DERA_TRY(current_device(&dev));
  const int we = elem_size(weight_dtype);
  DERA_TRY(check_ptrs({{x, elem_size(in_dtype)}, {weight, we}, {bias, we}, {y, elem_size(out_dtype)}, {mean, 4}, {rstd, 4}},
                      dev));
  LnArgs a = {};
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.xs = rows > 1 ? x_stride : cols;
  a.C = cols;
  a.eps = eps;
  a.x_fmt = fmt_of(in_dtype);
  a.w_fmt = fmt_of(weight_dtype);
  a.y_fmt = fmt_of(out_dtype);
  a.status = status_ptr(dev);
  if (!a.status) return DERA_ERR_CUDA;
  const bool vec = cols % 8 == 0 && a.xs % 8 == 0 && aligned(x, 16) && aligned(y, 16);
  const int sms = sm_count(dev);
  return status_of(launch_ln(a, ln_plan(rows, cols, false, vec, sms), vec, sms, static_cast<cudaStream_t>(stream)));
}

dera_status dera_layer_norm_backward_workspace_size(int rows, int cols, size_t* bytes) {
  if (!bytes) return DERA_ERR_NULL;
  DERA_TRY(check_ln(rows, cols));
  *bytes = 0;
  if (rows == 0) return DERA_OK;
  int dev = 0;
  DERA_TRY(current_device(&dev));
  *bytes = ln_workspace(rows, cols, sm_count(dev));
  return DERA_OK;
}

dera_status dera_layer_norm_backward(const void* dy, const void* x, const float* mean, const float* rstd,
                                     const void* weight, const void* dres, void* dx, float* dweight, float* dbias,
                                     int rows, int cols, long long x_stride, dera_dtype in_dtype,
                                     dera_dtype weight_dtype, dera_dtype dout_dtype, dera_dtype grad_dtype,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  DERA_TRY(check_ln(rows, cols));
  if (rows > 1 && x_stride < cols) return DERA_ERR_SHAPE;
  if (!ln_types(in_dtype, dout_dtype) || !(grad_dtype == DERA_F32 || grad_dtype == in_dtype) ||
      (weight && !ln_weight_type(weight_dtype, in_dtype, dout_dtype)))
    return DERA_ERR_DTYPE;
  if ((dweight == nullptr) != (dbias == nullptr)) return DERA_ERR_NULL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int dev = 0;
  if (rows == 0) {   // only the parameters' gradients are written, as zeros
    if (!dweight) return DERA_OK;
    DERA_TRY(current_device(&dev));
    DERA_TRY(check_ptrs({{dweight, 4}, {dbias, 4}}, dev));
    for (float* p : {dweight, dbias})
      if (cudaMemsetAsync(p, 0, cols * sizeof(float), s) != cudaSuccess) return DERA_ERR_CUDA;
    return DERA_OK;
  }
  if (!dy || !x || !mean || !rstd || !dx) return DERA_ERR_NULL;
  DERA_TRY(current_device(&dev));
  DERA_TRY(check_ptrs({{dy, elem_size(dout_dtype)}, {x, elem_size(in_dtype)}, {mean, 4}, {rstd, 4},
                       {weight, elem_size(weight_dtype)}, {dres, elem_size(grad_dtype)}, {dx, elem_size(grad_dtype)},
                       {dweight, 4}, {dbias, 4}},
                      dev));
  const int sms = sm_count(dev);
  if (dweight) DERA_TRY(check_workspace(workspace, workspace_bytes, ln_workspace(rows, cols, sms), dev));
  LnArgs a = {};
  a.x = x;
  a.w = weight;
  a.dy = dy;
  a.dres = dres;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.dx = dx;
  a.parts = dweight ? static_cast<float*>(workspace) : nullptr;
  a.rows = rows;
  a.xs = rows > 1 ? x_stride : cols;
  a.C = cols;
  a.x_fmt = fmt_of(in_dtype);
  a.w_fmt = fmt_of(weight_dtype);
  a.y_fmt = fmt_of(dout_dtype);
  a.dx_fmt = fmt_of(grad_dtype);
  a.status = status_ptr(dev);
  if (!a.status) return DERA_ERR_CUDA;
  const bool vec = cols % 8 == 0 && a.xs % 8 == 0 && aligned(x, 16) && aligned(dy, 16) && aligned(dres, 16) && aligned(dx, 16);
  return status_of(launch_ln_backward(a, ln_plan(rows, cols, true, vec, sms), vec, dweight, dbias, s));
}

dera_status dera_linear(const dera_heads* x, const void* weight, const void* bias, const void* residual, void* y,
                        void* pre, int B, int N, int heads, int head_dim, int out_features, dera_activation activation,
                        dera_dtype in_dtype, dera_dtype bias_dtype, dera_dtype out_dtype, void* stream) {
  DERA_TRY(check_linear(B, N, heads, head_dim, out_features));
  if (!is16(in_dtype) || !(out_dtype == DERA_F32 || out_dtype == in_dtype) || activation < 0 || activation >= kActs ||
      (bias && !(bias_dtype == DERA_F32 || bias_dtype == in_dtype)))
    return DERA_ERR_DTYPE;
  if (B == 0 || N == 0) return DERA_OK;
  HeadsPtr xt;
  DERA_TRY(take_tokens(x, B, N, heads, head_dim, false, &xt));
  DERA_TRY(check_host({weight, y}));
  for (const void* p : {bias, residual, static_cast<const void*>(pre)})
    if (p && !aligned(p, 16)) return DERA_ERR_ALIGN;
  int dev = 0;
  DERA_TRY(current_device(&dev));
  for (const void* p : {static_cast<const void*>(xt.data), weight, bias, residual, static_cast<const void*>(y),
                        static_cast<const void*>(pre)})
    if (p) DERA_TRY(check_ptr(p, dev));
  const int K = heads * head_dim;
  join_heads(xt, &heads, &head_dim);
  const Tokens tok(B, N, {&xt});
  LinArgs a = {};
  a.bias = bias;
  a.aux = residual;
  a.pre = pre;
  a.out = y;
  a.status = status_ptr(dev);
  if (!a.status) return DERA_ERR_CUDA;
  a.out_at = a.aux_at = view_of(tok.of(rows_of(y, N, out_features), N), 1, out_features);
  a.steps = a.steps_batch = ceil_div(K, 64);
  a.act = activation;
  a.fmt = fmt_of(in_dtype);
  a.bias_fmt = fmt_of(bias_dtype);
  a.aux_fmt = a.out_fmt = fmt_of(out_dtype);
  // (linear_pair.cuh has both sides measured; with one slot a warp there is no room for a residual and an argument)
  const bool long_epilogue = activation > DERA_ACT_RELU && a.steps <= (activation == DERA_ACT_GELU ? 16 : 12) && !residual &&
                             out_dtype != DERA_F32;
  const LinPlan p = token_plan(tok, out_features, a.steps, out_dtype == DERA_F32, long_epilogue, sm_count(dev));
  if (!(p.turned ? cut(&a, p, 1, out_features, tok.N) : cut(&a, p, tok.B, tok.N, out_features))) return DERA_ERR_SHAPE;
  LinMaps m = {};
  const HeadsPtr xm = tok.of(xt, N), wm = rows_of(weight, out_features, K);
  CUtensorMap *mx = p.turned ? &m.b : &m.a, *mw = p.turned ? &m.a : &m.b;
  (p.turned ? a.b_d : a.a_d) = heads > 1 ? head_dim : 0;
  if (!map_tokens(mx, xm, in_dtype, tok.B, tok.N, heads, head_dim, p.turned ? p.bn : 128) ||
      !map_tokens(mw, wm, in_dtype, 1, out_features, 1, K, p.turned ? 128 : p.bn / 2))
    return DERA_ERR_CUDA;
  if (!p.turned) {
    const HeadsPtr ym = tok.of(rows_of(y, N, out_features), N), rm = {const_cast<char*>(static_cast<const char*>(residual)), ym.sb, ym.st, 0},
                   pm = {static_cast<char*>(pre), ym.sb, ym.st, 0};
    const int box = p.epi == 16 && pre ? 32 : box_columns(out_dtype);   // as the kernel's `narrow`
    if (!map_boxes(&m.out, ym, out_dtype, tok.B, tok.N, 1, out_features, box) ||
        (residual && !map_boxes(&m.aux, rm, out_dtype, tok.B, tok.N, 1, out_features, box)) ||
        (pre && !map_boxes(&m.pre, pm, in_dtype, tok.B, tok.N, 1, out_features, box)))
      return DERA_ERR_CUDA;
  }
  return status_of(launch_linear_forward(m, a, p, static_cast<cudaStream_t>(stream)));
}

dera_status dera_linear_backward_workspace_size(int B, int N, int heads, int head_dim, int out_features, size_t* bytes) {
  if (!bytes) return DERA_ERR_NULL;
  DERA_TRY(check_linear(B, N, heads, head_dim, out_features));
  *bytes = 0;
  if (B == 0 || N == 0) return DERA_OK;
  int dev = 0;
  DERA_TRY(current_device(&dev));
  *bytes = linear_backward_workspace(B, N, heads * head_dim, out_features, sm_count(dev));
  return DERA_OK;
}

dera_status dera_linear_backward(const void* dy, const dera_heads* x, const void* weight, const dera_heads* input_pre,
                                 const dera_heads* dx, void* dweight, float* dbias, int B, int N, int heads, int head_dim,
                                 int out_features, dera_activation input_activation, dera_dtype in_dtype,
                                 dera_dtype grad_dtype, dera_dtype weight_grad_dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  DERA_TRY(check_linear(B, N, heads, head_dim, out_features));
  if (!is16(in_dtype) || !(grad_dtype == DERA_F32 || grad_dtype == in_dtype) ||
      !(weight_grad_dtype == DERA_F32 || weight_grad_dtype == in_dtype) || input_activation < 0 ||
      input_activation >= kActs)
    return DERA_ERR_DTYPE;
  const int K = heads * head_dim;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int dev = 0;
  for (const void* p : {static_cast<const void*>(dweight), static_cast<const void*>(dbias)})
    if (p && !aligned(p, 16)) return DERA_ERR_ALIGN;
  if (B == 0 || N == 0) {   // no tokens: only the parameters' gradients are written, as zeros
    if (!dweight && !dbias) return DERA_OK;
    DERA_TRY(current_device(&dev));
    for (const void* p : {static_cast<const void*>(dweight), static_cast<const void*>(dbias)})
      if (p) DERA_TRY(check_ptr(p, dev));
    if (dweight && cudaMemsetAsync(dweight, 0, static_cast<size_t>(out_features) * K * elem_size(weight_grad_dtype), s) !=
                       cudaSuccess)
      return DERA_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, out_features * sizeof(float), s) != cudaSuccess) return DERA_ERR_CUDA;
    return DERA_OK;
  }
  DERA_TRY(check_host({dy}));
  HeadsPtr xt = {}, pt = {}, dt = {};
  if (dweight) DERA_TRY(take_tokens(x, B, N, heads, head_dim, false, &xt));
  if (dx) {
    DERA_TRY(check_host({weight}));
    DERA_TRY(take_tokens(dx, B, N, heads, head_dim, true, &dt));
    if ((input_pre == nullptr) != (input_activation == DERA_ACT_NONE)) return DERA_ERR_NULL;
    if (input_pre) DERA_TRY(take_tokens(input_pre, B, N, heads, head_dim, false, &pt));
  }
  DERA_TRY(current_device(&dev));
  for (const void* p : {dy, static_cast<const void*>(xt.data), dx ? weight : nullptr, static_cast<const void*>(pt.data),
                        static_cast<const void*>(dt.data), static_cast<const void*>(dweight),
                        static_cast<const void*>(dbias)})
    if (p) DERA_TRY(check_ptr(p, dev));
  const int sms = sm_count(dev);
  if (dweight || dbias)
    DERA_TRY(check_workspace(workspace, workspace_bytes, linear_backward_workspace(B, N, K, out_features, sms), dev));
  int* status = status_ptr(dev);
  if (!status) return DERA_ERR_CUDA;
  const HeadsPtr gt = rows_of(dy, N, out_features);
  if (dx) {
    const Tokens tok(B, N, {&dt, &pt});
    int h = heads, d = head_dim;
    LinArgs a = {};
    a.aux = pt.data;
    a.out = dt.data;
    a.status = status;
    a.out_at = view_of(tok.of(dt, N), h, d);
    a.aux_at = view_of(tok.of(pt, N), h, d);
    a.steps = a.steps_batch = ceil_div(out_features, 64);
    a.act = input_activation;
    a.fmt = a.aux_fmt = fmt_of(in_dtype);
    a.out_fmt = fmt_of(grad_dtype);
    const bool long_epilogue = input_activation == DERA_ACT_GELU || (input_activation > DERA_ACT_RELU && a.steps <= 12);
    const LinPlan p = token_plan(tok, K, a.steps, grad_dtype == DERA_F32, long_epilogue, sms);
    LinMaps m = {};
    CUtensorMap *mg = p.turned ? &m.b : &m.a, *mw = p.turned ? &m.a : &m.b;
    if (!(p.turned ? cut(&a, p, 1, K, tok.N) : cut(&a, p, tok.B, tok.N, K))) return DERA_ERR_SHAPE;
    if (!map_tokens(mg, tok.of(gt, N), in_dtype, tok.B, tok.N, 1, out_features, p.turned ? p.bn : 128) ||
        !map_tokens(mw, rows_of(weight, out_features, K), in_dtype, 1, out_features, 1, K, 64))
      return DERA_ERR_CUDA;
    const int box = box_columns(grad_dtype);
    if (!p.turned && (!map_boxes(&m.out, tok.of(dt, N), grad_dtype, tok.B, tok.N, h, d, box) ||
                      (pt.data && !map_boxes(&m.aux, tok.of(pt, N), in_dtype, tok.B, tok.N, h, d, box))))
      return DERA_ERR_CUDA;
    DERA_TRY(status_of(launch_linear_input(m, a, p, s)));
  }
  LinJoin join = {};
  if (dweight) {
    int h = heads, d = head_dim;
    join_heads(xt, &h, &d);
    const Tokens tok(B, N, {&xt});
    LinArgs a = {};
    a.out = dweight;
    a.status = status;
    a.out_at = {0, K, 0, 0};
    a.b_d = h > 1 ? d : 0;
    a.steps_batch = ceil_div(tok.N, 64);
    if (static_cast<long long>(tok.B) * a.steps_batch > 0x7fffffffLL) return DERA_ERR_SHAPE;
    a.steps = tok.B * a.steps_batch;
    a.fmt = fmt_of(in_dtype);
    a.out_fmt = fmt_of(weight_grad_dtype);
    WeightPlan w = weight_plan(out_features, K, a.steps, sms);
    w.p.beside = dx != nullptr;
    if (!cut(&a, w.p, 1, out_features, K)) return DERA_ERR_SHAPE;
    if (w.p.pieces > 1) a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + sums_bytes(static_cast<long long>(B) * N, out_features, sms));
    LinMaps m = {};
    if (!map_tokens(&m.a, tok.of(gt, N), in_dtype, tok.B, tok.N, 1, out_features, 64) ||
        !map_tokens(&m.b, tok.of(xt, N), in_dtype, tok.B, tok.N, h, d, 64))
      return DERA_ERR_CUDA;
    DERA_TRY(status_of(launch_linear_weight(m, a, w.p, s)));
    if (w.p.pieces > 1) {
      join.parts = a.parts;
      join.dw = dweight;
      join.n = static_cast<long long>(out_features) * K;
      join.pieces = w.p.pieces;
      join.dw_fmt = a.out_fmt;
    }
  }
  if (dbias) {
    const long long rows = static_cast<long long>(B) * N;
    join.sum_rows = sum_blocks(rows, out_features, sms);
    join.sums = static_cast<float*>(workspace);
    join.db = dbias;
    join.out = out_features;
    DERA_TRY(status_of(launch_column_sums(dy, rows, out_features, fmt_of(in_dtype), static_cast<float*>(workspace),
                                          join.sum_rows, dx || dweight, s)));
  }
  if (join.dw || join.db) DERA_TRY(status_of(launch_linear_join(join, s)));
  return DERA_OK;
}

dera_status dera_activation_backward(const void* dy, const void* pre, void* dpre, long long n, dera_activation activation,
                                     dera_dtype pre_dtype, dera_dtype dout_dtype, dera_dtype grad_dtype, void* stream) {
  if (n < 0) return DERA_ERR_SHAPE;
  if (activation <= DERA_ACT_NONE || activation >= kActs || !is_float(pre_dtype) ||
      !(dout_dtype == DERA_F32 || dout_dtype == pre_dtype) || !(grad_dtype == DERA_F32 || grad_dtype == pre_dtype))
    return DERA_ERR_DTYPE;
  if (n == 0) return DERA_OK;
  DERA_TRY(check_host({dy, pre, dpre}));
  int dev = 0;
  DERA_TRY(current_device(&dev));
  for (const void* p : {dy, pre, static_cast<const void*>(dpre)}) DERA_TRY(check_ptr(p, dev));
  const ActArgs a = {dy, pre, dpre, n, activation, fmt_of(pre_dtype), fmt_of(dout_dtype), fmt_of(grad_dtype)};
  return status_of(launch_act_backward(a, sm_count(dev), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
