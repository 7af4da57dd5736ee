// C entry points of dera_train.h: argument checks and launches.
#include "../../include/dera_train.h"

#include <cmath>
#include <cstdint>
#include <utility>

#include "host.cuh"
#include "train.cuh"

using namespace dera;

namespace {

constexpr int kMaxHeads = 16384;   // so that the groups of q, k and v fit one grid dimension

dera_status check_workspace(const void* ws, size_t have, size_t need, int dev) {
  if (need == 0) return DERA_OK;
  if (!ws || have < need) return DERA_ERR_SCRATCH;
  if (reinterpret_cast<uintptr_t>(ws) % 256 != 0) return DERA_ERR_ALIGN;
  return check_ptr(ws, dev);
}

// One tensor in token order, its strides made ready for the kernels (0 where the
// dimension has size one).  `distinct`: no two rows may share an element.
dera_status take_heads(const dera_heads* t, int B, int N, int heads, int d, bool distinct, HeadsPtr* out) {
  if (!t || !t->data) return DERA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(t->data) % 16 != 0) return DERA_ERR_ALIGN;
  long long st[3] = {t->stride_batch, t->stride_token, t->stride_head};
  long long n[3] = {B, N, heads};
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) st[i] = 0;
    if (st[i] < 0) return DERA_ERR_SHAPE;
    if (st[i] % 8 != 0) return DERA_ERR_ALIGN;
  }
  *out = {static_cast<char*>(t->data), st[0], st[1], st[2]};
  if (!distinct) return DERA_OK;
  // innermost first, every stride steps over all that lies inside it
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[j] < st[i]) {
        std::swap(st[i], st[j]);
        std::swap(n[i], n[j]);
      }
  __int128 inside = d;
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (st[i] < inside) return DERA_ERR_SHAPE;
    inside += static_cast<__int128>(n[i] - 1) * st[i];
  }
  return DERA_OK;
}

dera_status check_qk(int B, int N, int q_heads, int kv_heads, int head_dim) {
  if (head_dim != 64 && head_dim != 128) return DERA_ERR_HEAD_DIM;
  if (B < 0 || N < 0 || q_heads < 1 || kv_heads < 1 || q_heads > kMaxHeads || kv_heads > kMaxHeads)
    return DERA_ERR_SHAPE;
  if (static_cast<long long>(B) * N > 0x7fffffffLL) return DERA_ERR_SHAPE;
  return DERA_OK;
}

// The arguments that the forward and the backward share, into `a`.
dera_status take_qk(QkArgs* a, const void* q_weight, const void* k_weight, const float* cos, const float* sin,
                    const int* positions, int B, int N, int q_heads, int kv_heads, bool v, int rotary_dim,
                    int table_rows, float eps, int dev) {
  if ((q_weight == nullptr) != (k_weight == nullptr)) return DERA_ERR_NULL;
  if (rotary_dim > 0) DERA_TRY(check_host({cos, sin}));
  for (const void* p : {q_weight, k_weight, static_cast<const void*>(rotary_dim > 0 ? cos : nullptr),
                        static_cast<const void*>(rotary_dim > 0 ? sin : nullptr),
                        static_cast<const void*>(rotary_dim > 0 ? positions : nullptr)})
    if (p) {
      if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return DERA_ERR_ALIGN;
      DERA_TRY(check_ptr(p, dev));
    }
  a->w[0] = q_weight;
  a->w[1] = k_weight;
  a->cos = cos;
  a->sin = sin;
  a->positions = positions;
  a->heads[0] = q_heads;
  a->heads[1] = kv_heads;
  a->heads[2] = v ? kv_heads : 0;
  a->N = N;
  a->table_rows = table_rows;
  a->half = rotary_dim / 2;
  a->tokens = static_cast<long long>(B) * N;
  a->eps = eps;
  return DERA_OK;
}

dera_status check_rotary(int N, int head_dim, int rotary_dim, int table_rows, const int* positions, float eps) {
  if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 16 != 0) return DERA_ERR_SHAPE;
  if (rotary_dim > 0 && (table_rows < 1 || (!positions && table_rows < N))) return DERA_ERR_SHAPE;
  if (!(eps >= 0.f) || std::isinf(eps)) return DERA_ERR_SHAPE;
  return DERA_OK;
}

int rotation_mode(int rotary_dim, int interleaved) {
  return rotary_dim == 0 ? kRotNone : (interleaved ? kRotPairs : kRotHalf);
}

size_t qk_workspace(int B, int N, int q_heads, int kv_heads, int head_dim, int sms) {
  size_t most = 0;
  for (int v = 0; v < 2; ++v) {   // with v or without: the larger of the two plans
    const int heads[3] = {q_heads, kv_heads, v ? kv_heads : 0};
    const QkPlan p = qk_plan(static_cast<long long>(B) * N, heads, head_dim, true, sms);
    const size_t bytes = align256(static_cast<size_t>(p.part_rows_q + p.part_rows_k) * head_dim * sizeof(float));
    most = bytes > most ? bytes : most;
  }
  return most;
}

// Workspace of the compact-bias backward: fp32 regions, each 256-byte aligned.
struct CbLayout {
  int n_tiles, units, rows_steps, cols_steps;
  CbSplit rows, cols;
  size_t hl, rw, nD, parts_rows, parts_cols, total;
  CbLayout(int BH, int H, int W, int d, int sms) {
    const int N = H * W;
    n_tiles = (N + 127) / 128;
    units = BH * n_tiles;
    cb_split(units, cb_rows_steps(H, W), (N + 63) / 64, sms, &rows, &cols);
    const size_t blocks = static_cast<size_t>(BH) * 2 * n_tiles;
    size_t o = 0;
    auto take = [&](size_t floats) {
      const size_t at = o;
      o += align256(floats * sizeof(float));
      return at;
    };
    hl = take(blocks * H * kCbRow);
    rw = take(blocks * W * kCbRow);
    nD = take(blocks * 64);
    parts_rows = take(static_cast<size_t>(rows.tail(units)) * rows.split * 128 * (d + W));
    parts_cols = take(static_cast<size_t>(cols.tail(units)) * cols.split * 128 * 2 * d);
    total = o;
  }
};

dera_status check_cb(int BH, int H, int W, int head_dim) {
  DERA_TRY(check_shape(BH, H, W, head_dim));
  const long long tiles = (static_cast<long long>(H) * W + 127) / 128;
  return tiles * BH > (1ll << 30) ? DERA_ERR_SHAPE : DERA_OK;
}

// CTAs of the projection's backward for one 64-column slice: one an SM over all slices, no more
// than there are tiles.
int pb_ctas(int BH, int H, int W, int d, int sms) {
  const long long tiles = (static_cast<long long>(BH) * H * W + 127) / 128;
  const long long most = sms >= d / 64 ? sms / (d / 64) : 1;
  return static_cast<int>(tiles < most ? tiles : most);
}
size_t pb_workspace(int BH, int H, int W, int d, int sms) {
  return align256(static_cast<size_t>(pb_ctas(BH, H, W, d, sms)) * (2 * H - 1 + 2 * W - 1) * d * sizeof(float));
}

}  // namespace

extern "C" {

dera_status dera_qk_norm_rope(const dera_heads* q, const dera_heads* k, const dera_heads* v, const void* q_weight,
                              const void* k_weight, const float* cos, const float* sin, const int* positions,
                              void* q_out, void* k_out, void* v_out, int B, int N, int q_heads, int kv_heads,
                              int head_dim, int rotary_dim, int table_rows, int interleaved, float eps,
                              dera_dtype in_dtype, dera_dtype weight_dtype, void* stream) {
  DERA_TRY(check_qk(B, N, q_heads, kv_heads, head_dim));
  DERA_TRY(check_rotary(N, head_dim, rotary_dim, table_rows, positions, eps));
  if (!is16(in_dtype) || (q_weight && !(weight_dtype == DERA_F32 || weight_dtype == in_dtype))) return DERA_ERR_DTYPE;
  if (B == 0 || N == 0) return DERA_OK;
  if ((v == nullptr) != (v_out == nullptr)) return DERA_ERR_NULL;
  QkArgs a = {};
  DERA_TRY(take_heads(q, B, N, q_heads, head_dim, false, &a.x[0]));
  DERA_TRY(take_heads(k, B, N, kv_heads, head_dim, false, &a.x[1]));
  if (v) DERA_TRY(take_heads(v, B, N, kv_heads, head_dim, false, &a.x[2]));
  DERA_TRY(check_host({q_out, k_out}));
  if (v) DERA_TRY(check_host({v_out}));
  if ((q_weight == nullptr) != (k_weight == nullptr)) return DERA_ERR_NULL;
  int dev = 0;
  DERA_TRY(current_device(&dev));
  for (const void* p : {static_cast<const void*>(a.x[0].data), static_cast<const void*>(a.x[1].data),
                        static_cast<const void*>(a.x[2].data), static_cast<const void*>(q_out),
                        static_cast<const void*>(k_out), static_cast<const void*>(v_out)})
    if (p) DERA_TRY(check_ptr(p, dev));
  DERA_TRY(take_qk(&a, q_weight, k_weight, cos, sin, positions, B, N, q_heads, kv_heads, v != nullptr, rotary_dim,
                   table_rows, eps, dev));
  a.zo[0] = q_out;
  a.zo[1] = k_out;
  a.zo[2] = v_out;
  a.w_fmt = fmt_of(weight_dtype);
  const QkPlan p = qk_plan(a.tokens, a.heads, head_dim, false, sm_count(dev));
  return launch_qk(a, p, head_dim, rotation_mode(rotary_dim, interleaved), in_dtype == DERA_BF16, q_weight != nullptr,
                   false, nullptr, nullptr, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? DERA_OK
             : DERA_ERR_CUDA;
}

dera_status dera_qk_norm_rope_backward_workspace_size(int B, int N, int q_heads, int kv_heads, int head_dim,
                                                      size_t* bytes) {
  if (!bytes) return DERA_ERR_NULL;
  DERA_TRY(check_qk(B, N, q_heads, kv_heads, head_dim));
  *bytes = 0;
  if (B == 0 || N == 0) return DERA_OK;
  int dev = 0;
  DERA_TRY(current_device(&dev));
  *bytes = qk_workspace(B, N, q_heads, kv_heads, head_dim, sm_count(dev));
  return DERA_OK;
}

dera_status dera_qk_norm_rope_backward(const dera_heads* q, const dera_heads* k, const void* q_weight,
                                       const void* k_weight, const float* cos, const float* sin, const int* positions,
                                       const void* dq_out, const void* dk_out, const void* dv_out,
                                       const dera_heads* dq, const dera_heads* dk, const dera_heads* dv,
                                       float* dq_weight, float* dk_weight, int B, int N, int q_heads, int kv_heads,
                                       int head_dim, int rotary_dim, int table_rows, int interleaved, float eps,
                                       dera_dtype in_dtype, dera_dtype weight_dtype, dera_dtype dout_dtype,
                                       dera_dtype grad_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  DERA_TRY(check_qk(B, N, q_heads, kv_heads, head_dim));
  DERA_TRY(check_rotary(N, head_dim, rotary_dim, table_rows, positions, eps));
  const bool norm = q_weight != nullptr;
  if (!is16(in_dtype) || (norm && !(weight_dtype == DERA_F32 || weight_dtype == in_dtype)) ||
      !(dout_dtype == DERA_F32 || dout_dtype == in_dtype) || !(grad_dtype == DERA_F32 || grad_dtype == in_dtype))
    return DERA_ERR_DTYPE;
  if ((q_weight == nullptr) != (k_weight == nullptr)) return DERA_ERR_NULL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int dev = 0;
  if (B == 0 || N == 0) {   // no rows: only the weights' gradients are written, as zeros
    if (!norm) return DERA_OK;
    DERA_TRY(check_host({dq_weight, dk_weight}));
    DERA_TRY(current_device(&dev));
    for (float* p : {dq_weight, dk_weight}) {
      DERA_TRY(check_ptr(p, dev));
      if (cudaMemsetAsync(p, 0, head_dim * sizeof(float), s) != cudaSuccess) return DERA_ERR_CUDA;
    }
    return DERA_OK;
  }
  if ((dv == nullptr) != (dv_out == nullptr)) return DERA_ERR_NULL;
  QkArgs a = {};
  if (norm) {
    DERA_TRY(take_heads(q, B, N, q_heads, head_dim, false, &a.x[0]));
    DERA_TRY(take_heads(k, B, N, kv_heads, head_dim, false, &a.x[1]));
    DERA_TRY(check_host({dq_weight, dk_weight}));
  }
  DERA_TRY(take_heads(dq, B, N, q_heads, head_dim, true, &a.dx[0]));
  DERA_TRY(take_heads(dk, B, N, kv_heads, head_dim, true, &a.dx[1]));
  if (dv) DERA_TRY(take_heads(dv, B, N, kv_heads, head_dim, true, &a.dx[2]));
  DERA_TRY(check_host({dq_out, dk_out}));
  if (dv) DERA_TRY(check_host({dv_out}));
  DERA_TRY(current_device(&dev));
  for (const void* p : {static_cast<const void*>(a.x[0].data), static_cast<const void*>(a.x[1].data),
                        static_cast<const void*>(a.dx[0].data), static_cast<const void*>(a.dx[1].data),
                        static_cast<const void*>(a.dx[2].data), dq_out, dk_out, dv_out,
                        static_cast<const void*>(norm ? dq_weight : nullptr),
                        static_cast<const void*>(norm ? dk_weight : nullptr)})
    if (p) DERA_TRY(check_ptr(p, dev));
  DERA_TRY(take_qk(&a, q_weight, k_weight, cos, sin, positions, B, N, q_heads, kv_heads, dv != nullptr, rotary_dim,
                   table_rows, eps, dev));
  const int sms = sm_count(dev);
  if (norm)
    DERA_TRY(check_workspace(workspace, workspace_bytes, qk_workspace(B, N, q_heads, kv_heads, head_dim, sms), dev));
  a.z[0] = dq_out;
  a.z[1] = dk_out;
  a.z[2] = dv_out;
  a.parts = static_cast<float*>(workspace);
  a.w_fmt = fmt_of(weight_dtype);
  a.z_fmt = fmt_of(dout_dtype);
  a.dx_fmt = fmt_of(grad_dtype);
  const QkPlan p = qk_plan(a.tokens, a.heads, head_dim, true, sms);
  return launch_qk(a, p, head_dim, rotation_mode(rotary_dim, interleaved), in_dtype == DERA_BF16, norm, true, dq_weight,
                   dk_weight, s) == cudaSuccess
             ? DERA_OK
             : DERA_ERR_CUDA;
}

dera_status dera_relpos_attention_lse(const void* q, const void* k, const void* v, const void* rel_h,
                                      const void* rel_w, void* out, float* lse, int BH, int H, int W, int head_dim,
                                      float scale, dera_dtype in_dtype, dera_dtype bias_dtype, dera_dtype out_dtype,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  DERA_TRY(check_shape(BH, H, W, head_dim));
  if (!is16(in_dtype) || !is_float(bias_dtype) || !(out_dtype == DERA_F32 || out_dtype == in_dtype))
    return DERA_ERR_DTYPE;
  if (BH == 0) return DERA_OK;
  DERA_TRY(check_host({q, k, v, rel_h, rel_w, out, lse}));
  int dev = 0;
  DERA_TRY(current_device(&dev));
  for (const void* p : {q, k, v, rel_h, rel_w, static_cast<const void*>(out), static_cast<const void*>(lse)})
    DERA_TRY(check_ptr(p, dev));
  if (workspace) {
    if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return DERA_ERR_ALIGN;
    DERA_TRY(check_ptr(workspace, dev));
  }
  return run_attention(q, k, v, rel_h, rel_w, out, BH, H, W, head_dim, scale, in_dtype, bias_dtype, out_dtype, false,
                       workspace, workspace_bytes, stream, lse);
}

dera_status dera_relpos_attention_backward_workspace_size(int BH, int H, int W, int head_dim, size_t* bytes) {
  if (!bytes) return DERA_ERR_NULL;
  DERA_TRY(check_cb(BH, H, W, head_dim));
  *bytes = 0;
  if (BH == 0) return DERA_OK;
  int dev = 0;
  DERA_TRY(current_device(&dev));
  *bytes = CbLayout(BH, H, W, head_dim, sm_count(dev)).total;
  return DERA_OK;
}

dera_status dera_relpos_attention_backward(const void* q, const void* k, const void* v, const void* rel_h,
                                           const void* rel_w, const void* out, const float* lse, const void* dout,
                                           void* dq, void* dk, void* dv, float* drel_h, float* drel_w, int BH, int H,
                                           int W, int head_dim, float scale, dera_dtype in_dtype,
                                           dera_dtype bias_dtype, dera_dtype out_dtype, dera_dtype grad_dtype,
                                           void* workspace, size_t workspace_bytes, void* stream) {
  DERA_TRY(check_cb(BH, H, W, head_dim));
  if (!is16(in_dtype) || !is_float(bias_dtype) || !(out_dtype == DERA_F32 || out_dtype == in_dtype) ||
      !(grad_dtype == DERA_F32 || grad_dtype == in_dtype))
    return DERA_ERR_DTYPE;
  if (BH == 0) return DERA_OK;
  DERA_TRY(check_host({q, k, v, rel_h, rel_w, out, lse, dout, dq, dk, dv, drel_h, drel_w}));
  int dev = 0;
  DERA_TRY(current_device(&dev));
  for (const void* p : {q, k, v, rel_h, rel_w, out, static_cast<const void*>(lse), dout, static_cast<const void*>(dq),
                        static_cast<const void*>(dk), static_cast<const void*>(dv), static_cast<const void*>(drel_h),
                        static_cast<const void*>(drel_w)})
    DERA_TRY(check_ptr(p, dev));
  const CbLayout L(BH, H, W, head_dim, sm_count(dev));
  DERA_TRY(check_workspace(workspace, workspace_bytes, L.total, dev));
  const int N = H * W, WP = cb_width(W), KHT = WP <= 16 ? 4 : (WP <= 32 ? 2 : 1);
  CbMaps m;
  if (!map_rows(&m.q64, q, in_dtype, BH, N, head_dim, 64) || !map_rows(&m.dout64, dout, in_dtype, BH, N, head_dim, 64) ||
      !map_keys(&m.kg, k, in_dtype, BH, H, W, head_dim, WP, KHT) ||
      !map_keys(&m.vg, v, in_dtype, BH, H, W, head_dim, WP, KHT) ||
      !map_rows(&m.k, k, in_dtype, BH, N, head_dim) || !map_rows(&m.v, v, in_dtype, BH, N, head_dim))
    return DERA_ERR_CUDA;
  char* ws = static_cast<char*>(workspace);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  CbArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.rel_h = rel_h;
  a.rel_w = rel_w;
  a.lse = lse;
  a.out = out;
  a.dout = dout;
  a.hl = at(L.hl);
  a.rw = at(L.rw);
  a.nD = at(L.nD);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.drel_h = drel_h;
  a.drel_w = drel_w;
  a.parts_rows = at(L.parts_rows);
  a.parts_cols = at(L.parts_cols);
  a.status = status_ptr(dev);
  if (!a.status) return DERA_ERR_CUDA;
  a.BH = BH;
  a.H = H;
  a.W = W;
  a.N = N;
  a.n_tiles = L.n_tiles;
  a.n_blocks = 2 * L.n_tiles;
  a.rows_full = L.rows.full;
  a.rows_split = L.rows.split;
  a.cols_full = L.cols.full;
  a.cols_split = L.cols.split;
  a.scale = scale;
  a.scale_log2 = scale * kLog2e;
  a.out_fmt = fmt_of(out_dtype);
  a.grad_fmt = fmt_of(grad_dtype);
  a.bias_fmt = fmt_of(bias_dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = in_dtype == DERA_BF16;
  return (head_dim == 128 ? launch_cb_d128(m, a, bf16, s) : launch_cb_d64(m, a, bf16, s)) == cudaSuccess ? DERA_OK
                                                                                                       : DERA_ERR_CUDA;
}

dera_status dera_relpos_project_backward_workspace_size(int BH, int H, int W, int head_dim, size_t* bytes) {
  if (!bytes) return DERA_ERR_NULL;
  DERA_TRY(check_shape(BH, H, W, head_dim));
  *bytes = 0;
  if (BH == 0) return DERA_OK;
  int dev = 0;
  DERA_TRY(current_device(&dev));
  *bytes = pb_workspace(BH, H, W, head_dim, sm_count(dev));
  return DERA_OK;
}

dera_status dera_relpos_project_backward(const void* q, const void* rel_pos_h, const void* rel_pos_w,
                                         const float* drel_h, const float* drel_w, const void* dq_in, void* dq,
                                         float* drel_pos_h, float* drel_pos_w, int BH, int H, int W, int head_dim,
                                         dera_dtype in_dtype, dera_dtype grad_dtype, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  DERA_TRY(check_shape(BH, H, W, head_dim));
  if (!is16(in_dtype) || !(grad_dtype == DERA_F32 || grad_dtype == in_dtype)) return DERA_ERR_DTYPE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int dev = 0;
  if (BH == 0) {   // no rows: only the tables' gradients are written, as zeros
    DERA_TRY(check_host({drel_pos_h, drel_pos_w}));
    DERA_TRY(current_device(&dev));
    DERA_TRY(check_ptr(drel_pos_h, dev));
    DERA_TRY(check_ptr(drel_pos_w, dev));
    const size_t row = static_cast<size_t>(head_dim) * sizeof(float);
    if (cudaMemsetAsync(drel_pos_h, 0, (2 * H - 1) * row, s) != cudaSuccess ||
        cudaMemsetAsync(drel_pos_w, 0, (2 * W - 1) * row, s) != cudaSuccess)
      return DERA_ERR_CUDA;
    return DERA_OK;
  }
  DERA_TRY(check_host({q, rel_pos_h, rel_pos_w, drel_h, drel_w, dq, drel_pos_h, drel_pos_w}));
  if (dq_in) DERA_TRY(check_host({dq_in}));
  DERA_TRY(current_device(&dev));
  for (const void* p : {q, rel_pos_h, rel_pos_w, static_cast<const void*>(drel_h), static_cast<const void*>(drel_w),
                        dq_in, static_cast<const void*>(dq), static_cast<const void*>(drel_pos_h),
                        static_cast<const void*>(drel_pos_w)})
    if (p) DERA_TRY(check_ptr(p, dev));
  const int sms = sm_count(dev);
  DERA_TRY(check_workspace(workspace, workspace_bytes, pb_workspace(BH, H, W, head_dim, sms), dev));
  PbArgs a = {};
  a.q = q;
  a.th = rel_pos_h;
  a.tw = rel_pos_w;
  a.drel_h = drel_h;
  a.drel_w = drel_w;
  a.dq_in = dq_in;
  a.dq = dq;
  a.parts = static_cast<float*>(workspace);
  a.dth = drel_pos_h;
  a.dtw = drel_pos_w;
  a.status = status_ptr(dev);
  if (!a.status) return DERA_ERR_CUDA;
  a.H = H;
  a.W = W;
  a.N = H * W;
  a.D = head_dim;
  a.tokens = static_cast<long long>(BH) * a.N;
  a.n_tiles = (a.tokens + 127) / 128;
  a.grad_fmt = fmt_of(grad_dtype);
  return launch_project_backward(a, pb_ctas(BH, H, W, head_dim, sms), in_dtype == DERA_BF16, s) == cudaSuccess
             ? DERA_OK
             : DERA_ERR_CUDA;
}

}  // extern "C"
