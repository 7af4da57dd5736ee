// Layer norm of rows of C values, forward and backward.
//
//   forward   m = sum x / C,  r = 1 / sqrt(sum (x - m)^2 / C + eps),  h = (x - m) r,  y = h w + b
//   backward  g = dy w,  dx = r (g - sum g / C - h sum(g h) / C) + dres,  dw = sum over rows of dy h,  db = of dy
//
// Both should be bound by memory: every element is read and written once, for about 8 and 16 operations.  At 6.8 TB/s an
// SM has 22 to 31 bytes a clock (2.07 to 1.46 GHz), so 17 to 24 issue slots for 32 elements of a 16-bit row read and written, and
// instructions count, too:
// arithmetic is on packed pairs, addresses advance by additions, and a row's sums are joined by few shuffles.
//
// A row lies over `tpr` threads (whole warps, as many as C needs), NV times eight neighbouring elements each, so that a thread
// keeps its columns' weights, and in the backward their sums, in registers over all rows of its block.  A block holds as many
// rows side by side as fit 256 threads; bulk copies bring whole rows into a ring in shared memory several sets ahead (loads
// into registers do not reach far enough: 4.4 TB/s), and one barrier serves a set's sums and frees its place in the ring.  Rows that
// are not whole 16-byte chunks are read directly.  The weights' gradients are partial rows, one a block, that partial_rows_kernel
// adds in a fixed order.
//
// Measured: forward, 32768 x 2048 fp16, 268 MB: 51.6 us, 5.2 TB/s (a plain copy reaches 6.8); 32768 x 1024 bf16 25 us.  Backward with
// the residual's gradient, 32768 x 1024: fp32 stream, 470 MB, 74.7 us, 6.3 TB/s; bf16, 268 MB, 49 us, 5.4 TB/s; the weights' sums
// are 4 to 5 us of each.  Rows of an odd number of columns, element by element: 32768 x 1001 bf16 61 us, backward 108.
#pragma once
#include "activation.cuh"
#include "block.cuh"
#include "common.cuh"

namespace dera {

// Element of thread t's eight: neighbours where rows are whole 16-byte chunks, else every tpr-th.
template <bool VEC>
__device__ __forceinline__ int ln_col(int i, int e, int t, int tpr) {
  return VEC ? (i * tpr + t) * 8 + e : (i * 8 + e) * tpr + t;
}

// Eight elements of a row as they lie, 0 past its end, or (`repeat`) its last ones again.  FMT < 0: the type at run time.
template <int FMT, bool VEC>
struct LnRaw {
  uint4 lo, hi;   // hi: the second half of fp32's
  __device__ __forceinline__ void load(const char* row, int i, int t, int tpr, int C, bool there, int fmt, bool repeat = false) {
    const int f = FMT >= 0 ? FMT : fmt, at = ln_col<VEC>(i, 0, t, tpr), c = repeat ? min(at, C - 8) : at;
    lo = hi = make_uint4(0u, 0u, 0u, 0u);
    if (!there || c >= C) return;
    const uint4* q = reinterpret_cast<const uint4*>(row + static_cast<size_t>(c) * (f == kF32 ? 4 : 2));
    lo = *q;
    if (f == kF32) hi = q[1];
  }
  __device__ __forceinline__ void get(float2 (&v)[4], int fmt) const {
    const int f = FMT >= 0 ? FMT : fmt;
    if (f == kF32) {
      v[0] = make_float2(__uint_as_float(lo.x), __uint_as_float(lo.y));
      v[1] = make_float2(__uint_as_float(lo.z), __uint_as_float(lo.w));
      v[2] = make_float2(__uint_as_float(hi.x), __uint_as_float(hi.y));
      v[3] = make_float2(__uint_as_float(hi.z), __uint_as_float(hi.w));
    } else {
      v[0] = unpack_in(lo.x, f);
      v[1] = unpack_in(lo.y, f);
      v[2] = unpack_in(lo.z, f);
      v[3] = unpack_in(lo.w, f);
    }
  }
};
template <int FMT>
struct LnRaw<FMT, false> {
  float x[8];
  __device__ __forceinline__ void load(const char* row, int i, int t, int tpr, int C, bool there, int fmt, bool repeat = false) {
    #pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int at = ln_col<false>(i, e, t, tpr), c = repeat ? min(at, C - 1) : at;
      x[e] = there && c < C ? load_elem(row, c, FMT >= 0 ? FMT : fmt) : 0.f;
    }
  }
  __device__ __forceinline__ void get(float2 (&v)[4], int) const {
    #pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = make_float2(x[2 * e], x[2 * e + 1]);
  }
};

template <bool VEC>
__device__ __forceinline__ void ln_store(char* row, int i, int t, int tpr, int C, int fmt, const float2 (&v)[4]) {
  const float x[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
  if (VEC) {
    const int c = ln_col<VEC>(i, 0, t, tpr);
    if (c < C) store8(row, c, x, fmt);
  } else {
    #pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = ln_col<VEC>(i, e, t, tpr);
      if (c >= C) continue;
      if (fmt == kF32) reinterpret_cast<float*>(row)[c] = x[e];
      else reinterpret_cast<uint16_t*>(row)[c] = static_cast<uint16_t>(pack_in(x[e], 0.f, fmt));
    }
  }
}

// A parameter's columns of a thread (`none` where there is none, 0 past the row's end).
template <bool VEC, int NV>
__device__ __forceinline__ void ln_params(const void* p, float none, int t, int tpr, int C, int fmt, float2 (&w)[NV][4]) {
  #pragma unroll
  for (int i = 0; i < NV; ++i) {
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = ln_col<VEC>(i, 2 * e, t, tpr), c1 = ln_col<VEC>(i, 2 * e + 1, t, tpr);
      w[i][e].x = p && c < C ? load_elem(p, c, fmt) : none;
      w[i][e].y = p && c1 < C ? load_elem(p, c1, fmt) : none;
    }
  }
}

// A ring of sets of rows in shared memory: of each of up to three tensors, the block's G rows one after another.
struct LnRing {
  uint64_t* full;   // [sets]
  char* data;
  volatile int* abort_flag;
  int* status;
  int sets, bytes;  // of a set
  int at;           // the set that is read
  uint32_t phase;
  __device__ __forceinline__ void init(const LnArgs& a, char* smem, int G, int row_bytes) {
    full = reinterpret_cast<uint64_t*>(smem);
    abort_flag = reinterpret_cast<volatile int*>(smem + 64);
    data = smem + 128;
    status = a.status;
    sets = a.sets;
    bytes = G * row_bytes;
    at = 0;
    phase = 0;
    if (threadIdx.x == 0) {
      *abort_flag = 0;
      for (int i = 0; i < sets; ++i) mbar_init(&full[i], 1);
      fence_mbar_init();
    }
    __syncthreads();
  }
  // `rows` rows of `row` bytes, `stride` apart, to byte `to` of set i
  __device__ __forceinline__ void copy(int i, int to, const char* src, long long stride, int row, int rows) {
    char* dst = data + i * bytes + to;
    if (stride == row) {
      bulk_load(dst, src, row * rows, &full[i]);
    } else {
      for (int k = 0; k < rows; ++k) bulk_load(dst + k * row, src + k * stride, row, &full[i]);
    }
  }
  // If a copy does not come in time the status word says so; what is computed then is of no use, but every thread goes on.
  __device__ __forceinline__ void wait() { mbar_wait(&full[at], phase, abort_flag, status); }
  __device__ __forceinline__ void next() {
    if (++at == sets) {
      at = 0;
      phase ^= 1;
    }
  }
  // If a wait gave up: copies still in flight land before the block leaves (with a limit).
  __device__ __forceinline__ void drain() {
    if (threadIdx.x != 0 || !*abort_flag) return;
    for (int i = 0; i < sets; ++i) mbar_wait_budget(&full[i], i >= at ? phase : phase ^ 1, kWaitBudgetCycles);
  }
};
constexpr int kLnRingHead = 128;

// Where a row's warps join what each has: `warps` of them from `first` on, padded to a power of two, so that a warp takes
// several values at a time, one a group of lanes.
struct LnJoin {
  int first, warps, width, lane;
  __device__ __forceinline__ LnJoin(int tpr) {
    warps = tpr >> 5;
    first = (threadIdx.x >> 5) / warps * warps;
    width = warps <= 1 ? 1 : 1 << (32 - __clz(warps - 1));
    lane = threadIdx.x & 31;
  }
  __device__ __forceinline__ float sum(float x) const {
    for (int o = 1; o < width; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  }
};

__device__ __forceinline__ float ln_warp_sum(float s) {
  #pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
__device__ __forceinline__ float2 ln_pair(float x) { return make_float2(x, x); }

// Forward.  The statistics of a warp's columns are found in registers, mean first, then the squares about it; the warps of
// a row join theirs with one barrier:  M2 = sum M2_w + n_w (m_w - m)^2, a sum of squares again: no cancellation whatever
// the mean is.
template <int XF, int MAXT, int NV, bool VEC>
__global__ void __launch_bounds__(MAXT) layer_norm_kernel(const LnArgs a) {
  __shared__ float2 red[2][32];
  __shared__ float columns[32];   // of each warp
  extern __shared__ __align__(128) char ring_smem[];
  const int g = threadIdx.x / a.tpr, t = threadIdx.x - g * a.tpr, G = blockDim.x / a.tpr, C = a.C;
  const LnJoin j(a.tpr);
  const int warp = threadIdx.x >> 5;
  const int xe = a.x_fmt == kF32 ? 4 : 2, ye = a.y_fmt == kF32 ? 4 : 2;
  const long long step = static_cast<long long>(gridDim.x) * G;
  long long r0 = static_cast<long long>(blockIdx.x) * G;   // the block's first row, r this thread's
  LnRing ring;
  auto fetch = [&](int set, long long first) {   // by one thread
    if (first >= a.rows) return;
    const int n = static_cast<int>(min(static_cast<long long>(G), a.rows - first));
    mbar_arrive_expect_tx(&ring.full[set], n * C * xe);
    ring.copy(set, 0, static_cast<const char*>(a.x) + first * a.xs * xe, a.xs * xe, C * xe, n);
  };
  if (VEC) {
    ring.init(a, ring_smem, G, C * xe);
    if (threadIdx.x == 0)
      for (int i = 0; i < ring.sets; ++i) fetch(i, r0 + i * step);
  }
  float2 w[NV][4], b[NV][4];
  ln_params<VEC>(a.w, 1.f, t, a.tpr, C, a.w_fmt, w);
  ln_params<VEC>(a.b, 0.f, t, a.tpr, C, a.w_fmt, b);
  int own = 0;   // this thread's columns
  #pragma unroll
  for (int i = 0; i < NV; ++i) {
    #pragma unroll
    for (int e = 0; e < 8; ++e) own += ln_col<VEC>(i, e, t, a.tpr) < C;
  }
  const float n_warp = static_cast<float>(__reduce_add_sync(0xffffffffu, own));   // this warp's columns of a row
  const float inv_warp = n_warp > 0.f ? 1.f / n_warp : 0.f, inv = 1.f / C;
  if (j.lane == 0) columns[warp] = n_warp;
  long long r = r0 + g;
  const char* xp = static_cast<const char*>(a.x) + r * a.xs * xe;
  char* yp = static_cast<char*>(a.y) + r * C * ye;
  const long long x_step = step * a.xs * xe, y_step = step * C * ye;
  for (int buf = 0; r0 < a.rows; r0 += step, r += step, xp += x_step, yp += y_step, buf ^= 1) {
    if (VEC) {
      ring.wait();
      xp = ring.data + ring.at * ring.bytes + g * C * xe;
    }
    LnRaw<XF, VEC> raw[NV];
    #pragma unroll
    for (int i = 0; i < NV; ++i) raw[i].load(xp, i, t, a.tpr, C, r < a.rows, a.x_fmt);
    float2 v[NV][4], s2 = ln_pair(0.f);
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      raw[i].get(v[i], a.x_fmt);
      #pragma unroll
      for (int e = 0; e < 4; ++e) s2 = fadd2(s2, v[i][e]);
    }
    const float mw = ln_warp_sum(s2.x + s2.y) * inv_warp;
    float q = 0.f;
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      float2 p = ln_pair(0.f);
      #pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[i][e] = fadd2(v[i][e], ln_pair(-mw));
        float2 d = v[i][e];
        if (!VEC) {
          if (ln_col<VEC>(i, 2 * e, t, a.tpr) >= C) d.x = 0.f;
          if (ln_col<VEC>(i, 2 * e + 1, t, a.tpr) >= C) d.y = 0.f;
        }
        p = ffma2(d, d, p);
      }
      if (!VEC || ln_col<VEC>(i, 0, t, a.tpr) < C) q += p.x + p.y;
    }
    q = ln_warp_sum(q);
    if (j.lane == 0) red[buf][warp] = make_float2(mw, q);
    if (VEC || j.warps > 1) __syncthreads();
    if (VEC) {   // every thread has its part of the set
      if (threadIdx.x == 0) fetch(ring.at, r0 + ring.sets * step);
      ring.next();
    }
    float mean = mw, m2 = q;
    if (j.warps > 1) {
      const int k = j.lane & (j.width - 1);
      const float2 p = k < j.warps ? red[buf][j.first + k] : make_float2(0.f, 0.f);
      const float n = k < j.warps ? columns[j.first + k] : 0.f;
      mean = j.sum(n * p.x) * inv;
      m2 = j.sum(fmaf(n * (p.x - mean), p.x - mean, p.y));
    }
    if (r < a.rows) {
      const float rs = rsqrtf(fmaf(m2, inv, a.eps));
      const float2 off = ln_pair(mw - mean), rr = ln_pair(rs);
      #pragma unroll
      for (int i = 0; i < NV; ++i) {
        #pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = ffma2(fmul2(fadd2(v[i][e], off), rr), w[i][e], b[i][e]);
        ln_store<VEC>(yp, i, t, a.tpr, C, a.y_fmt, v[i]);
      }
      if (t == 0) {
        a.mean[r] = mean;
        a.rstd[r] = rs;
      }
    }
  }
  if (VEC) ring.drain();
}

// Forward for rows of up to 2048 columns, a row a warp: its sums are shuffles alone, and what a row costs apart from its
// elements (waits, shuffles, addresses: about 100 instructions) is paid by one warp instead of four.  32768 x 1024, bf16: 43 us with four
// warps a row, 25 with one.  Every warp has a ring of its own; the parameters lie in shared memory as fp32, the first and the
// last four of every eight apart, so that lanes read neighbouring 16-byte chunks.
constexpr int ln_warp_blocks(int nv) { return nv <= 4 ? 3 : 2; }   // of an SM
template <int XF, int NV>
__global__ void __launch_bounds__(256, ln_warp_blocks(NV)) layer_norm_warp_kernel(const LnArgs a) {
  extern __shared__ __align__(128) char ring_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, C = a.C, xe = XF == kF32 ? 4 : 2, ye = a.y_fmt == kF32 ? 4 : 2;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring_smem) + 8 * warp;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ring_smem + 512);
  float4* params = reinterpret_cast<float4*>(ring_smem + 640);   // [weight lo, weight hi, bias lo, bias hi][C / 8]
  const int row_bytes = C * xe, chunks = C / 8;
  char* ring = ring_smem + 640 + (a.w ? 2 * (a.b ? 2 : 1) * chunks * 16 : 0);
  ring += warp * a.sets * row_bytes;
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < 64; ++i) mbar_init(reinterpret_cast<uint64_t*>(ring_smem) + i, 1);
    fence_mbar_init();
  }
  for (int k = threadIdx.x; k < chunks; k += 256) {
    float v[8];
    if (a.w) {
      for (int e = 0; e < 8; ++e) v[e] = load_elem(a.w, 8 * k + e, a.w_fmt);
      params[k] = make_float4(v[0], v[1], v[2], v[3]);
      params[chunks + k] = make_float4(v[4], v[5], v[6], v[7]);
    }
    if (a.b) {
      for (int e = 0; e < 8; ++e) v[e] = load_elem(a.b, 8 * k + e, a.w_fmt);
      params[2 * chunks + k] = make_float4(v[0], v[1], v[2], v[3]);
      params[3 * chunks + k] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
  __syncthreads();
  const long long step = static_cast<long long>(gridDim.x) * 8, x_step = step * a.xs * xe, y_step = step * C * ye;
  long long r = static_cast<long long>(blockIdx.x) * 8 + warp, ahead = r;   // ahead: the next row to be fetched
  const char* src = static_cast<const char*>(a.x) + r * a.xs * xe;
  char* yp = static_cast<char*>(a.y) + r * C * ye;
  auto fetch = [&](int set) {
    if (ahead < a.rows && lane == 0) {
      mbar_arrive_expect_tx(&full[set], row_bytes);
      bulk_load(ring + set * row_bytes, src, row_bytes, &full[set]);
    }
    ahead += step;
    src += x_step;
  };
  for (int i = 0; i < a.sets; ++i) fetch(i);
  const float inv = 1.f / C;
  int at = 0;
  uint32_t phase = 0;
  for (; r < a.rows; r += step, yp += y_step) {
    mbar_wait(&full[at], phase, abort_flag, a.status);   // out of time: the status word says so, what follows is of no use
    float2 v[NV][4], s2 = ln_pair(0.f);
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      LnRaw<XF, true> raw;
      raw.load(ring + at * row_bytes, i, lane, 32, C, true, XF);
      raw.get(v[i], XF);
      #pragma unroll
      for (int e = 0; e < 4; ++e) s2 = fadd2(s2, v[i][e]);
    }
    __syncwarp();   // the row is in registers
    fetch(at);
    if (++at == a.sets) {
      at = 0;
      phase ^= 1;
    }
    const float mean = ln_warp_sum(s2.x + s2.y) * inv;
    const float2 off = ln_pair(-mean);
    float2 q = ln_pair(0.f);
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      #pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = fadd2(v[i][e], off);
      if (i * 32 + lane < chunks) {
        #pragma unroll
        for (int e = 0; e < 4; ++e) q = ffma2(v[i][e], v[i][e], q);
      }
    }
    const float rs = rsqrtf(fmaf(ln_warp_sum(q.x + q.y), inv, a.eps));
    const float2 rr = ln_pair(rs);
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = i * 32 + lane;
      if (k >= chunks) continue;
      #pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = fmul2(v[i][e], rr);
      if (a.w) {
        const float4 lo = params[k], hi = params[chunks + k];
        float4 blo = make_float4(0.f, 0.f, 0.f, 0.f), bhi = blo;
        if (a.b) blo = params[2 * chunks + k], bhi = params[3 * chunks + k];
        v[i][0] = ffma2(v[i][0], make_float2(lo.x, lo.y), make_float2(blo.x, blo.y));
        v[i][1] = ffma2(v[i][1], make_float2(lo.z, lo.w), make_float2(blo.z, blo.w));
        v[i][2] = ffma2(v[i][2], make_float2(hi.x, hi.y), make_float2(bhi.x, bhi.y));
        v[i][3] = ffma2(v[i][3], make_float2(hi.z, hi.w), make_float2(bhi.z, bhi.w));
      }
      ln_store<true>(yp, i, lane, 32, C, a.y_fmt, v[i]);
    }
    if (lane == 0) {
      a.mean[r] = mean;
      a.rstd[r] = rs;
    }
  }
  if (*abort_flag && lane == 0)   // copies still in flight land before the block leaves (with a limit)
    for (int i = 0; i < a.sets; ++i) mbar_wait_budget(&full[i], i >= at ? phase : phase ^ 1, kWaitBudgetCycles);
}

// Backward.  The two sums of a row go through the shuffles as one: after the first step even lanes hold the one, odd lanes
// the other.
template <int XF, int ZF, int MAXT, int NV, bool VEC, int BLOCKS>
__global__ void __launch_bounds__(MAXT, BLOCKS) layer_norm_bwd_kernel(const LnArgs a) {
  __shared__ float red[2][2][32];
  extern __shared__ __align__(128) char ring_smem[];   // and after the rows [2][G][C] sums
  grid_launch_dependents();         // partial_rows_kernel starts as these blocks run out
  const int g = threadIdx.x / a.tpr, t = threadIdx.x - g * a.tpr, G = blockDim.x / a.tpr, C = a.C;
  const LnJoin j(a.tpr);
  const long long step = static_cast<long long>(gridDim.x) * G;
  const int xe = a.x_fmt == kF32 ? 4 : 2, ze = a.y_fmt == kF32 ? 4 : 2, de = a.dx_fmt == kF32 ? 4 : 2;
  const bool dres = a.dres != nullptr;
  long long r0 = static_cast<long long>(blockIdx.x) * G;   // the block's first row, r this thread's
  LnRing ring;
  auto fetch = [&](int set, long long first) {   // by one thread
    if (first >= a.rows) return;
    const int n = static_cast<int>(min(static_cast<long long>(G), a.rows - first));
    mbar_arrive_expect_tx(&ring.full[set], n * C * (xe + ze + (dres ? de : 0)));
    ring.copy(set, 0, static_cast<const char*>(a.x) + first * a.xs * xe, a.xs * xe, C * xe, n);
    ring.copy(set, G * C * xe, static_cast<const char*>(a.dy) + first * C * ze, C * ze, C * ze, n);
    if (dres) ring.copy(set, G * C * (xe + ze), static_cast<const char*>(a.dres) + first * C * de, C * de, C * de, n);
  };
  if (VEC) {
    ring.init(a, ring_smem, G, C * (xe + ze + (dres ? de : 0)));
    if (threadIdx.x == 0)
      for (int i = 0; i < ring.sets; ++i) fetch(i, r0 + i * step);
  }
  float2 w[NV][4], dw[NV][4], db[NV][4];
  ln_params<VEC>(a.w, 1.f, t, a.tpr, C, a.w_fmt, w);
  #pragma unroll
  for (int i = 0; i < NV; ++i) {
    #pragma unroll
    for (int e = 0; e < 4; ++e) dw[i][e] = db[i][e] = ln_pair(0.f);
  }
  const float inv = 1.f / C;
  long long r = r0 + g;
  const char* xp = static_cast<const char*>(a.x) + r * a.xs * xe;
  const char* zp = static_cast<const char*>(a.dy) + r * C * ze;
  const long long x_step = step * a.xs * xe, z_step = step * C * ze, d_step = step * C * de;
  long long d_at = r * C * de;
  float mu = r < a.rows ? a.mean_in[r] : 0.f, rs = r < a.rows ? a.rstd_in[r] : 0.f;
  for (int buf = 0; r0 < a.rows; r0 += step, r += step, xp += x_step, zp += z_step, d_at += d_step, buf ^= 1) {
    const char* dp = static_cast<const char*>(a.dres) + d_at;
    if (VEC) {
      ring.wait();
      char* set = ring.data + ring.at * ring.bytes;
      xp = set + g * C * xe;
      zp = set + G * C * xe + g * C * ze;
      dp = set + G * C * (xe + ze) + g * C * de;
    }
    LnRaw<XF, VEC> x[NV];
    LnRaw<ZF, VEC> z[NV];
    LnRaw<-1, VEC> d[NV];
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      // past the row's end an x of the row, not 0: (0 - mean) rstd may be an infinity where no h of the row is, and 0 times it would
      // reach the sums
      x[i].load(xp, i, t, a.tpr, C, r < a.rows, a.x_fmt, true);
      z[i].load(zp, i, t, a.tpr, C, r < a.rows, a.y_fmt);
      d[i].load(dp, i, t, a.tpr, C, r < a.rows && dres, a.dx_fmt);
    }
    float2 h[NV][4], q[NV][4], f[NV][4], s1 = ln_pair(0.f), s2 = ln_pair(0.f);
    const float2 r1 = ln_pair(rs), m0 = ln_pair(-mu);
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i].get(h[i], a.x_fmt);
      z[i].get(q[i], a.y_fmt);
      d[i].get(f[i], a.dx_fmt);
      #pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[i][e] = fmul2(fadd2(h[i][e], m0), r1);
        db[i][e] = fadd2(db[i][e], q[i][e]);
        dw[i][e] = ffma2(q[i][e], h[i][e], dw[i][e]);
        q[i][e] = fmul2(q[i][e], w[i][e]);   // 0 past the row's end
        s1 = fadd2(s1, q[i][e]);
        s2 = ffma2(q[i][e], h[i][e], s2);
      }
    }
    if (r + step < a.rows) {   // the next row's statistics are on their way
      mu = a.mean_in[r + step];
      rs = a.rstd_in[r + step];
    } else {
      mu = rs = 0.f;
    }
    const float t1 = s1.x + s1.y, t2 = s2.x + s2.y;
    const bool odd = j.lane & 1;
    float s = (odd ? t2 : t1) + __shfl_xor_sync(0xffffffffu, odd ? t1 : t2, 1);
    #pragma unroll
    for (int o = 2; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (j.lane < 2) red[buf][j.lane][threadIdx.x >> 5] = s;
    if (VEC || j.warps > 1) __syncthreads();
    if (VEC) {   // every thread has its part of the set
      if (threadIdx.x == 0) fetch(ring.at, r0 + ring.sets * step);
      ring.next();
    }
    if (j.warps > 1) {
      const int k = j.lane & (j.width - 1);
      const bool there = k < j.warps;
      if (j.width <= 16) {   // both at once, each in half of the warp
        s = j.sum(there ? red[buf][j.lane >> 4][j.first + k] : 0.f);
      } else {
        const float p1 = j.sum(there ? red[buf][0][j.first + k] : 0.f), p2 = j.sum(there ? red[buf][1][j.first + k] : 0.f);
        s = j.lane < 16 ? p1 : p2;
      }
    }
    const int second = j.warps > 1 ? 16 : 1;
    const float2 m1 = ln_pair(-inv * __shfl_sync(0xffffffffu, s, 0)), m2 = ln_pair(-inv * __shfl_sync(0xffffffffu, s, second));
    if (r < a.rows) {
      #pragma unroll
      for (int i = 0; i < NV; ++i) {
        #pragma unroll
        for (int e = 0; e < 4; ++e) f[i][e] = ffma2(r1, fadd2(ffma2(m2, h[i][e], q[i][e]), m1), f[i][e]);
        ln_store<VEC>(static_cast<char*>(a.dx) + d_at, i, t, a.tpr, C, a.dx_fmt, f[i]);
      }
    }
  }
  if (VEC) ring.drain();
  if (!a.parts) return;
  // The block's G rows of sums, by column, then one partial row of 2 C floats.
  float* out = a.parts + static_cast<size_t>(blockIdx.x) * 2 * C;
  float* sums = reinterpret_cast<float*>(ring_smem + kLnRingHead);
  if (G > 1) __syncthreads();   // the ring has been read
  #pragma unroll
  for (int p = 0; p < 2; ++p) {
    float* to = G > 1 ? sums + (p * G + g) * C : out + p * C;
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float2(&v)[4] = p == 0 ? dw[i] : db[i];
      ln_store<VEC>(reinterpret_cast<char*>(to), i, t, a.tpr, C, kF32, v);
    }
  }
  if (G == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * C; c += blockDim.x) {
    const float* from = sums + (c < C ? c : (G - 1) * C + c);
    float v = from[0];
    for (int k = 1; k < G; ++k) v += from[k * C];
    out[c] = v;
  }
}

// dst[c] = the sum of column c of `rows` partial rows of n columns in a fixed order: thread (c, i) adds rows i, i + 32, ...,
// then the 32 sums are added one after another.  The first n1 columns go to d1, the others to d2.
__global__ void __launch_bounds__(1024) partial_rows_kernel(const float* parts, int rows, int n, int n1, float* d1, float* d2) {
  __shared__ float red[32][33];
  grid_wait_prerequisites();   // every partial row is written
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < n) {
    #pragma unroll 8
    for (int r = threadIdx.y; r < rows; r += 32) v += parts[static_cast<size_t>(r) * n + c];
  }
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < n) {
    float s = 0.f;
    #pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    if (c < n1) d1[c] = s;
    else d2[c - n1] = s;
  }
}

}  // namespace dera
