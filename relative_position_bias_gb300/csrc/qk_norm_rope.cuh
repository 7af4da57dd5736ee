// Norms of queries and keys for each head and the rotation by position, forward
// and backward, with the move between token order and [B * heads, N, D].
//
// Per row x of D values (one token, one head):
//   y = x r w, r = 1 / sqrt(mean(x^2) + eps);  z = R(p) y
// and backward, with y' = R(p)^T dz and g = y' w:
//   dx = r (g - x r^2 mean(g x)),  dw = sum over rows of y' x r.
//
// Both are bound by memory: 2 bytes read and written per element, about ten
// operations.  A row is held by D / 8 lanes, eight elements (16 bytes) each, so a
// row's sums are shuffles and nothing passes through shared memory.  A thread
// keeps one (token, slot) and walks over heads: the angles and weights of its slot are
// loaded once and stay in registers.  Reads are whole rows of 128 or 256 bytes in
// token order, writes whole rows of consecutive tokens of a head.
//
// Measured: forward, 8 x 4096 tokens, 3 x 16 heads of 128, fp16, 806 MB: 123 us, 6.5 TB/s (a plain copy reaches
// 6.8).  Backward, 8 x 4096 tokens, 3 x 12 heads of 64, bf16, 404 MB: 76 us, 5.3 TB/s (705 MB in fp32 as the binding's
// defaults give them: 138 us with the weights' sums, 5.1 TB/s); it issues in 57 % of the cycles (two sums of eight lanes a
// row) and waits for loads in most others, those of its spilled registers among them.  The weights' sums
// are 4 us more (7 when their kernel was not launched ahead of this one's end).
#pragma once
#include <cstdint>

#include "common.cuh"
#include "train.cuh"

namespace dera {

// Sum over the D / 8 lanes of a row (in a fixed order, so every lane gets the same bits).
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
  #pragma unroll
  for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// mean(x^2) of a row.  The squares are taken of x / 16, so that the sum of a row of bf16 values
// overflows fp32 only where its mean square comes within 2^8 / D of doing so.
template <int D>
__device__ __forceinline__ float mean_square(const float (&v)[8]) {
  float s = 0.f;
  #pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = v[e] * 0.0625f;
    s = fmaf(t, t, s);
  }
  return row_sum<D / 8>(s) * (256.f / D);
}

// The angles of one thread's eight elements: z = y c + partner s (s is signed).
template <int D, int MODE>
struct Angles {
  float c[8], s[8];
  int partner;   // lane that holds the partners (kRotHalf)
  bool turned;   // this thread's elements are among the first rotary_dim; the others pass as they are

  __device__ __forceinline__ void load(const QkArgs& a, long long t, int n, int slot, int lane) {
    partner = lane;
    turned = false;
    if (MODE == kRotNone) return;
    const int e0 = slot * 8, half = a.half;
    if (e0 >= 2 * half) return;
    turned = true;
    const bool upper = MODE == kRotHalf && e0 >= half;
    if (MODE == kRotHalf) partner = lane + (upper ? -half / 8 : half / 8);
    const int p = a.positions ? a.positions[t] : n;
    const bool there = p >= 0 && p < a.table_rows;
    const size_t at = static_cast<size_t>(there ? p : 0) * half + (MODE == kRotHalf ? e0 - (upper ? half : 0) : e0 / 2);
    const float4* cp = reinterpret_cast<const float4*>(a.cos + at);
    const float4* sp = reinterpret_cast<const float4*>(a.sin + at);
    const float nan = __int_as_float(0x7fffffff);
    if (MODE == kRotHalf) {
      #pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 cv = __ldg(cp + h), sv = __ldg(sp + h);
        const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          c[4 * h + i] = there ? cc[i] : nan;
          s[4 * h + i] = upper ? ss[i] : -ss[i];
        }
      }
    } else {
      const float4 cv = __ldg(cp), sv = __ldg(sp);
      const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
      #pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[2 * i] = c[2 * i + 1] = there ? cc[i] : nan;
        s[2 * i] = -ss[i];
        s[2 * i + 1] = ss[i];
      }
    }
  }

  // x turned by the angle (sign 1) or back (sign -1)
  __device__ __forceinline__ void turn(float (&x)[8], float sign) const {
    if (MODE == kRotNone) return;
    float p[8];
    #pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = MODE == kRotHalf ? __shfl_sync(0xffffffffu, x[i], partner) : x[i ^ 1];
    if (!turned) return;   // not even by an angle of zero: 0 times an infinite neighbour is NaN
    #pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], c[i], sign * s[i] * p[i]);
  }
};

// Which tensor (q, k or v) and heads a block takes, from its y index.
struct QkBlock {
  int kind, h0, h1, y;   // y: the block's index among its tensor's
  __device__ __forceinline__ QkBlock(const QkArgs& a, int yy) {
    kind = 0;
    y = yy;
    while (kind < 2 && y >= a.groups[kind]) y -= a.groups[kind++];
    h0 = y * a.per;
    h1 = min(h0 + a.per, a.heads[kind]);
  }
};

template <bool BF16, int D, int MODE, bool NORM>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_kernel(const QkArgs a) {
  constexpr int LANES = D / 8, TOK = kQkThreads / LANES, U = 4;
  constexpr int fmt = BF16 ? kBF16 : kF16;
  const QkBlock blk(a, blockIdx.y);
  const int lane = threadIdx.x & 31, slot = threadIdx.x % LANES;
  const long long t0 = static_cast<long long>(blockIdx.x) * TOK + threadIdx.x / LANES;
  const bool valid = t0 < a.tokens;
  const long long t = valid ? t0 : a.tokens - 1;   // lanes past the end take part in the shuffles
  const long long b = t / a.N;
  const int n = static_cast<int>(t - b * a.N);
  const HeadsPtr x = a.x[blk.kind];
  const uint16_t* src = reinterpret_cast<const uint16_t*>(x.data) + b * x.sb + n * x.st + 8 * slot;
  uint16_t* dst = reinterpret_cast<uint16_t*>(a.zo[blk.kind]) +
                  (static_cast<size_t>(b) * a.heads[blk.kind] * a.N + n) * D + 8 * slot;
  const size_t hstep = static_cast<size_t>(a.N) * D;
  if (blk.kind == 2) {   // v is moved as it is
    for (int h = blk.h0; h < blk.h1; h += U) {
      uint4 u[U];
      #pragma unroll
      for (int i = 0; i < U; ++i)
        if (h + i < blk.h1) u[i] = __ldg(reinterpret_cast<const uint4*>(src + (h + i) * x.sh));
      #pragma unroll
      for (int i = 0; i < U; ++i)
        if (h + i < blk.h1 && valid) *reinterpret_cast<uint4*>(dst + (h + i) * hstep) = u[i];
    }
    return;
  }
  Angles<D, MODE> ang;
  ang.load(a, t, n, slot, lane);
  float w[8];
  #pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = NORM ? load_elem(a.w[blk.kind], 8 * slot + i, a.w_fmt) : 1.f;
  for (int h = blk.h0; h < blk.h1; h += U) {
    uint4 u[U];
    #pragma unroll
    for (int i = 0; i < U; ++i)   // U rows in flight; one past the group reads the last row again
      u[i] = __ldg(reinterpret_cast<const uint4*>(src + min(h + i, blk.h1 - 1) * x.sh));
    #pragma unroll
    for (int i = 0; i < U; ++i) {
      if (h + i >= blk.h1) break;
      float v[8];
      unpack8(u[i], v, fmt);
      if (NORM) {
        const float r = rsqrtf(mean_square<D>(v) + a.eps);
        #pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= r * w[e];
      }
      ang.turn(v, 1.f);
      if (valid) *reinterpret_cast<uint4*>(dst + (h + i) * hstep) = pack8(v, fmt);
    }
  }
}

// Eight values of a gradient as they lie: 16 bytes, or 32 in fp32.
template <bool F32>
struct Grad8 {
  uint4 u[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, size_t i) {
    const uint4* at = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (F32 ? 4 : 2));
    u[0] = __ldg(at);
    if (F32) u[F32 ? 1 : 0] = __ldg(at + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8], int fmt) const {
    if (F32) {
      const uint4 lo = u[0], hi = u[F32 ? 1 : 0];
      x[0] = __uint_as_float(lo.x), x[1] = __uint_as_float(lo.y), x[2] = __uint_as_float(lo.z), x[3] = __uint_as_float(lo.w);
      x[4] = __uint_as_float(hi.x), x[5] = __uint_as_float(hi.y), x[6] = __uint_as_float(hi.z), x[7] = __uint_as_float(hi.w);
    } else {
      unpack8(u[0], x, fmt);
    }
  }
};

// The weights' gradients are sums over every row of every token: a block takes
// every gridDim.x-th run of tokens and keeps its slots' sums in registers, one partial row
// per block, which qk_weight_grad_kernel adds in a fixed order.  Four rows in flight a thread and three blocks an
// SM: 76 us on the case above; three rows 93, two 95.  That leaves 80 registers a thread, which with a norm are too few
// (half split: 144 bytes of spill stores and 260 of loads, with fp32 gradients 224 and 460; interleaved 104 and 136).
template <bool BF16, int D, int MODE, bool NORM, bool ZF32>
__global__ void __launch_bounds__(kQkThreads, 3) qk_norm_rope_bwd_kernel(const QkArgs a) {
  constexpr int LANES = D / 8, TOK = kQkThreads / LANES, WARPS = kQkThreads / 32, U = 4;
  constexpr int fmt = BF16 ? kBF16 : kF16;
  grid_launch_dependents();   // qk_weight_grad_kernel starts as these blocks run out
  __shared__ float red[WARPS][D];
  const QkBlock blk(a, blockIdx.y);
  const int lane = threadIdx.x & 31, slot = threadIdx.x % LANES;
  const HeadsPtr x = a.x[blk.kind], dx = a.dx[blk.kind];
  const int heads = a.heads[blk.kind];
  const bool v_rows = blk.kind == 2;   // v's gradient is moved as it is
  float w[8], dw[8];
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = (NORM && !v_rows) ? load_elem(a.w[blk.kind], 8 * slot + i, a.w_fmt) : 1.f;
    dw[i] = 0.f;
  }
  const long long step = static_cast<long long>(gridDim.x) * TOK;
  for (long long tb = static_cast<long long>(blockIdx.x) * TOK; tb < a.tokens; tb += step) {
    const long long t0 = tb + threadIdx.x / LANES;
    const bool valid = t0 < a.tokens;
    const long long t = valid ? t0 : a.tokens - 1;
    const long long b = t / a.N;
    const int n = static_cast<int>(t - b * a.N);
    const size_t zrow = (static_cast<size_t>(b) * heads * a.N + n) * D + 8 * slot;
    const size_t hstep = static_cast<size_t>(a.N) * D;
    const uint16_t* xrow = reinterpret_cast<const uint16_t*>(x.data) + b * x.sb + n * x.st + 8 * slot;
    const long long dxrow = b * dx.sb + n * dx.st + 8 * slot;
    Angles<D, MODE> ang;
    if (!v_rows) ang.load(a, t, n, slot, lane);
    for (int h = blk.h0; h < blk.h1; h += U) {
      Grad8<ZF32> z[U];
      uint4 xv[U];
      #pragma unroll
      for (int i = 0; i < U; ++i) {   // U rows in flight; one past the group reads the last row again
        const int hh = min(h + i, blk.h1 - 1);
        z[i].load(a.z[blk.kind], zrow + hh * hstep);
        if (NORM && !v_rows) xv[i] = __ldg(reinterpret_cast<const uint4*>(xrow + hh * x.sh));
      }
      #pragma unroll
      for (int i = 0; i < U; ++i) {
        if (h + i >= blk.h1) break;
        float g[8];
        z[i].get(g, fmt);
        if (!v_rows) {
          ang.turn(g, -1.f);
          if (NORM) {
            float v[8];
            unpack8(xv[i], v, fmt);
            float gx = 0.f;
            #pragma unroll
            for (int e = 0; e < 8; ++e) gx = fmaf(g[e] * w[e], v[e], gx);
            const float r = rsqrtf(mean_square<D>(v) + a.eps);
            const float m = row_sum<LANES>(gx) * (1.f / D) * r * r;
            #pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (valid) dw[e] = fmaf(g[e], v[e] * r, dw[e]);
              g[e] = r * fmaf(-m, v[e], g[e] * w[e]);
            }
          }
        }
        if (valid) store8(dx.data, dxrow + (h + i) * dx.sh, g, a.dx_fmt == kF32 ? kF32 : fmt);
      }
    }
  }
  if (!NORM || v_rows) return;
  #pragma unroll
  for (int e = 0; e < 8; ++e) {
    #pragma unroll
    for (int o = LANES; o < 32; o <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], o);
    if (lane < LANES) red[threadIdx.x >> 5][8 * slot + e] = dw[e];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float v = 0.f;
    #pragma unroll
    for (int i = 0; i < WARPS; ++i) v += red[i][threadIdx.x];
    const size_t row = (blk.kind == 1 ? static_cast<size_t>(a.groups[0]) * gridDim.x : 0) +
                       static_cast<size_t>(blk.y) * gridDim.x + blockIdx.x;
    a.parts[row * D + threadIdx.x] = v;
  }
}

// dst[kind][c] = the sum of the kind's partial rows in a fixed order: thread (c, i)
// adds rows i, i + 32, ..., then the 32 sums are added one after another.
__global__ void __launch_bounds__(1024) qk_weight_grad_kernel(const float* parts, int rows_q, int rows_k, int D,
                                                             float* dqw, float* dkw) {
  __shared__ float red[32][33];
  grid_wait_prerequisites();   // every partial row is written
  const bool is_k = blockIdx.y == 1;
  const float* p = parts + (is_k ? static_cast<size_t>(rows_q) * D : 0) + blockIdx.x * 32 + threadIdx.x;
  const int rows = is_k ? rows_k : rows_q;
  float v = 0.f;
  #pragma unroll 8
  for (int r = threadIdx.y; r < rows; r += 32) v += p[static_cast<size_t>(r) * D];
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0) {
    float s = 0.f;
    #pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    (is_k ? dkw : dqw)[blockIdx.x * 32 + threadIdx.x] = s;
  }
}

}  // namespace dera
