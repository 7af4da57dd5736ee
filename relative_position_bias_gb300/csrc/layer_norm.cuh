// Layer norm of rows of C values, forward and backward.
//
//   forward   m = sum x / C,  r = 1 / sqrt(sum (x - m)^2 / C + eps),  h = (x - m) r,  y = h w + b
//   backward  g = dy w,  dx = r (g - sum g / C - h sum(g h) / C) + dres,  dw = sum over rows of dy h,  db = of dy
//
// Both are bound by memory: every element is read and written once, for about 8 and 16 operations.  A row lies over
// `tpr` threads (whole warps, as many as C needs), eight neighbouring elements each, so that a thread keeps its columns'
// weights, and in the backward their sums, in registers over all rows of its block.  A block holds as many rows side by
// side as fit 256 threads and U of those sets at once: their loads are in flight together, and one barrier serves the sums of all.
// The variance is summed from centred values, a second pass over registers: no cancellation whatever the mean is.
// The weights' gradients are partial rows, one a block, that partial_rows_kernel adds in a fixed order.
#pragma once
#include "block.cuh"
#include "common.cuh"

namespace dera {

// Element of thread t's eight: neighbours where rows are whole 16-byte chunks, else every tpr-th.
template <bool VEC>
__device__ __forceinline__ int ln_col(int i, int e, int t, int tpr) {
  return VEC ? (i * tpr + t) * 8 + e : (i * 8 + e) * tpr + t;
}

// Eight elements of a row; 0 past its end.  FMT < 0: the type at run time.
template <int FMT, bool VEC>
__device__ __forceinline__ void ln_load(const void* p, size_t row, int i, int t, int tpr, int C, int fmt, float (&v)[8]) {
  const int f = FMT >= 0 ? FMT : fmt;
  if (VEC) {
    const int c = ln_col<VEC>(i, 0, t, tpr);
    #pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
    if (c < C) load8(p, row + c, v, f);
  } else {
    #pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = ln_col<VEC>(i, e, t, tpr);
      v[e] = c < C ? load_elem(p, row + c, f) : 0.f;
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void ln_store(void* p, size_t row, int i, int t, int tpr, int C, int fmt, const float (&v)[8]) {
  if (VEC) {
    const int c = ln_col<VEC>(i, 0, t, tpr);
    if (c < C) store8(p, row + c, v, fmt);
  } else {
    #pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = ln_col<VEC>(i, e, t, tpr);
      if (c >= C) continue;
      if (fmt == kF32) reinterpret_cast<float*>(p)[row + c] = v[e];
      else reinterpret_cast<uint16_t*>(p)[row + c] = static_cast<uint16_t>(pack_in(v[e], 0.f, fmt));
    }
  }
}

// s[] summed over the threads of each row, in a fixed order, to all of them.  `red`: [32][n] floats that the last
// sum before this one did not use; a row's warps follow one another.
template <int n>
__device__ __forceinline__ void ln_row_sums(float (&s)[n], float* red, int warps_per_row) {
  #pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    #pragma unroll
    for (int i = 0; i < n; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  }
  if (warps_per_row == 1) return;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    #pragma unroll
    for (int i = 0; i < n; ++i) red[warp * n + i] = s[i];
  }
  __syncthreads();
  const float* first = red + warp / warps_per_row * warps_per_row * n;
  #pragma unroll
  for (int i = 0; i < n; ++i) s[i] = first[i];
  for (int w = 1; w < warps_per_row; ++w) {
    #pragma unroll
    for (int i = 0; i < n; ++i) s[i] += first[w * n + i];
  }
}

template <int XF, int MAXT, int NV, bool VEC, int U>
__global__ void __launch_bounds__(MAXT) layer_norm_kernel(const LnArgs a) {
  __shared__ float red[2][32 * U];
  const int g = threadIdx.x / a.tpr, t = threadIdx.x - g * a.tpr, G = blockDim.x / a.tpr, C = a.C;
  float w[NV][8], b[NV][8];
  #pragma unroll
  for (int i = 0; i < NV; ++i) {
    #pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = ln_col<VEC>(i, e, t, a.tpr);
      w[i][e] = a.w && c < C ? load_elem(a.w, c, a.w_fmt) : 1.f;
      b[i][e] = a.b && c < C ? load_elem(a.b, c, a.w_fmt) : 0.f;
    }
  }
  const long long step = static_cast<long long>(gridDim.x) * G;
  const float inv = 1.f / C;
  for (long long r0 = static_cast<long long>(blockIdx.x) * G; r0 < a.rows; r0 += U * step) {
    float v[U][NV][8], s[U];
    #pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = r0 + u * step + g;
      #pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (r < a.rows) {
          ln_load<XF, VEC>(a.x, static_cast<size_t>(r) * a.xs, i, t, a.tpr, C, a.x_fmt, v[u][i]);
        } else {
          #pragma unroll
          for (int e = 0; e < 8; ++e) v[u][i][e] = 0.f;
        }
      }
    }
    #pragma unroll
    for (int u = 0; u < U; ++u) {
      s[u] = 0.f;
      #pragma unroll
      for (int i = 0; i < NV; ++i) {
        #pragma unroll
        for (int e = 0; e < 8; ++e) s[u] += v[u][i][e];
      }
    }
    ln_row_sums(s, red[0], a.tpr >> 5);
    float mean[U];
    #pragma unroll
    for (int u = 0; u < U; ++u) {
      mean[u] = s[u] * inv;
      s[u] = 0.f;
      #pragma unroll
      for (int i = 0; i < NV; ++i) {
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[u][i][e] -= mean[u];
          const float d = ln_col<VEC>(i, e, t, a.tpr) < C ? v[u][i][e] : 0.f;
          s[u] = fmaf(d, d, s[u]);
        }
      }
    }
    ln_row_sums(s, red[1], a.tpr >> 5);
    #pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = r0 + u * step + g;
      if (r >= a.rows) break;
      const float rs = rsqrtf(fmaf(s[u], inv, a.eps));
      #pragma unroll
      for (int i = 0; i < NV; ++i) {
        #pragma unroll
        for (int e = 0; e < 8; ++e) v[u][i][e] = fmaf(v[u][i][e] * rs, w[i][e], b[i][e]);
        ln_store<VEC>(a.y, static_cast<size_t>(r) * C, i, t, a.tpr, C, a.y_fmt, v[u][i]);
      }
      if (t == 0) {
        a.mean[r] = mean[u];
        a.rstd[r] = rs;
      }
    }
  }
}

template <int XF, int ZF, int MAXT, int NV, bool VEC, int U>
__global__ void __launch_bounds__(MAXT) layer_norm_bwd_kernel(const LnArgs a) {
  __shared__ float red[2][32 * 2 * U];
  extern __shared__ float sums[];   // [2][G][NV * 8 * tpr], where a block holds more than one row
  grid_launch_dependents();         // partial_rows_kernel starts as these blocks run out
  const int g = threadIdx.x / a.tpr, t = threadIdx.x - g * a.tpr, G = blockDim.x / a.tpr, C = a.C;
  float w[NV][8], dw[NV][8], db[NV][8];
  #pragma unroll
  for (int i = 0; i < NV; ++i) {
    #pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = ln_col<VEC>(i, e, t, a.tpr);
      w[i][e] = a.w && c < C ? load_elem(a.w, c, a.w_fmt) : 1.f;
      dw[i][e] = db[i][e] = 0.f;
    }
  }
  const long long step = static_cast<long long>(gridDim.x) * G;
  const float inv = 1.f / C;
  int buf = 0;
  for (long long r0 = static_cast<long long>(blockIdx.x) * G; r0 < a.rows; r0 += U * step, buf ^= 1) {
    float v[U][NV][8], z[U][NV][8], s[2 * U], rs[U], mu[U];
    #pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = r0 + u * step + g;
      const bool there = r < a.rows;
      mu[u] = there ? a.mean_in[r] : 0.f;
      rs[u] = there ? a.rstd_in[r] : 0.f;
      #pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (there) {
          ln_load<XF, VEC>(a.x, static_cast<size_t>(r) * a.xs, i, t, a.tpr, C, a.x_fmt, v[u][i]);
          ln_load<ZF, VEC>(a.dy, static_cast<size_t>(r) * C, i, t, a.tpr, C, a.y_fmt, z[u][i]);
        } else {
          #pragma unroll
          for (int e = 0; e < 8; ++e) v[u][i][e] = z[u][i][e] = 0.f;
        }
      }
    }
    #pragma unroll
    for (int u = 0; u < U; ++u) {
      float s1 = 0.f, s2 = 0.f;
      #pragma unroll
      for (int i = 0; i < NV; ++i) {
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float h = (v[u][i][e] - mu[u]) * rs[u];
          v[u][i][e] = h;
          db[i][e] += z[u][i][e];
          dw[i][e] = fmaf(z[u][i][e], h, dw[i][e]);
          const float q = z[u][i][e] * w[i][e];   // 0 past the row's end
          z[u][i][e] = q;
          s1 += q;
          s2 = fmaf(q, h, s2);
        }
      }
      s[2 * u] = s1;
      s[2 * u + 1] = s2;
    }
    ln_row_sums(s, red[buf], a.tpr >> 5);
    #pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = r0 + u * step + g;
      if (r >= a.rows) break;
      const float m1 = s[2 * u] * inv, m2 = s[2 * u + 1] * inv;
      #pragma unroll
      for (int i = 0; i < NV; ++i) {
        float d[8];
        if (a.dres) {
          ln_load<-1, VEC>(a.dres, static_cast<size_t>(r) * C, i, t, a.tpr, C, a.dx_fmt, d);
        } else {
          #pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = 0.f;
        }
        #pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = fmaf(rs[u], fmaf(-m2, v[u][i][e], z[u][i][e] - m1), d[e]);
        ln_store<VEC>(a.dx, static_cast<size_t>(r) * C, i, t, a.tpr, C, a.dx_fmt, d);
      }
    }
  }
  if (!a.parts) return;
  // the block's rows side by side, then one partial row of 2 C floats
  if (G > 1) {
    const int n = NV * 8 * a.tpr;
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      #pragma unroll
      for (int e = 0; e < 8; ++e) {
        sums[g * n + (i * 8 + e) * a.tpr + t] = dw[i][e];
        sums[(G + g) * n + (i * 8 + e) * a.tpr + t] = db[i][e];
      }
    }
    __syncthreads();
    if (g > 0) return;
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      #pragma unroll
      for (int e = 0; e < 8; ++e) {
        for (int k = 1; k < G; ++k) {
          dw[i][e] += sums[k * n + (i * 8 + e) * a.tpr + t];
          db[i][e] += sums[(G + k) * n + (i * 8 + e) * a.tpr + t];
        }
      }
    }
  }
  float* out = a.parts + static_cast<size_t>(blockIdx.x) * 2 * C;
  #pragma unroll
  for (int i = 0; i < NV; ++i) {
    #pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = ln_col<VEC>(i, e, t, a.tpr);
      if (c >= C) continue;
      out[c] = dw[i][e];
      out[C + c] = db[i][e];
    }
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
