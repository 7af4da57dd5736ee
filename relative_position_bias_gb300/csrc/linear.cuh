// Products of tokens and weights for linear layers on tcgen05: forward, gradient of the input, gradient of the weight.
//
//   y = act(x W^T + bias) + residual,   dx = (dy W) * slope(input_pre),   dW = dy^T x
//
// D = A B^T in tiles of 128 x BN.  Each operand is read by TMA from where it lies, in boxes of 64 elements (one 128-byte
// swizzle atom) by its rows: K-major where the contraction is its contiguous dimension, else M- or N-major, so
// nothing is transposed on the way.  Tokens are addressed as (batch, token, head, element): the attention's output is read from
// its heads, and a gradient written to them.  What lies past an edge reads as zero.
#pragma once
#include "activation.cuh"
#include "block.cuh"
#include "common.cuh"

namespace dera {

constexpr int kLinThreads = 192;   // four epilogue warps, one that loads, one that multiplies
constexpr int kLinStep = 64;       // contraction elements of a step

template <int BN>
struct LinSmem {
  static constexpr int kA = 128 * 128, kB = BN * 128;
  static constexpr int kStage = kA + kB;
  static constexpr int NS = BN >= 128 ? 6 : 8;
  static constexpr int kBars = NS * kStage;
  static constexpr int kMisc = kBars + (2 * NS + 1) * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static_assert(kAlloc <= 232448, "shared memory");
};

// One operand's rows [r0, r0 + ROWS) of batch b for contraction step s.
template <bool MN, int ROWS>
__device__ __forceinline__ void lin_load(uint8_t* dst, const CUtensorMap* m, uint64_t* bar, int d, int r0, int b, int s,
                                         int steps_batch) {
  if (!MN) {
    const int f = kLinStep * s, h = d ? f / d : 0;
    tma_load_4d(dst, m, bar, f - h * d, r0, h, b);
  } else {
    const int bb = s / steps_batch, row = (s - bb * steps_batch) * kLinStep;
    #pragma unroll
    for (int j = 0; j < ROWS / 64; ++j) {
      const int f = r0 + 64 * j, h = d ? f / d : 0;
      tma_load_4d(dst + j * 64 * 128, m, bar, f - h * d, row, h, bb);
    }
  }
}

__device__ __forceinline__ size_t lin_at(const LinView& v, int b, int n, int f) {
  const int h = v.d ? f / v.d : 0;
  return static_cast<size_t>(b * v.sb + n * v.sn + h * v.sh + (f - h * v.d));
}

__device__ __forceinline__ void store_elem(void* p, size_t i, float x, int fmt) {
  if (fmt == kF32) reinterpret_cast<float*>(p)[i] = x;
  else reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(pack_in(x, 0.f, fmt));
}

// 32 neighbouring columns from f of one row (token n of batch b, or a row of dW): what becomes of them, and their store.
template <int KIND>
__device__ __forceinline__ void lin_finish(const LinArgs& a, float (&v)[32], int b, int n, int f) {
  const int left = min(4, (a.cols - f) / 8);   // columns come in eights
  if (KIND == kLinForward) {
    const size_t at = lin_at(a.out_at, b, n, f);
    if (a.bias) {
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x[8];
        if (j < left) {
          load8(a.bias, f + 8 * j, x, a.bias_fmt);
          #pragma unroll
          for (int e = 0; e < 8; ++e) v[8 * j + e] += x[e];
        }
      }
    }
    if (a.pre) {
      #pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) store8(a.pre, at + 8 * j, *reinterpret_cast<const float(*)[8]>(&v[8 * j]), a.fmt);
    }
    if (a.act != kActNone)
      with_act(a.act, [&](auto A) {
        #pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = act_of<decltype(A)::value>(v[j]);
      });
    if (a.aux) {
      const size_t from = lin_at(a.aux_at, b, n, f);
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x[8];
        if (j < left) {
          load8(a.aux, from + 8 * j, x, a.aux_fmt);
          #pragma unroll
          for (int e = 0; e < 8; ++e) v[8 * j + e] += x[e];
        }
      }
    }
  }
  if (KIND == kLinInput && a.aux) {
    const size_t from = lin_at(a.aux_at, b, n, f);
    float x[32];
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
      float y[8];
      #pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = 0.f;
      if (j < left) load8(a.aux, from + 8 * j, y, a.aux_fmt);
      #pragma unroll
      for (int e = 0; e < 8; ++e) x[8 * j + e] = y[e];
    }
    with_act(a.act, [&](auto A) {
      #pragma unroll
      for (int j = 0; j < 32; ++j) v[j] *= act_slope<decltype(A)::value>(x[j]);
    });
  }
  const size_t at = lin_at(a.out_at, b, n, f);
  #pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < left) store8(a.out, at + 8 * j, *reinterpret_cast<const float(*)[8]>(&v[8 * j]), a.out_fmt);
}

// The same with the operands swapped: one feature f of `count` tokens from n.
template <int KIND>
__device__ __forceinline__ void lin_finish_turned(const LinArgs& a, float (&v)[32], int n, int f, int count) {
  if (KIND == kLinForward) {
    const float bias = a.bias ? load_elem(a.bias, f, a.bias_fmt) : 0.f;
    #pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += bias;
    if (a.pre) {
      #pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < count) store_elem(a.pre, lin_at(a.out_at, 0, n + j, f), v[j], a.fmt);
    }
    if (a.act != kActNone)
      with_act(a.act, [&](auto A) {
        #pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = act_of<decltype(A)::value>(v[j]);
      });
    if (a.aux) {
      #pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < count) v[j] += load_elem(a.aux, lin_at(a.aux_at, 0, n + j, f), a.aux_fmt);
    }
  }
  if (KIND == kLinInput && a.aux) {
    float x[32];
    #pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = j < count ? load_elem(a.aux, lin_at(a.aux_at, 0, n + j, f), a.aux_fmt) : 0.f;
    with_act(a.act, [&](auto A) {
      #pragma unroll
      for (int j = 0; j < 32; ++j) v[j] *= act_slope<decltype(A)::value>(x[j]);
    });
  }
  #pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j < count) store_elem(a.out, lin_at(a.out_at, 0, n + j, f), v[j], a.out_fmt);
}

// One tile a CTA.
template <int KIND, int BN, bool TURNED, bool BF16>
__global__ void __launch_bounds__(kLinThreads) linear_kernel(const __grid_constant__ CUtensorMap map_a,
                                                             const __grid_constant__ CUtensorMap map_b,
                                                             const __grid_constant__ LinArgs a) {
  using SM = LinSmem<BN>;
  constexpr int NS = SM::NS;
  constexpr bool A_MN = KIND == kLinInput && TURNED, B_MN = KIND == kLinInput && !TURNED;   // W's columns in the input's gradient
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBars);
  uint64_t* empty = full + NS;
  uint64_t* done = empty + NS;
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + SM::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x, mt = tile / a.n_tiles, b = mt / a.m_tiles;
  const int r0 = (mt - b * a.m_tiles) * 128, c0 = (tile - mt * a.n_tiles) * BN;
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < 2 * NS + 1; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(slot, BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *slot;
  if (warp == 4) {
    if (lane == 0) {
      int s = 0;
      for (; s < a.steps; ++s) {
        const int st = s % NS;
        if (!mbar_wait(&empty[st], ((s / NS) & 1) ^ 1, abort_flag, a.status)) break;
        mbar_arrive_expect_tx(&full[st], SM::kStage);
        lin_load<A_MN, 128>(smem + st * SM::kStage, &map_a, &full[st], a.a_d, r0, b, s, a.steps_batch);
        lin_load<B_MN, BN>(smem + st * SM::kStage + SM::kA, &map_b, &full[st], a.b_d, c0, 0, s, a.steps_batch);
      }
      // the copies have landed: at once after a whole run, and with a limit if some role gave up
      for (int i = max(0, s - NS); i < s; ++i) mbar_wait_budget(&full[i % NS], (i / NS) & 1, kWaitBudgetCycles);
    }
    __syncwarp();
  } else if (warp == 5) {
    constexpr uint32_t fmt = BF16 ? 1 : 0;
    constexpr uint32_t id = idesc_f16(128, BN, fmt, fmt, A_MN, B_MN);
    constexpr uint32_t ka = A_MN ? 128 : 2, kb = B_MN ? 128 : 2;   // 16 contraction elements further, in 16 bytes
    const uint64_t da = sdesc_sw128(smem_u32(smem), A_MN ? 8192 : 16, 1024);
    const uint64_t db = sdesc_sw128(smem_u32(smem) + SM::kA, B_MN ? 8192 : 16, 1024);
    for (int s = 0; s < a.steps; ++s) {
      const int st = s % NS;
      const bool ok = mbar_wait(&full[st], (s / NS) & 1, abort_flag, a.status);
      if (!warp_all(ok)) break;
      tc_fence_after();
      #pragma unroll
      for (int k = 0; k < 4; ++k)
        umma_ss_w(tbase, da + st * (SM::kStage >> 4) + ka * k, db + st * (SM::kStage >> 4) + kb * k, id,
                  (s > 0 || k > 0) ? 1u : 0u);
      umma_commit_w(&empty[st]);
    }
    umma_commit_w(done);
    mbar_wait_budget(done, 0, kWaitBudgetCycles);
    __syncwarp();
  } else {
    const bool ok = mbar_wait(done, 0, abort_flag, a.status);
    if (warp_all(ok)) {
      tc_fence_after();
      const int row = r0 + 32 * warp + lane;
      const bool valid = row < a.rows;
      #pragma unroll 1
      for (int c = 0; c < BN && c0 + c < a.cols; c += 32) {
        uint32_t u[32];
        tmem_ld32(tbase + (static_cast<uint32_t>(32 * warp) << 16) + c, u);
        tmem_wait_ld();
        float v[32];
        #pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
        if (!valid) continue;
        if (TURNED) lin_finish_turned<KIND>(a, v, c0 + c, row, min(32, a.cols - c0 - c));
        else lin_finish<KIND>(a, v, b, row, c0 + c);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) tmem_dealloc(tbase, BN);
}

}  // namespace dera
