// Products of tokens and weights for linear layers on tcgen05: forward, gradient of the input, gradient of the weight.
//
//   y = act(x W^T + bias) + residual,   dx = (dy W) * slope(input_pre),   dW = dy^T x
//
// D = A B^T in tiles.  Each operand is read by TMA from where it lies, in boxes of 64 elements (one 128-byte
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
  static constexpr int NS = BN == 256 ? 4 : (BN == 128 ? 6 : 8);
  static constexpr int kBars = NS * kStage;
  static constexpr int kMisc = kBars + (2 * NS + 3) * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static_assert(kAlloc <= 232448, "shared memory");
};

// Where an operand's loads are: rows [r0, r0 + ROWS) of a tile, contraction steps one after another.  One thread walks it, so
// that a step is additions only: with divisions it took longer than the step's products.
template <bool MN, int ROWS>
struct LinCursor {
  int d, steps_batch;
  int b, h, f, row, left;   // of the next step: batch, head and feature in it, row; steps left in the batch
  int fj[ROWS >= 64 ? ROWS / 64 : 1], hj[ROWS >= 64 ? ROWS / 64 : 1];   // MN: features and heads of the 64-column blocks
  // d: features a head (0: one head); batch: of a K-major operand
  __device__ __forceinline__ LinCursor(int d_, int r0, int batch, int s, int steps_batch_) : d(d_), steps_batch(steps_batch_) {
    if (!MN) {
      f = kLinStep * s;
      h = d && s > 0 ? f / d : 0;
      f -= h * d;
      row = r0;
      b = batch;
    } else {
      b = s > 0 ? s / steps_batch : 0;
      left = steps_batch - (s - b * steps_batch);
      row = (s - b * steps_batch) * kLinStep;
      #pragma unroll
      for (int j = 0; j < ROWS / 64; ++j) {
        hj[j] = d ? (r0 + 64 * j) / d : 0;
        fj[j] = r0 + 64 * j - hj[j] * d;
      }
    }
  }
  // load(dst, feature, row, head, batch) for each box of the step, and on to the next one
  template <class Load>
  __device__ __forceinline__ void step(uint8_t* dst, Load&& load) {
    if (!MN) {
      load(dst, f, row, h, b);
      f += kLinStep;
      if (f == d) {
        f = 0;
        ++h;
      }
    } else {
      #pragma unroll
      for (int j = 0; j < ROWS / 64; ++j) load(dst + j * 64 * 128, fj[j], row, hj[j], b);
      row += kLinStep;
      if (--left == 0) {
        left = steps_batch;
        row = 0;
        ++b;
      }
    }
  }
};

__device__ __forceinline__ long long lin_feature(const LinView& v, int f) {   // offset of feature f in its token
  const int h = v.d ? f / v.d : 0;
  return h * v.sh + (f - h * v.d);
}

__device__ __forceinline__ void store_elem(void* p, size_t i, float x, int fmt) {
  if (fmt == kF32) reinterpret_cast<float*>(p)[i] = x;
  else reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(pack_in(x, 0.f, fmt));
}

// An epilogue warp's part of a tile: 32 rows of D, COLS columns, a row a lane as TMEM gives them.  What is read and written beside D
// goes through shared memory by TMA, in boxes of 32 rows x 128 bytes (64 columns in 16 bits, 32 in fp32),
// swizzled so that lanes meet different banks: whole lines of memory, asynchronously, and edges are left to TMA.  (Plain stores from
// this layout touch 32 lines an instruction: 216 us for 32768 x 1024 x 4096; turned in shared memory first, 156, and 195 where gelu's
// argument is kept.)
struct LinEpi {
  uint8_t* slot;       // [SLOTS][32 rows x 128 bytes]
  float* row;          // [32] (forward)
  uint64_t* bars;      // [2]: a box beside D landed
  uint32_t phases;     // bit i: of the next one
  const CUtensorMap* out;
  const CUtensorMap* aux;
  const CUtensorMap* pre;
};

// 16-byte chunk c of this lane's row in a box of 128-byte (or, narrow, 64-byte) rows.
__device__ __forceinline__ uint4* lin_chunk(uint8_t* slot, int c) {
  const int lane = threadIdx.x & 31;
  return reinterpret_cast<uint4*>(slot + lane * 128 + ((c ^ (lane & 7)) << 4));
}
__device__ __forceinline__ uint4* lin_chunk_narrow(uint8_t* slot, int c) {
  const int lane = threadIdx.x & 31;
  return reinterpret_cast<uint4*>(slot + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4));
}
// 32 columns of this lane's row: of fp32 a whole box; of 16 bits half `half` of one, or a narrow one.
__device__ __forceinline__ void lin_write(uint8_t* slot, const float* v, int fmt, int half, bool narrow) {
  if (fmt == kF32) {
    #pragma unroll
    for (int c = 0; c < 8; ++c)
      *lin_chunk(slot, c) = make_uint4(__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]),
                                       __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3]));
  } else {
    #pragma unroll
    for (int c = 0; c < 4; ++c)
      *(narrow ? lin_chunk_narrow(slot, c) : lin_chunk(slot, c + 4 * half)) =
          pack8(*reinterpret_cast<const float(*)[8]>(&v[8 * c]), fmt);
  }
}
__device__ __forceinline__ void lin_read(uint8_t* slot, float (&x)[32], int fmt, int half, bool narrow) {
  if (fmt == kF32) {
    #pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 u = *lin_chunk(slot, c);
      x[4 * c] = __uint_as_float(u.x), x[4 * c + 1] = __uint_as_float(u.y);
      x[4 * c + 2] = __uint_as_float(u.z), x[4 * c + 3] = __uint_as_float(u.w);
    }
  } else {
    #pragma unroll
    for (int c = 0; c < 4; ++c)
      unpack8(*(narrow ? lin_chunk_narrow(slot, c) : lin_chunk(slot, c + 4 * half)), *reinterpret_cast<float(*)[8]>(&x[8 * c]), fmt);
  }
}

// wait() returns whether D is complete (of the whole warp), done() says that it has been read.  SLOTS: of 4 KB, one or two a warp.
//   16-bit output            a box a group of 64 columns, with two slots each group's its own
//   ... and an argument      a slot each; with one slot (then nothing is read beside D) half a slot each, a box a half group
//   fp32 output              a box a half group, with two slots its own; an argument goes through the half's slot first
// FINE: D is not in TMEM, but after wait() in acc.
template <int KIND, int COLS, int SLOTS, bool FINE, class Wait, class Done>
__device__ __forceinline__ bool lin_epilogue(const LinArgs& a, LinEpi& e, uint32_t taddr, float (&acc)[FINE ? COLS : 1], int b, int row0,
                                             int f0, volatile int* abort_flag, Wait&& wait, Done&& done) {
  static_assert(COLS == 64 || (COLS == 128 && SLOTS == 2), "one or two groups of 64 columns");
  static_assert(!FINE || SLOTS == 2, "registers for D");
  constexpr int GROUPS = COLS / 64;
  const int lane = threadIdx.x & 31;
  const bool out16 = a.out_fmt != kF32, own = out16 && !(KIND == kLinForward && a.pre);
  const bool narrow = SLOTS == 1 && KIND == kLinForward && a.pre;   // boxes of 64-byte rows
  const bool halves = !out16 || narrow;   // a box a half group
  const bool rows_in = row0 < a.rows;
  auto fetch = [&](int f, int i) {   // by one lane: the box beside D from column f into slot i
    if (!rows_in || f >= a.cols) return;
    const int h = a.aux_at.d ? f / a.aux_at.d : 0;
    mbar_arrive_expect_tx(&e.bars[i], halves && a.aux_fmt != kF32 ? 2048 : 4096);
    tma_load_4d(e.slot + 4096 * i, e.aux, &e.bars[i], f - h * a.aux_at.d, row0, h, b);
  };
  auto fetch_group = [&](int f) {
    fetch(f, 0);
    if (SLOTS == 2 && halves) fetch(f + 32, 1);
  };
  float bias[COLS / 32];   // a column a lane (every lane reading all 32 from memory took 1100 cycles a half group, shuffles 550)
  #pragma unroll
  for (int c = 0; c < COLS / 32; ++c) {
    const int f = f0 + 32 * c + lane;
    bias[c] = KIND == kLinForward && a.bias && f < a.cols ? load_elem(a.bias, f, a.bias_fmt) : 0.f;
  }
  // boxes asked for and not waited for, should this warp give up: they land before it leaves (with a limit)
  uint32_t pending = 0;
  auto give_up = [&] {
    if (lane == 0)
      for (int i = 0; i < 2; ++i)
        if (pending >> i & 1) mbar_wait_budget(&e.bars[i], e.phases >> i & 1, kWaitBudgetCycles);
    return false;
  };
  if (lane == 0) bulk_wait_read();   // the last tile's boxes
  if (a.aux && rows_in && f0 < a.cols) {
    pending = 1;
    if (SLOTS == 2 && halves && f0 + 32 < a.cols) pending = 3;
    if (GROUPS > 1 && own && f0 + 64 < a.cols) pending = 3;
    if (lane == 0) {
      fetch_group(f0);
      if (GROUPS > 1 && own) fetch(f0 + 64, 1);
    }
  }
  if (!wait()) return give_up();
  #pragma unroll(FINE ? GROUPS : 1)
  for (int g = 0; g < GROUPS; ++g) {
    uint32_t u[SLOTS][32];
    if (FINE) {
      #pragma unroll
      for (int j = 0; j < 64; ++j) u[SLOTS == 2 ? j / 32 : 0][j & 31] = __float_as_uint(acc[FINE ? 64 * g + j : 0]);
    } else {
      if (g > 0) __syncwarp();   // one lane stored the last group, the whole warp loads this one
      tmem_ld32(taddr + 64 * g, u[0]);
      if (SLOTS == 2) tmem_ld32(taddr + 64 * g + 32, u[SLOTS - 1]);
      tmem_wait_ld();
      if (SLOTS == 2 && g + 1 == GROUPS) done();
    }
    const int fg = f0 + 64 * g;
    const bool in = rows_in && fg < a.cols;
    if (SLOTS == 2 && !in) continue;
    if (g > 0 && !own) {   // the last group's boxes have been read
      if (lane == 0) {
        bulk_wait_read();
        if (a.aux) fetch_group(fg);
      }
      if (a.aux) pending = halves && fg + 32 < a.cols ? 3 : 1;
      __syncwarp();
    }
    const int h = a.out_at.d ? fg / a.out_at.d : 0, fh = fg - h * a.out_at.d;
    #pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int f = fg + 32 * half;
      if (SLOTS == 1 && half == 1) {
        __syncwarp();   // as above
        tmem_ld32(taddr + 32, u[0]);
        tmem_wait_ld();
        done();
      }
      if (!in || f >= a.cols) continue;
      const int i = SLOTS == 1 ? 0 : (out16 ? (own ? g : 0) : half);   // its slot
      uint8_t* const slot = e.slot + 4096 * i;
      if (SLOTS == 1 && half == 1 && halves) {   // the first half's boxes have been read
        if (lane == 0) {
          bulk_wait_read();
          if (a.aux) fetch(f, 0);
        }
        if (a.aux) pending = 1;
        __syncwarp();
      }
      float v[32];
      #pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[SLOTS == 1 ? 0 : half][j]);
      if (KIND == kLinForward && a.bias) {
        const float at = GROUPS > 1 && g > 0 ? bias[COLS / 32 - 2 + half] : bias[half];
        __syncwarp();
        e.row[lane] = at;
        __syncwarp();
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 y = reinterpret_cast<const float4*>(e.row)[j];
          v[4 * j] += y.x, v[4 * j + 1] += y.y, v[4 * j + 2] += y.z, v[4 * j + 3] += y.w;
        }
      }
      float x[32];
      if (a.aux) {
        if (halves || half == 0) {
          if (!warp_all(mbar_wait(&e.bars[i], e.phases >> i & 1, abort_flag, a.status))) return give_up();
          e.phases ^= 1u << i;
          pending &= ~(1u << i);
        }
        lin_read(slot, x, a.aux_fmt, half, halves);
        if (halves) __syncwarp();   // rows of different types do not lie at the same bytes
      }
      if (KIND == kLinForward) {
        if (a.pre) {
          if (out16) {
            lin_write(e.slot + (narrow ? 2048 : 4096), v, a.fmt, half, narrow);
          } else {
            lin_write(slot, v, a.fmt, 0, true);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_4d(e.pre, slot, fh + 32 * half, row0, h, b);
              bulk_commit();
              bulk_wait_read();
            }
            __syncwarp();
          }
        }
        if (a.act != kActNone) with_act(a.act, [&](auto A) { act_all<decltype(A)::value>(v); });
        if (a.aux) {
          #pragma unroll
          for (int j = 0; j < 32; ++j) v[j] += x[j];
        }
      }
      if (KIND == kLinInput && a.aux) with_act(a.act, [&](auto A) { slope_all<decltype(A)::value>(v, x); });
      lin_write(slot, v, a.out_fmt, half, narrow);
      if (!halves && half == 0 && f + 32 < a.cols) continue;   // the other half of the box
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        const int at = halves ? fh + 32 * half : fh;
        if (KIND == kLinForward && a.pre && out16) tma_store_4d(e.pre, e.slot + (narrow ? 2048 : 4096), at, row0, h, b);
        tma_store_4d(e.out, slot, at, row0, h, b);
        bulk_commit();
      }
    }
  }
  return true;
}

// With the operands swapped: one feature f of T tokens from n, `count` of them there.
template <int KIND, int T>
__device__ __forceinline__ void lin_finish_turned(const LinArgs& a, float (&v)[T], int n, int f, int count) {
  static_assert(T % 2 == 0, "pairs");
  const size_t out = static_cast<size_t>(n * a.out_at.sn + lin_feature(a.out_at, f));
  const size_t aux = static_cast<size_t>(n * a.aux_at.sn + lin_feature(a.aux_at, f));
  float x[T];
  if (a.aux) {
    #pragma unroll
    for (int j = 0; j < T; ++j) x[j] = j < count ? load_elem(a.aux, aux + j * a.aux_at.sn, a.aux_fmt) : 0.f;
  }
  if (KIND == kLinForward) {
    const float bias = a.bias ? load_elem(a.bias, f, a.bias_fmt) : 0.f;
    #pragma unroll
    for (int j = 0; j < T; ++j) v[j] += bias;
    if (a.pre) {
      #pragma unroll
      for (int j = 0; j < T; ++j)
        if (j < count) store_elem(a.pre, out + j * a.out_at.sn, v[j], a.fmt);
    }
    if (a.act != kActNone) with_act(a.act, [&](auto A) { act_all<decltype(A)::value>(v); });
    if (a.aux) {
      #pragma unroll
      for (int j = 0; j < T; ++j) v[j] += x[j];
    }
  }
  if (KIND == kLinInput && a.aux) with_act(a.act, [&](auto A) { slope_all<decltype(A)::value>(v, x); });
  #pragma unroll
  for (int j = 0; j < T; ++j)
    if (j < count) store_elem(a.out, out + j * a.out_at.sn, v[j], a.out_fmt);
}

// Sixteen columns of TMEM added to v, and v of `accs` sums, `apart` columns from one to the next.
__device__ __forceinline__ void lin_add_to(uint32_t taddr, float (&v)[16]) {
  uint32_t u[16];
  tmem_ld16(taddr, u);
  tmem_wait_ld();
  #pragma unroll
  for (int j = 0; j < 16; ++j) v[j] += __uint_as_float(u[j]);
}
__device__ __forceinline__ void lin_sum_of(uint32_t taddr, int apart, int accs, float (&v)[16]) {
  #pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = 0.f;
  for (int i = 0; i < accs; ++i) lin_add_to(taddr + i * apart, v);
}

// Few tokens: 128 features by BN tokens a tile, the features as rows, so that a product of few tokens still fills the tensor
// core's 128 rows.  What counts then is how many SMs read the weight: a cluster of CTAs shares a tile, each with a piece of the
// contraction, and each adds up all of their parts for its share of the tokens, through distributed shared memory and in order.
// 32 tokens x 1024 x 4096: 5.8 us (9.6 without clusters; the weight's 8 MB take 1.2 at 6.8 TB/s), 32 x 4096 x 1024 6.7 (19 without); the
// rest is the kernel's start, two trips to memory and the exchange.
template <int KIND, int BN, bool BF16>
__global__ void __launch_bounds__(kLinThreads) linear_few_kernel(const __grid_constant__ CUtensorMap map_a,
                                                                 const __grid_constant__ CUtensorMap map_b,
                                                                 const __grid_constant__ LinArgs a) {
  using SM = LinSmem<BN>;
  constexpr int NS = SM::NS;
  constexpr bool A_MN = KIND == kLinInput;   // W's columns in the input's gradient
  // A piece's steps go to four sums (two of 256 tokens) in turn, which are added at the end: the tensor core cuts towards zero when
  // it adds, and a long chain drifts (linear_pair.cuh).  Where the result is fp32 and a sum would have more than kLinChain steps, one of
  // them is a total, to which the epilogue's warps add the others after every `round` steps; the loads run on meanwhile (fp32, 32 x 4096 x
  // 32000 50 us either way, 100 x 16384 x 9800 84 for 74, 200 x 16384 x 264, one sum and a total, 24 for 19; the pairs' chains took 87 and 63).
  constexpr int ACCS = BN == 256 ? 2 : 4;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBars);
  uint64_t* empty = full + NS;
  uint64_t* done = empty + NS;
  uint64_t* round_full = done + 1;
  uint64_t* round_empty = done + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + SM::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM::kMisc + 4);
  float4* part = reinterpret_cast<float4*>(smem);   // [BN / 4][128 features] four tokens, once the products are done
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), pieces = a.pieces;
  const int r0 = blockIdx.x / pieces * 128, c0 = blockIdx.y * BN;   // first feature and token
  const int s0 = rank * a.steps / pieces, s1 = (rank + 1) * a.steps / pieces;
  const bool rounds = a.out_fmt == kF32 && s1 - s0 > kLinChain * ACCS;
  const int live = rounds ? ACCS - 1 : ACCS, round = rounds ? kLinChain * live : s1 - s0, last = rounds ? (s1 - s0 - 1) / round : 0;
  if (KIND == kLinInput) grid_launch_dependents();   // as in linear_pair.cuh
  if (threadIdx.x == 128) {
    tma_prefetch_desc(&map_a);
    tma_prefetch_desc(&map_b);
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < 2 * NS + 2; ++i) mbar_init(&full[i], 1);
    mbar_init(round_empty, 4);
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(slot, ACCS * BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *slot;
  if (warp == 4) {
    if (lane == 0) {
      LinCursor<A_MN, 128> at_a(a.a_d, r0, 0, s0, a.steps);
      LinCursor<false, BN> at_b(a.b_d, c0, 0, s0, a.steps);
      int n = 0;
      for (int s = s0; s < s1; ++s, ++n) {
        const int st = n % NS;
        if (!mbar_wait(&empty[st], ((n / NS) & 1) ^ 1, abort_flag, a.status)) break;
        mbar_arrive_expect_tx(&full[st], SM::kStage);
        at_a.step(smem + st * SM::kStage, [&](uint8_t* dst, int f, int row, int h, int bb) {
          tma_load_4d(dst, &map_a, &full[st], f, row, h, bb);
        });
        at_b.step(smem + st * SM::kStage + SM::kA, [&](uint8_t* dst, int f, int row, int h, int bb) {
          tma_load_4d(dst, &map_b, &full[st], f, row, h, bb);
        });
      }
      // the copies have landed: at once after a whole run, and with a limit if some role gave up
      for (int i = max(0, n - NS); i < n; ++i) mbar_wait_budget(&full[i % NS], (i / NS) & 1, kWaitBudgetCycles);
    }
    __syncwarp();
  } else if (warp == 5) {
    constexpr uint32_t fmt = BF16 ? 1 : 0;
    constexpr uint32_t id = idesc_f16(128, BN, fmt, fmt, A_MN, 0);
    constexpr uint32_t ka = A_MN ? 128 : 2;   // 16 contraction elements further, in 16 bytes
    const uint64_t da = sdesc_sw128(smem_u32(smem), A_MN ? 8192 : 16, 1024);
    const uint64_t db = sdesc_sw128(smem_u32(smem) + SM::kA, 16, 1024);
    int at = 0, sum = 0, r = 0;   // the step in its round, its sum, the round
    for (int n = 0; n < s1 - s0; ++n, ++at) {
      const int st = n % NS;
      if (at == round) {
        umma_commit_w(round_full);
        if (!warp_all(mbar_wait(round_empty, r & 1, abort_flag, a.status))) break;
        at = sum = 0;
        ++r;
      }
      const bool ok = mbar_wait(&full[st], (n / NS) & 1, abort_flag, a.status);
      if (!warp_all(ok)) break;
      tc_fence_after();
      #pragma unroll
      for (int k = 0; k < 4; ++k)
        umma_ss_w(tbase + BN * sum, da + st * (SM::kStage >> 4) + ka * k, db + st * (SM::kStage >> 4) + 2 * k, id,
                  (at >= live || k > 0) ? 1u : 0u);
      if (++sum == live) sum = 0;
      umma_commit_w(&empty[st]);
    }
    umma_commit_w(done);
    mbar_wait_budget(done, 0, kWaitBudgetCycles);
    __syncwarp();
  }
  const uint32_t taddr = tbase + (static_cast<uint32_t>(32 * warp) << 16), total = taddr + BN * (ACCS - 1);
  if (warp < 4) {
    for (int r = 0; r < last && warp_all(mbar_wait(round_full, r & 1, abort_flag, a.status)); ++r) {
      tc_fence_after();
      #pragma unroll 1
      for (int c = 0; c < BN; c += 16) {
        float v[16];
        lin_sum_of(taddr + c, BN, live, v);
        if (r > 0) lin_add_to(total + c, v);
        #pragma unroll
        for (int j = 0; j < 16; j += 8) {
          uint32_t u[8];
          #pragma unroll
          for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(v[j + i]);
          tmem_st8(total + c + j, u);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(round_empty);
    }
  }
  const bool ok = warp < 4 && warp_all(mbar_wait(done, 0, abort_flag, a.status));
  const int f = r0 + threadIdx.x;   // this thread's feature
  const int accs = min(live, s1 - s0 - last * round);
  tc_fence_after();
  if (pieces > 1) {
    if (ok) {
      #pragma unroll 1
      for (int c = 0; c < BN; c += 16) {
        float v[16];
        lin_sum_of(taddr + c, BN, accs, v);
        if (rounds) lin_add_to(total + c, v);
        #pragma unroll
        for (int j = 0; j < 4; ++j)
          part[(c / 4 + j) * 128 + threadIdx.x] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
    }
    __syncwarp();
    cluster_sync_all();
    // this CTA's share of the tokens, T at a time; every CTA's part of them, added in order (their loads are all on their way before
    // the first is needed)
    const int share = BN / pieces;
    auto join = [&](auto tokens) {
      constexpr int T = decltype(tokens)::value;
      #pragma unroll 1
      for (int t = rank * share; t < (rank + 1) * share && c0 + t < a.cols; t += T) {
        float v[T];
        #pragma unroll
        for (int j = 0; j < T; ++j) v[j] = 0.f;
        const float4* from = part + t / 4 * 128 + threadIdx.x;
        #pragma unroll 4
        for (int p = 0; p < pieces; ++p) {
          const uint32_t at = cluster_map(from, p);
          #pragma unroll
          for (int j = 0; j < T / 4; ++j) {
            const float4 x = ld_cluster4(at + j * 2048);
            v[4 * j] += x.x, v[4 * j + 1] += x.y, v[4 * j + 2] += x.z, v[4 * j + 3] += x.w;
          }
        }
        lin_finish_turned<KIND>(a, v, c0 + t, f, min(T, a.cols - c0 - t));
      }
    };
    if (warp < 4 && f < a.rows) {
      if (share >= 8) join(std::integral_constant<int, 8>());
      else join(std::integral_constant<int, 4>());
    }
    __syncwarp();
    cluster_sync_all_relaxed();   // no CTA leaves while its part is read
  } else if (ok) {
    #pragma unroll 1
    for (int c = 0; c < BN && c0 + c < a.cols; c += 16) {
      float v[16];
      lin_sum_of(taddr + c, BN, accs, v);
      if (rounds) lin_add_to(total + c, v);
      if (f < a.rows) lin_finish_turned<KIND>(a, v, c0 + c, f, min(16, a.cols - c0 - c));
      __syncwarp();   // lanes without a feature left it out; the whole warp loads what follows
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 5) tmem_dealloc(tbase, ACCS * BN);
}

}  // namespace dera
