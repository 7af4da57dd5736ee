// Backward of the attention with a compact bias (head_dim 64 or 128), on tcgen05.
//
// With Z = scale q k^T + rel_h[n, kh(m)] + rel_w[n, kw(m)], P = softmax(Z) recomputed from
// the forward's base-2 log-sum-exp, D[n] = dO[n] . out[n] and dZ = P * (dO v^T - D):
//   dv = P^T dO,  dk = scale dZ^T q,  dq = scale dZ k,
//   drel_h[n, kh] = sum_kw dZ[n, (kh, kw)],  drel_w[n, kw] = sum_kh dZ[n, (kh, kw)].
// A row's dZ add up to zero, so on an axis of length one the gradient is zero and written as that: the sum in
// numbers would be what out's rounding leaves in D (1e-3 in fp16, 4e-2 in bf16).
//
// Kernels, in stream order:
//   prep   one pass over the bias, out and dO: the exponent's two terms, laid out so that one bulk
//          copy brings what a step needs, hl = log2(e) rel_h - lse and rw = log2(e) rel_w by
//          query column, and -D.  Whatever type the bias has, masks and empty rows end
//          here: hl is -inf where P has to be 0.
//   rows   one CTA per (head, 128 queries), steps of up to 64 keys: S = q k^T and dP = dO v^T,
//          dZ on the softmax threads (a query row each), dq += dZ k on the tensor core; drel_h
//          and drel_w are sums of the fp32 dZ.
//   cols   one CTA per (head, 128 keys), steps of 64 queries: S^T = k q^T and dP^T = v dO^T, P^T
//          and dZ^T on the softmax threads (a key each), dv += P^T dO and dk += dZ^T q.
//   join   adds the pieces of the units that were split (see CbSplit).
// S and dP are formed twice, so that dq, dk and dv are each complete in one CTA: no atomics, and
// the same result on every run.
//
// In rows and cols two or three softmax warpgroups (in cols two pairs of them) take the steps in turn,
// each with its own S and dP in TMEM: while one exponentiates step i the tensor core forms S and dP
// of the next steps for the others and adds step i - 1 to the accumulators.
//
// Measured, 12 heads of 64 x 64 tokens, bf16 (each kernel by itself, caches cold; together, overlapped, 210 us):
//   head_dim 64    prep 16 us (38 MB read, as much written to L2), rows 105 (38 % of the tensor cycles), cols 116
//                  (44 %), join 7.  330 us with head_dim 128.
#pragma once
#include <cfloat>

#include "common.cuh"
#include "train.cuh"

namespace dera {

constexpr int kCbColsThreads = 128 + 512;   // TMA, S and dP, accumulators, idle; two pairs of softmax warpgroups
// registers at launch (the most that 640 threads get), and what the two kinds of warps make of them
constexpr int kCbColsLaunchRegs = 96, kCbColsRegsCtl = 64, kCbColsRegsSmx = 104;
static_assert(kCbColsRegsCtl + 4 * kCbColsRegsSmx <= 5 * kCbColsLaunchRegs, "register split exceeds the launch pool");

// Key steps of the rows kernel: KHT whole grid rows of WP >= W columns, so that a column's kw
// is known at compile time and a thread's rel_w row and drel_w sums stay in registers.
template <int WP>
struct CbKeys {
  static constexpr int KHT = WP <= 16 ? 4 : (WP <= 32 ? 2 : 1);
  static constexpr int BN = KHT * WP;
  static_assert(BN <= 64 && BN % 16 == 0, "tcgen05 N, and two steps of S and dP in TMEM");
};

// Barriers of both kernels.
enum : int {
  kCbAFull = 0,                    // the CTA's own tiles are where the products read them
  kCbRingFull = 1,                 // [8]
  kCbRingEmpty = kCbRingFull + 8,  // [8]
  kCbSFull = kCbRingEmpty + 8,     // [3] S and dP of a step are in TMEM
  kCbPFull = kCbSFull + 3,         // [3] the softmax threads have read S and dP and written dZ (and P)
  kCbAccDone = kCbPFull + 3,       // [3] the products that read dZ (and P) are complete
  kCbAllDone = kCbAccDone + 3,     // every product of the accumulators is complete
  kCbSDone = kCbAllDone + 1,       // and every S and dP
  kCbSFree = kCbSDone + 1,         // [2] cols: S^T and dP^T of a step are in registers
  kCbJoin = kCbSFree + 2,        // the softmax threads among themselves
  kCbBars = kCbJoin + 1
};

constexpr int cb_align(int x) { return (x + 1023) / 1024 * 1024; }

// rows: NB steps in flight, one softmax warpgroup each.  (Registers moved from the control warps to the
// softmax warps, 56 and 152 instead of 128 each, measured the same.)
template <int D>
struct CbRowsDims {
  static constexpr int NB = D == 64 ? 3 : 2;
  static constexpr int kThreads = 128 * (NB + 1);   // TMA, S and dP, accumulators, idle; then the softmax threads
  // TMEM columns: S_b [128 b, 128 b + 64) (dZ_b over it), dP_b 64 further, dq, then q and dO as packed pairs
  static constexpr uint32_t tmDQ = 128 * NB, tmQ = tmDQ + D, tmDO = tmQ + D / 2;
  static_assert(tmDO + D / 2 <= 512, "TMEM");
};

template <int WP, int D>
struct CbRowsSmem {
  static constexpr int AT = atoms_of<D>(), BN = CbKeys<WP>::BN, KHT = CbKeys<WP>::KHT, NB = CbRowsDims<D>::NB;
  static constexpr int KS = D == 64 ? 8 : 4;
  static constexpr int kRing = 0;
  static constexpr int kKV = AT * BN * kRowBytes;              // K or V of a step
  static constexpr int kHl = 2 * kKV;                          // within a stage: hl of the step, by 64 queries
  static constexpr int kHlBlock = KHT * kCbRow * 4;
  static constexpr int kStage = kHl + cb_align(2 * kHlBlock);
  static constexpr int kBwStride = WP + 4;                     // floats: rows 16-byte aligned, in different banks
  static constexpr int kBw = kRing + KS * kStage;              // [128] rw rows
  static constexpr int kDh = kBw + kBlockM * kBwStride * 4;    // [128][65] drel_h
  static constexpr int kBars = kDh + kBlockM * 65 * 4;
  static constexpr int kMisc = kBars + kCbBars * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static_assert(kAlloc <= 232448, "shared memory");
  static_assert(KS * kStage >= NB * kBlockM * (WP + 1) * 4, "the drel_w sums are joined in the ring");
};

template <int D>
struct CbColsSmem {
  static constexpr int AT = atoms_of<D>(), KS = D == 64 ? 6 : 3;
  static constexpr bool kTmemA = D == 64;                      // k and v are read from TMEM, else from here
  static constexpr int kK = 0, kV = AT * kTileBytes, kRing = kTmemA ? 0 : 2 * AT * kTileBytes;
  static constexpr int kQ = AT * 64 * kRowBytes;               // Q or dO of a step
  static constexpr int kBias = 2 * kQ;                         // within a stage: W rows of rw, then the key tile's
  // grid rows of hl (128 consecutive keys touch at most 127 / W + 2 of them, and at most H), then -D
  static constexpr int kMaxRows = 68;
  static constexpr int kND = kBias + kMaxRows * kCbRow * 4;
  static constexpr int kStage = cb_align(kND + 256);
  static constexpr int kBars = kRing + KS * kStage;
  static constexpr int kMisc = kBars + kCbBars * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static_assert(kAlloc <= 232448, "shared memory");
};

struct CbCta {
  uint8_t* smem;
  uint64_t* bars;
  volatile int* abort_flag;
  uint32_t tbase;
};

// `on_a`, `on_step`, `all`: threads that arrive on kCbAFull, on a step's kCbPFull, on kCbJoin.
template <class SM>
__device__ __forceinline__ CbCta cb_setup(uint8_t* smem_raw, int warp, int on_a, int on_step, int all) {
  CbCta c;
  const uint32_t raw = smem_u32(smem_raw);
  c.smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  c.bars = reinterpret_cast<uint64_t*>(c.smem + SM::kBars);
  uint32_t* slot = reinterpret_cast<uint32_t*>(c.smem + SM::kMisc);
  c.abort_flag = reinterpret_cast<volatile int*>(c.smem + SM::kMisc + 4);
  static_assert(kCbBars <= 32, "one thread a barrier");
  if (threadIdx.x < kCbBars) {
    const int i = threadIdx.x;
    if (i == 0) *c.abort_flag = 0;
    const bool step = (i >= kCbPFull && i < kCbPFull + 3) || i == kCbSFree || i == kCbSFree + 1;
    mbar_init(&c.bars[i], i == kCbAFull ? on_a : (step ? on_step : (i == kCbJoin ? all : 1)));
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  c.tbase = *slot;
  return c;
}

__device__ __forceinline__ void cb_teardown(uint32_t tbase, int warp) {
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Waits until the ring's copies have landed, all `issued` of them: at once after a whole run, and with
// a limit if some role gave up.
template <int KS>
__device__ __forceinline__ void cb_drain(uint64_t* bars, int issued) {
  for (int i = max(0, issued - KS); i < issued; ++i)
    mbar_wait_budget(&bars[kCbRingFull + i % KS], (i / KS) & 1, kWaitBudgetCycles);
}

// A row of a [BH, N, D] tensor (zeros if !valid) on its way into TMEM as an A operand: this thread's lane, D / 2
// columns of packed pairs.  Reading A from TMEM leaves shared memory, which a 128 x 64 product
// would keep busy for 48 cycles a step of 16 (4 KB of A, 2 KB of B; the product takes 32), to B.
template <int D>
struct CbOwnRow {
  uint4 v[D / 8];
  __device__ __forceinline__ void load(const void* src, size_t row, bool valid) {
    #pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      v[c] = make_uint4(0u, 0u, 0u, 0u);
      if (valid) v[c] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(src) + row * D + 8 * c));
    }
  }
  __device__ __forceinline__ void to_tmem(uint32_t taddr) const {
    #pragma unroll
    for (int h = 0; h < D / 64; ++h) {
      uint32_t u[32];
      #pragma unroll
      for (int c = 0; c < 8; ++c)
        u[4 * c] = v[8 * h + c].x, u[4 * c + 1] = v[8 * h + c].y, u[4 * c + 2] = v[8 * h + c].z, u[4 * c + 3] = v[8 * h + c].w;
      tmem_st32(taddr + 32 * h, u);
    }
    tmem_wait_st();
  }
};

// What a CTA computes: a whole unit (a 128-row tile of a head), or a piece of one of the
// units past the last full wave of CTAs.
struct CbUnit {
  int bh, tile, i0, i1, piece;   // steps [i0, i1); piece < 0: whole
  __device__ __forceinline__ CbUnit(int block, int full, int split, int n_tiles, int steps) {
    int u = block, p = 0;
    piece = -1;
    i0 = 0;
    i1 = steps;
    if (block >= full && split > 1) {
      piece = block - full;
      u = full + piece / split;
      p = piece - (u - full) * split;
      i0 = static_cast<int>(static_cast<long long>(steps) * p / split);
      i1 = static_cast<int>(static_cast<long long>(steps) * (p + 1) / split);
    }
    bh = u / n_tiles;
    tile = u - bh * n_tiles;
  }
};

// ---------------------------------------------------------------------------
// prep: one CTA per (128 queries, head).  Reads 4 (H + W) bytes (fp32 bias) and
// 4 D of out and dO per query and writes 4 (H + W): bound by memory.  Half of the threads take rel_h, half
// rel_w, a query's row each: all of its loads are in flight at once, and every store is a run of queries.
constexpr int kCbPrepThreads = 2 * kBlockM;
constexpr float kLostLse = -1048576.f;

// A row of L <= 64 bias values in base 2, in fp32 (unused entries are left alone).
__device__ __forceinline__ void cb_load_row(const void* src, size_t at, int L, int fmt, float (&x)[64]) {
  if (fmt == kF32 && L % 4 == 0) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(src) + at);
    #pragma unroll
    for (int c = 0; c < 16; ++c)
      if (4 * c < L) {
        const float4 v = __ldg(p + c);
        x[4 * c] = bias2(v.x), x[4 * c + 1] = bias2(v.y), x[4 * c + 2] = bias2(v.z), x[4 * c + 3] = bias2(v.w);
      }
  } else if (fmt != kF32 && L % 8 == 0) {
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(src) + at);
    #pragma unroll
    for (int c = 0; c < 8; ++c)
      if (8 * c < L) {
        float v[8];
        unpack8(__ldg(p + c), v, fmt);
        #pragma unroll
        for (int e = 0; e < 8; ++e) x[8 * c + e] = bias2(v[e]);
      }
  } else {
    #pragma unroll
    for (int c = 0; c < 64; ++c)
      if (c < L) x[c] = bias2(load_elem(src, at + c, fmt));
  }
}

template <bool BF16, int D>
__global__ void __launch_bounds__(kCbPrepThreads) relpos_cb_prep_kernel(const CbArgs a) {
  constexpr int fmt = BF16 ? kBF16 : kF16, LANES = D / 8;
  const int bh = blockIdx.y, n0 = blockIdx.x * kBlockM;
  const int rows = min(kBlockM, a.N - n0);
  const size_t row0 = static_cast<size_t>(bh) * a.N + n0;
  const float inf = __int_as_float(0x7f800000);
  #pragma unroll
  for (int i = 0; i < kBlockM * LANES / kCbPrepThreads; ++i) {
    const int r = threadIdx.x / LANES + i * (kCbPrepThreads / LANES), c = threadIdx.x % LANES;
    float s = 0.f;
    if (r < rows) {
      const size_t at = (row0 + r) * D + 8 * c;
      float g[8], o[8];
      load8(a.dout, at, g, fmt);
      load8(a.out, at, o, a.out_fmt);
      #pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(g[e], o[e], s);
    }
    #pragma unroll
    for (int o = 1; o < LANES; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (c == 0) a.nD[static_cast<size_t>(bh) * a.n_blocks * 64 + n0 + r] = -s;
  }
  const bool is_w = threadIdx.x >= kBlockM;
  const int r = threadIdx.x & (kBlockM - 1), L = is_w ? a.W : a.H;
  float x[64];
  // rows past N take rw = 0 and hl = -inf, and so does a row without keys: lse = -inf, or so low (a mask of -1e9 on
  // every key) that its rounding leaves nothing of the probabilities (from 2^20 on they are off by 4 % and more)
  float off = 0.f;
  if (r < rows) {
    if (!is_w) off = a.lse[row0 + r];
    cb_load_row(is_w ? a.rel_w : a.rel_h, (row0 + r) * L, L, a.bias_fmt, x);
  }
  const bool none = !is_w && (r >= rows || off <= kLostLse);
  float* dst = (is_w ? a.rw : a.hl) + (static_cast<size_t>(bh) * a.n_blocks + 2 * blockIdx.x + (r >> 6)) * L * kCbRow;
  #pragma unroll
  for (int c = 0; c < 64; ++c)
    if (c < L) dst[cb_at(c, r & 63)] = none ? -inf : (r < rows ? x[c] - off : 0.f);
}

// ---------------------------------------------------------------------------
// rows.  What a step of 64 keys costs an SM: the products 384 cycles (head_dim 64), the exponents 256
// and the packed fp32 arithmetic about 400 on each scheduler.  It takes 870 to 1000: the chain from S through the
// exponents to dZ is not hidden by three steps in flight, and TMEM has no room for a fourth.  A CTA's start and
// end are 12,000 of its 68,000 cycles (64 steps).  Two CTAs an SM with one step in flight each were slower (249 us
// for the call above when one CTA took 213).
template <int WP, bool BF16, int D>
__global__ void __launch_bounds__(CbRowsDims<D>::kThreads, 1)
relpos_cb_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const CbArgs a) {
  using SM = CbRowsSmem<WP, D>;
  using DM = CbRowsDims<D>;
  constexpr int KHT = SM::KHT, BN = SM::BN, KS = SM::KS, AT = SM::AT, NB = DM::NB;
  constexpr int fmt = BF16 ? kBF16 : kF16;
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_launch_dependents();   // cols reads nothing of this kernel: its blocks fill the SMs that run out of these
  const int n_kv = (a.H + KHT - 1) / KHT;
  const CbUnit unit(blockIdx.x, a.rows_full, a.rows_split, a.n_tiles, n_kv);
  const int bh = unit.bh, steps = unit.i1 - unit.i0;
  // a softmax thread's rw row, a part by each group, and q or dO's: on their way during the set-up
  constexpr int kPart = (WP + NB - 1) / NB;
  CbOwnRow<D> own;
  float w[kPart], nDn = 0.f;
  if (warp >= 4) {
    const int wg = (warp >> 2) - 1, r = threadIdx.x & 127, n = unit.tile * kBlockM + r;
    const float* src = a.rw + (static_cast<size_t>(bh) * a.n_blocks + 2 * unit.tile + (r >> 6)) * a.W * kCbRow;
    if (wg < 2) own.load(wg == 0 ? a.q : a.dout, static_cast<size_t>(bh) * a.N + n, n < a.N);
    #pragma unroll
    for (int e = 0; e < kPart; ++e) {
      const int kw = wg * kPart + e;
      w[e] = kw < a.W ? __ldg(src + cb_at(kw, r & 63)) : -__int_as_float(0x7f800000);
    }
    nDn = __ldg(a.nD + static_cast<size_t>(bh) * a.n_blocks * 64 + n);
  }
  const CbCta cta = cb_setup<SM>(smem_raw, warp, 2 * kBlockM, kBlockM, NB * kBlockM);
  uint8_t* smem = cta.smem;
  uint64_t* bars = cta.bars;
  volatile int* abort_flag = cta.abort_flag;
  const uint32_t tbase = cta.tbase;
  int* status = a.status;
  auto stage = [&](int i) { return smem + SM::kRing + (i % KS) * SM::kStage; };

  if (warp < 4) {
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------------- TMA
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      const float* hl = a.hl + (static_cast<size_t>(bh) * a.n_blocks + 2 * unit.tile) * a.H * kCbRow;
      int i = 0;
      for (; i < steps; ++i) {
        if (!mbar_wait(&bars[kCbRingEmpty + i % KS], ((i / KS) & 1) ^ 1, abort_flag, status)) break;
        uint64_t* full = &bars[kCbRingFull + i % KS];
        const int kh0 = (unit.i0 + i) * KHT;
        const uint32_t hb = static_cast<uint32_t>(min(KHT, a.H - kh0)) * kCbRow * 4;
        mbar_arrive_expect_tx(full, 2 * SM::kKV + 2 * hb);
        #pragma unroll
        for (int t = 0; t < AT; ++t) {
          tma_load_4d(stage(i) + t * BN * kRowBytes, &tm_k, full, 64 * t, 0, kh0, bh);
          tma_load_4d(stage(i) + SM::kKV + t * BN * kRowBytes, &tm_v, full, 64 * t, 0, kh0, bh);
        }
        #pragma unroll
        for (int b = 0; b < 2; ++b)
          bulk_load(stage(i) + SM::kHl + b * SM::kHlBlock, hl + (static_cast<size_t>(b) * a.H + kh0) * kCbRow, hb, full);
      }
      cb_drain<KS>(bars, i);
    } else if (warp == 1) {
      // -------------------------------------------------------------- S and dP
      constexpr uint32_t id_s = idesc_f16(kBlockM, BN, fmt, fmt, 0, 0);   // both K-major
      const uint64_t d_ring = sdesc_sw128(smem_u32(smem + SM::kRing), 16, 1024);
      constexpr uint32_t kStep = SM::kStage >> 4, kV = SM::kKV >> 4, kB = (BN * kRowBytes) >> 4;
      bool ok = warp_all(mbar_wait(&bars[kCbAFull], 0, abort_flag, status));
      for (int i = 0; ok && i < steps; ++i) {
        // the buffer is free once the products of step i - NB are complete
        ok = (i < NB || mbar_wait(&bars[kCbAccDone + i % NB], (i / NB - 1) & 1, abort_flag, status)) &&
             mbar_wait(&bars[kCbRingFull + i % KS], (i / KS) & 1, abort_flag, status);
        ok = warp_all(ok);
        if (!ok) break;
        tc_fence_after();
        const uint64_t k = d_ring + (i % KS) * kStep;
        const uint32_t t = tbase + 128u * (i % NB);
        #pragma unroll
        for (int c = 0; c < D / 16; ++c)
          umma_ts_w(t, tbase + DM::tmQ + 8 * c, k + (c / 4) * kB + 2 * (c % 4), id_s, c > 0);
        #pragma unroll
        for (int c = 0; c < D / 16; ++c)
          umma_ts_w(t + 64, tbase + DM::tmDO + 8 * c, k + kV + (c / 4) * kB + 2 * (c % 4), id_s, c > 0);
        umma_commit_w(&bars[kCbSFull + i % NB]);
      }
      // every product issued here completes before TMEM is released
      umma_commit_w(&bars[kCbSDone]);
      mbar_wait_budget(&bars[kCbSDone], 0, kWaitBudgetCycles);
      __syncwarp();
    } else if (warp == 2) {
      // -------------------------------------------------------------- dq += dZ k
      constexpr uint32_t id_n = idesc_f16(kBlockM, 64, fmt, fmt, 0, 1);   // k N-major, 64 columns at a time
      const uint64_t d_ring = sdesc_sw128(smem_u32(smem + SM::kRing), 16, 1024);
      constexpr uint32_t kStep = SM::kStage >> 4, kB = (BN * kRowBytes) >> 4;
      for (int i = 0; i < steps; ++i) {
        if (!warp_all(mbar_wait(&bars[kCbPFull + i % NB], (i / NB) & 1, abort_flag, status))) break;
        tc_fence_after();
        #pragma unroll
        for (int t = 0; t < AT; ++t)
          #pragma unroll
          for (int c = 0; c < BN / 16; ++c)
            umma_ts_w(tbase + DM::tmDQ + 64 * t, tbase + 128 * (i % NB) + 8 * c,
                      d_ring + (i % KS) * kStep + t * kB + 128 * c, id_n, (i > 0 || c > 0) ? 1u : 0u);
        umma_commit_w(&bars[kCbAccDone + i % NB]);
        umma_commit_w(&bars[kCbRingEmpty + i % KS]);
      }
      // every product issued here completes before TMEM is read at the end or released
      umma_commit_w(&bars[kCbAllDone]);
      mbar_wait_budget(&bars[kCbAllDone], 0, kWaitBudgetCycles);
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- softmax threads
    const int H = a.H, W = a.W, N = a.N;
    const int wg = (warp >> 2) - 1, wq = warp & 3, r = wq * 32 + lane;
    const int n = unit.tile * kBlockM + r;
    const bool row_valid = n < N;
    const size_t row = static_cast<size_t>(bh) * N + n;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tbase + lanes + 128 * wg, tdP = tS + 64;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
    float* bw_row = reinterpret_cast<float*>(smem + SM::kBw) + r * SM::kBwStride;
    float* dh_row = reinterpret_cast<float*>(smem + SM::kDh) + r * 65;
    if (wg < 2) {
      own.to_tmem(tbase + lanes + (wg == 0 ? DM::tmQ : DM::tmDO));
      tc_fence_before();
      mbar_arrive(&bars[kCbAFull]);
    }
    #pragma unroll
    for (int e = 0; e < kPart; ++e)
      if (wg * kPart + e < WP) bw_row[wg * kPart + e] = w[e];
    const float2 nD = make_float2(nDn, nDn);
    float dRW[WP];
    #pragma unroll
    for (int kw = 0; kw < WP; ++kw) dRW[kw] = 0.f;
    auto join = [&](int phase) {
      mbar_arrive(&bars[kCbJoin]);
      return warp_all(mbar_wait(&bars[kCbJoin], phase, abort_flag, status));
    };
    bool ok = join(0);   // bw_row is complete
    for (int i = wg; ok && i < steps; i += NB) {
      const int kh0 = (unit.i0 + i) * KHT;
      ok = warp_all(mbar_wait(&bars[kCbRingFull + i % KS], (i / KS) & 1, abort_flag, status));
      if (!ok) break;
      float bh_[KHT];
      {
        // row g of the stage is grid row kh0 + g, whose chunks are permuted by its own number
        const float* hl = reinterpret_cast<const float*>(stage(i) + SM::kHl + (r >> 6) * SM::kHlBlock);
        #pragma unroll
        for (int g = 0; g < KHT; ++g)
          bh_[g] = (KHT == 1 || kh0 + g < H) ? hl[cb_at(kh0 + g, r & 63) - kh0 * kCbRow] : NEG_INF;
      }
      ok = warp_all(mbar_wait(&bars[kCbSFull + wg], (i / NB) & 1, abort_flag, status));
      if (!ok) break;
      tc_fence_after();
      float2 dRH[KHT];   // even and odd columns apart
      #pragma unroll
      for (int g = 0; g < KHT; ++g) dRH[g] = make_float2(0.f, 0.f);
      uint32_t us[2][16], up[2][16];
      tmem_ld16(tS, us[0]);
      tmem_ld16(tdP, up[0]);
      #pragma unroll
      for (int bb = 0; bb < BN / 16; ++bb) {
        const int cb = 16 * bb, cur = bb & 1;
        tmem_wait_ld();
        if (bb + 1 < BN / 16) {   // the next block's loads are in flight during this one
          tmem_ld16(tS + cb + 16, us[cur ^ 1]);
          tmem_ld16(tdP + cb + 16, up[cur ^ 1]);
        }
        uint32_t pk[8];
        #pragma unroll
        for (int k4 = 0; k4 < 16; k4 += 4) {
          const int g = (cb + k4) / WP, kw = (cb + k4) % WP;
          const float4 w4 = *reinterpret_cast<const float4*>(bw_row + kw);
          #pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const int k = k4 + e;
            const float2 w2 = e == 0 ? make_float2(w4.x, w4.y) : make_float2(w4.z, w4.w);
            const float2 s2 = make_float2(__uint_as_float(us[cur][k]), __uint_as_float(us[cur][k + 1]));
            const float2 dp = make_float2(__uint_as_float(up[cur][k]), __uint_as_float(up[cur][k + 1]));
            const float2 x = ffma2(s2, sl2, fadd2(w2, make_float2(bh_[g], bh_[g])));
            const float2 d = __fmul2_rn(make_float2(ex2_approx(x.x), ex2_approx(x.y)), fadd2(dp, nD));
            const float2 acc = fadd2(make_float2(dRW[kw + e], dRW[kw + e + 1]), d);
            dRW[kw + e] = acc.x;
            dRW[kw + e + 1] = acc.y;
            dRH[g] = fadd2(dRH[g], d);
            pk[k / 2] = pack_in(d.x, d.y, fmt);
          }
        }
        tmem_st8(tS + cb / 2, pk);   // dZ over columns of S that this thread has read
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars[kCbPFull + wg]);
      #pragma unroll
      for (int g = 0; g < KHT; ++g)
        if (KHT == 1 || kh0 + g < H) dh_row[i * KHT + g] = dRH[g].x + dRH[g].y;
    }
    if (ok) ok = warp_all(mbar_wait(&bars[kCbAllDone], 0, abort_flag, status));
    // drel_w: the groups' sums, side by side in the (now idle) ring, added as they are stored
    float* sum = reinterpret_cast<float*>(smem + SM::kRing);
    constexpr int kSum = kBlockM * (WP + 1);
    // an axis of length one (here, and not by a select where they are stored: that costs the 40x40 grid 1.2 %)
    if (W == 1) dRW[0] = 0.f;
    if (H == 1 && wg == 0) dh_row[0] = 0.f;
    if (ok) {
      #pragma unroll
      for (int kw = 0; kw < WP; ++kw) sum[wg * kSum + r * (WP + 1) + kw] = dRW[kw];
      ok = join(1);
    }
    if (ok) {
      const int n0 = unit.tile * kBlockM, rows = min(kBlockM, N - n0);
      const size_t row0 = static_cast<size_t>(bh) * N + n0;
      float* part = unit.piece < 0 ? nullptr : a.parts_rows + static_cast<size_t>(unit.piece) * kBlockM * (D + W);
      float* dw = part ? part + kBlockM * D : a.drel_w + row0 * W;
      const float* dh = reinterpret_cast<const float*>(smem + SM::kDh);
      const int h0 = unit.i0 * KHT, hn = min(H, unit.i1 * KHT) - h0;
      #pragma unroll 4
      for (int rr = warp - 4; rr < rows; rr += 4 * NB) {
        #pragma unroll
        for (int cc = 0; cc < WP; cc += 32) {
          const int c = cc + lane;
          if (c < W) {
            float v = sum[rr * (WP + 1) + c];
            #pragma unroll
            for (int b = 1; b < NB; ++b) v += sum[b * kSum + rr * (WP + 1) + c];
            dw[rr * W + c] = v;
          }
        }
        #pragma unroll
        for (int cc = 0; cc < 64; cc += 32)
          if (cc + lane < hn) a.drel_h[(row0 + rr) * H + h0 + cc + lane] = dh[rr * 65 + cc + lane];
      }
      // dq, 32 columns at a time
      tc_fence_after();
      for (int c0 = 32 * wg; c0 < D; c0 += 32 * NB) {
        uint32_t u[32];
        tmem_ld32(tbase + lanes + DM::tmDQ + c0, u);
        tmem_wait_ld();
        if (part) {   // column chunks of four, chunk by chunk: a warp's rows lie together
          #pragma unroll
          for (int c = 0; c < 8; ++c)
            reinterpret_cast<float4*>(part)[(c0 / 4 + c) * kBlockM + r] =
                make_float4(__uint_as_float(u[4 * c]), __uint_as_float(u[4 * c + 1]), __uint_as_float(u[4 * c + 2]),
                            __uint_as_float(u[4 * c + 3]));
        } else if (row_valid) {
          #pragma unroll
          for (int c = 0; c < 32; c += 8) {
            float v[8];
            #pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = a.scale * __uint_as_float(u[c + e]);
            store8(a.dq, row * D + c0 + c, v, a.grad_fmt);
          }
        }
      }
    }
  }
  cb_teardown(tbase, warp);
}

// ---------------------------------------------------------------------------
// cols.  128 consecutive keys of a head, whatever its grid, one per TMEM lane.  TMEM columns:
// S^T_b [128 b, 128 b + 64), dP^T_b 64 further, dv [256, 256 + D), dk, then (head_dim 64) k and v
// as packed pairs, and one P^T and dZ^T, which the threads hold in registers until the last step's have been
// read.  With 128 there is no room for either: k and v are read from shared memory, and P^T_b and dZ^T_b lie
// over S^T_b and dP^T_b, each thread's over columns that it has read.  Shared memory bounds it: a step's operands,
// bias and their reads keep it busy for about 900 cycles (head_dim 64; 1800 with 128, where TMEM has no room for k
// and v).  Deeper rings and other alignments of the bias measured the same.
template <bool BF16, int D>
__global__ void __launch_bounds__(kCbColsThreads, 1)
relpos_cb_cols_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const CbArgs a) {
  using SM = CbColsSmem<D>;
  constexpr int KS = SM::KS, AT = SM::AT;
  constexpr bool kTmemA = SM::kTmemA;
  constexpr bool kOver = D == 128;   // P^T and dZ^T over S^T and dP^T
  constexpr uint32_t tmDV = 256, tmDK = tmDV + D, tmK = tmDK + D, tmV = tmK + D / 2, tmP = tmV + D / 2;
  static_assert((kOver ? tmDK + D : tmP + 64) <= 512, "TMEM");
  // P^T of a buffer, dZ^T's distance from it, and the 16 queries c of both
  auto tm_p = [](int buf) { return kOver ? 128u * buf : tmP; };
  constexpr uint32_t kZ = kOver ? 64 : 32;
  auto at_step = [](int c) { return static_cast<uint32_t>(kOver ? 32 * (c >> 1) + 8 * (c & 1) : 8 * c); };
  constexpr int fmt = BF16 ? kBF16 : kF16;
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_steps = (a.N + 63) / 64;
  const CbUnit unit(blockIdx.x, a.cols_full, a.cols_split, a.n_tiles, n_steps);
  const int bh = unit.bh, steps = unit.i1 - unit.i0;
  CbOwnRow<D> own;   // k or v's row of a softmax thread of the first pair: on its way during the set-up
  if (kTmemA && warp >= 4 && warp < 12) {
    const int m = unit.tile * kBlockM + (threadIdx.x & 127);
    own.load(warp < 8 ? a.k : a.v, static_cast<size_t>(bh) * a.N + m, m < a.N);
  }
  const CbCta cta = cb_setup<SM>(smem_raw, warp, kTmemA ? 2 * kBlockM : 1, 2 * kBlockM, 1);
  uint8_t* smem = cta.smem;
  uint64_t* bars = cta.bars;
  volatile int* abort_flag = cta.abort_flag;
  const uint32_t tbase = cta.tbase;
  int* status = a.status;
  auto stage = [&](int i) { return smem + SM::kRing + (i % KS) * SM::kStage; };
  // grid rows of the tile's keys
  const int m0 = unit.tile * kBlockM, kh_first = m0 / a.W;
  const int kh_count = (min(m0 + kBlockM, a.N) - 1) / a.W - kh_first + 1;

  if (warp < 4) {
    regs_release<kCbColsRegsCtl>();
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA
      if (lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_do);
        if (!kTmemA) {
          mbar_arrive_expect_tx(&bars[kCbAFull], 2 * AT * kTileBytes);
          #pragma unroll
          for (int t = 0; t < AT; ++t) {
            tma_load_3d(smem + SM::kK + t * kTileBytes, &tm_k, &bars[kCbAFull], 64 * t, m0, bh);
            tma_load_3d(smem + SM::kV + t * kTileBytes, &tm_v, &bars[kCbAFull], 64 * t, m0, bh);
          }
        }
        const uint32_t wb = static_cast<uint32_t>(a.W) * kCbRow * 4, hb = static_cast<uint32_t>(kh_count) * kCbRow * 4;
        int i = 0;
        for (; i < steps; ++i) {
          if (!mbar_wait(&bars[kCbRingEmpty + i % KS], ((i / KS) & 1) ^ 1, abort_flag, status)) break;
          uint64_t* full = &bars[kCbRingFull + i % KS];
          const int blk = unit.i0 + i;
          const size_t at = static_cast<size_t>(bh) * a.n_blocks + blk;
          mbar_arrive_expect_tx(full, 2 * SM::kQ + wb + hb + 256);
          #pragma unroll
          for (int t = 0; t < AT; ++t) {
            tma_load_3d(stage(i) + t * 64 * kRowBytes, &tm_q, full, 64 * t, blk * 64, bh);
            tma_load_3d(stage(i) + SM::kQ + t * 64 * kRowBytes, &tm_do, full, 64 * t, blk * 64, bh);
          }
          bulk_load(stage(i) + SM::kBias, a.rw + at * a.W * kCbRow, wb, full);
          bulk_load(stage(i) + SM::kBias + wb, a.hl + (at * a.H + kh_first) * kCbRow, hb, full);
          bulk_load(stage(i) + SM::kND, a.nD + at * 64, 256, full);
        }
        cb_drain<KS>(bars, i);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- S^T and dP^T
      constexpr uint32_t id_s = idesc_f16(kBlockM, 64, fmt, fmt, 0, 0);   // both K-major
      const uint64_t d_k = sdesc_sw128(smem_u32(smem + SM::kK), 16, 1024);
      const uint64_t d_v = sdesc_sw128(smem_u32(smem + SM::kV), 16, 1024);
      const uint64_t d_ring = sdesc_sw128(smem_u32(smem + SM::kRing), 16, 1024);
      constexpr uint32_t kStep = SM::kStage >> 4, kDO = SM::kQ >> 4, kA = kTileBytes >> 4, kB = (64 * kRowBytes) >> 4;
      bool ok = warp_all(mbar_wait(&bars[kCbAFull], 0, abort_flag, status));
      for (int i = 0; ok && i < steps; ++i) {
        // the buffer is free once the products of step i - 2 are complete (kOver), or the threads have read it
        ok = (i < 2 || mbar_wait(&bars[(kOver ? kCbAccDone : kCbSFree) + (i & 1)], (i / 2 - 1) & 1, abort_flag, status)) &&
             mbar_wait(&bars[kCbRingFull + i % KS], (i / KS) & 1, abort_flag, status);
        ok = warp_all(ok);
        if (!ok) break;
        tc_fence_after();
        const uint64_t q = d_ring + (i % KS) * kStep;
        const uint32_t t = tbase + 128u * (i & 1);
        #pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint64_t b = q + (c / 4) * kB + 2 * (c % 4);
          if (kTmemA) umma_ts_w(t, tbase + tmK + 8 * c, b, id_s, c > 0);
          else umma_ss_w(t, d_k + (c / 4) * kA + 2 * (c % 4), b, id_s, c > 0);
        }
        #pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint64_t b = q + kDO + (c / 4) * kB + 2 * (c % 4);
          if (kTmemA) umma_ts_w(t + 64, tbase + tmV + 8 * c, b, id_s, c > 0);
          else umma_ss_w(t + 64, d_v + (c / 4) * kA + 2 * (c % 4), b, id_s, c > 0);
        }
        umma_commit_w(&bars[kCbSFull + (i & 1)]);
      }
      umma_commit_w(&bars[kCbSDone]);
      mbar_wait_budget(&bars[kCbSDone], 0, kWaitBudgetCycles);
      __syncwarp();
    } else if (warp == 2) {
      // ---------------------------------------------------------------- dv += P^T dO, dk += dZ^T q
      constexpr uint32_t id_n = idesc_f16(kBlockM, 64, fmt, fmt, 0, 1);   // q, dO N-major, 64 columns at a time
      const uint64_t d_ring = sdesc_sw128(smem_u32(smem + SM::kRing), 16, 1024);
      constexpr uint32_t kStep = SM::kStage >> 4, kDO = SM::kQ >> 4, kB = (64 * kRowBytes) >> 4;
      for (int i = 0; i < steps; ++i) {
        if (!warp_all(mbar_wait(&bars[kCbPFull + (i & 1)], (i >> 1) & 1, abort_flag, status))) break;
        tc_fence_after();
        const uint64_t q = d_ring + (i % KS) * kStep;
        const uint32_t p = tbase + tm_p(i & 1), z = p + kZ;
        #pragma unroll
        for (int t = 0; t < AT; ++t)
          #pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t acc = (i > 0 || c > 0) ? 1u : 0u;
            umma_ts_w(tbase + tmDV + 64 * t, p + at_step(c), q + kDO + t * kB + 128 * c, id_n, acc);
            umma_ts_w(tbase + tmDK + 64 * t, z + at_step(c), q + t * kB + 128 * c, id_n, acc);
          }
        umma_commit_w(&bars[kCbAccDone + (i & 1)]);
        umma_commit_w(&bars[kCbRingEmpty + i % KS]);
      }
      umma_commit_w(&bars[kCbAllDone]);
      mbar_wait_budget(&bars[kCbAllDone], 0, kWaitBudgetCycles);
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- softmax threads
    regs_claim<kCbColsRegsSmx>();
    // groups 0 and 2 take the even steps, 1 and 3 the odd ones, each 32 of a step's 64 queries
    const int wg = ((warp - 4) >> 2) & 1, half = (warp - 4) >> 3, wq = warp & 3, m = wq * 32 + lane;
    const bool key_valid = m0 + m < a.N;
    const int key = min(m0 + m, a.N - 1);   // lanes without a key compute what nobody stores
    const int kh = key / a.W, kw = key - kh * a.W;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tbase + lanes + 128 * wg, tdP = tS + 64;
    const int rw_at = kw * kCbRow, rw_x = kw & 7, hl_at = (a.W + kh - kh_first) * kCbRow, hl_x = kh & 7;
    const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
    if (kTmemA && half == 0) {
      own.to_tmem(tbase + lanes + (wg == 0 ? tmK : tmV));
      tc_fence_before();
      mbar_arrive(&bars[kCbAFull]);
    }
    bool ok = true;
    for (int i = wg; ok && i < steps; i += 2) {
      ok = warp_all(mbar_wait(&bars[kCbRingFull + i % KS], (i / KS) & 1, abort_flag, status));
      if (!ok) break;
      const float* bias = reinterpret_cast<const float*>(stage(i) + SM::kBias);
      const float* nDs = reinterpret_cast<const float*>(stage(i) + SM::kND);
      ok = warp_all(mbar_wait(&bars[kCbSFull + wg], (i >> 1) & 1, abort_flag, status));
      if (!ok) break;
      tc_fence_after();
      uint32_t us[2][16], up[2][16];
      #pragma unroll
      for (int bb = 0; bb < 2; ++bb) {
        tmem_ld16(tS + 32 * half + 16 * bb, us[bb]);
        tmem_ld16(tdP + 32 * half + 16 * bb, up[bb]);
      }
      tmem_wait_ld();
      if (!kOver) {   // S^T and dP^T of step i + 2 may go ahead
        tc_fence_before();
        mbar_arrive(&bars[kCbSFree + wg]);
      }
      uint32_t pp[2][8], pz[2][8];
      #pragma unroll
      for (int bb = 0; bb < 2; ++bb) {
        const int cb = 32 * half + 16 * bb;
        #pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const float4 w4 = *reinterpret_cast<const float4*>(bias + rw_at + ((((cb + k) >> 2) ^ rw_x) << 2));
          const float4 h4 = *reinterpret_cast<const float4*>(bias + hl_at + ((((cb + k) >> 2) ^ hl_x) << 2));
          const float4 d4 = *reinterpret_cast<const float4*>(nDs + cb + k);
          #pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 w2 = e == 0 ? make_float2(w4.x, w4.y) : make_float2(w4.z, w4.w);
            const float2 h2 = e == 0 ? make_float2(h4.x, h4.y) : make_float2(h4.z, h4.w);
            const float2 d2 = e == 0 ? make_float2(d4.x, d4.y) : make_float2(d4.z, d4.w);
            const float2 s2 = make_float2(__uint_as_float(us[bb][k + e]), __uint_as_float(us[bb][k + e + 1]));
            const float2 dp = make_float2(__uint_as_float(up[bb][k + e]), __uint_as_float(up[bb][k + e + 1]));
            const float2 x = ffma2(s2, sl2, fadd2(w2, h2));
            const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            const float2 z = __fmul2_rn(p, fadd2(dp, d2));
            pp[bb][(k + e) / 2] = pack_in(p.x, p.y, fmt);
            pz[bb][(k + e) / 2] = pack_in(z.x, z.y, fmt);
          }
        }
      }
      if (!kOver && i > 0) {   // the last step's P^T and dZ^T have been read
        ok = warp_all(mbar_wait(&bars[kCbAccDone + (wg ^ 1)], ((i - 1) >> 1) & 1, abort_flag, status));
        if (!ok) break;
        tc_fence_after();
      }
      #pragma unroll
      for (int bb = 0; bb < 2; ++bb) {
        tmem_st8(tbase + lanes + tm_p(wg) + at_step(2 * half + bb), pp[bb]);
        tmem_st8(tbase + lanes + tm_p(wg) + kZ + at_step(2 * half + bb), pz[bb]);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars[kCbPFull + wg]);
    }
    if (ok) ok = warp_all(mbar_wait(&bars[kCbAllDone], 0, abort_flag, status));
    if (ok) {
      // the even steps' groups store dv, the odd ones' dk, half of the columns each (tcgen05.ld is
      // warp-collective: every lane loads)
      tc_fence_after();
      const size_t row = static_cast<size_t>(bh) * a.N + m0 + m;
      float* part = unit.piece < 0 ? nullptr : a.parts_cols + static_cast<size_t>(unit.piece) * kBlockM * 2 * D + wg * kBlockM * D;
      void* dst = wg == 0 ? a.dv : a.dk;
      const float mul = wg == 0 ? 1.f : a.scale;
      #pragma unroll
      for (int hh = 0; hh < D / 64; ++hh) {
        const int h = half * (D / 64) + hh;
        uint32_t u[32];
        tmem_ld32(tbase + lanes + (wg == 0 ? tmDV : tmDK) + 32 * h, u);
        tmem_wait_ld();
        if (part) {
          #pragma unroll
          for (int c = 0; c < 8; ++c)
            reinterpret_cast<float4*>(part)[(8 * h + c) * kBlockM + m] =
                make_float4(__uint_as_float(u[4 * c]), __uint_as_float(u[4 * c + 1]), __uint_as_float(u[4 * c + 2]),
                            __uint_as_float(u[4 * c + 3]));
        } else if (key_valid) {
          #pragma unroll
          for (int c = 0; c < 32; c += 8) {
            float v[8];
            #pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = mul * __uint_as_float(u[c + e]);
            store8(dst, row * D + 32 * h + c, v, a.grad_fmt);
          }
        }
      }
    }
  }
  cb_teardown(tbase, warp);
  // rows may still run: this kernel must not be complete before it is, since what follows in the
  // stream waits for this one
  grid_wait_prerequisites();
}

// ---------------------------------------------------------------------------
// join: the pieces of a split unit added in order.  Blocks [0, rows_tail) in x take the rows kernel's
// units, the rest the cols kernel's; thread (r, y) of block y takes chunk 2 blockIdx.y + y of row r.
constexpr int kCbJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kCbJoinThreads) relpos_cb_join_kernel(const CbArgs a, int rows_tail) {
  const int r = threadIdx.x & 127, c = 2 * blockIdx.y + (threadIdx.x >> 7);
  const bool rows = static_cast<int>(blockIdx.x) < rows_tail;
  const int t = rows ? blockIdx.x : blockIdx.x - rows_tail;
  const int split = rows ? a.rows_split : a.cols_split;
  const int u = (rows ? a.rows_full : a.cols_full) + t;
  const int bh = u / a.n_tiles, n0 = (u - bh * a.n_tiles) * kBlockM;
  const int per = kBlockM * (rows ? D + a.W : 2 * D);
  const float* part = (rows ? a.parts_rows : a.parts_cols) + static_cast<size_t>(t) * split * per;
  const size_t row0 = static_cast<size_t>(bh) * a.N + n0;
  if (c < (rows ? D / 4 : D / 2)) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    #pragma unroll 4
    for (int p = 0; p < split; ++p) {
      const float4 v = reinterpret_cast<const float4*>(part + static_cast<size_t>(p) * per)[c * kBlockM + r];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    const bool first = c < D / 4;   // dq or dv, else dk
    const float mul = rows || !first ? a.scale : 1.f;
    void* dst = rows ? a.dq : (first ? a.dv : a.dk);
    if (n0 + r < a.N)
      st_grad4(dst, (row0 + r) * D + 4 * (first ? c : c - D / 4), mul * s.x, mul * s.y, mul * s.z, mul * s.w, a.grad_fmt);
  }
  if (!rows) return;
  const int n = min(kBlockM, a.N - n0) * a.W;
  for (int e = blockIdx.y * kCbJoinThreads + threadIdx.x; e < n; e += gridDim.y * kCbJoinThreads) {
    float s = 0.f;
    #pragma unroll 4
    for (int p = 0; p < split; ++p) s += part[static_cast<size_t>(p) * per + kBlockM * D + e];
    a.drel_w[row0 * a.W + e] = s;
  }
}

}  // namespace dera
