// Backward of the attention with a compact bias (head_dim 64 or 128), on tcgen05.
//
// With Z = scale q k^T + rel_h[n, kh(m)] + rel_w[n, kw(m)], P = softmax(Z) recomputed from
// the forward's base-2 log-sum-exp, D[n] = dO[n] . out[n] and dZ = P * (dO v^T - D):
//   dv = P^T dO,  dk = scale dZ^T q,  dq = scale dZ k,
//   drel_h[n, kh] = sum_kw dZ[n, (kh, kw)],  drel_w[n, kw] = sum_kh dZ[n, (kh, kw)].
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
// In rows and cols two softmax warpgroups take the steps in turn, each with its own S and dP in
// TMEM: while one exponentiates step i the tensor core forms S and dP of step i + 1 for the
// other and adds step i - 1 to the accumulators.  With one group (one warp a scheduler)
// every wait of the chain TMEM load, exponent, TMEM store, product stood in the open.
#pragma once
#include <cfloat>

#include "common.cuh"
#include "train.cuh"

namespace dera {

constexpr int kCbThreads = 64 + 256;   // TMA warp, MMA warp, two softmax warpgroups
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
  kCbAFull = 0,                    // the CTA's own tiles landed
  kCbRingFull = 1,                 // [4]
  kCbRingEmpty = kCbRingFull + 4,  // [4]
  kCbSFull = kCbRingEmpty + 4,     // [2] S and dP of a step are in TMEM
  kCbPFull = kCbSFull + 2,         // [2] the warpgroup has read S and dP and written dZ (and P)
  kCbAccDone = kCbPFull + 2,       // [2] the products that read dZ (and P) are complete
  kCbAllDone = kCbAccDone + 2,     // every product is complete
  kCbJoin = kCbAllDone + 1,        // the softmax threads, at the end (count 256)
  kCbBars = kCbJoin + 1
};

constexpr int cb_align(int x) { return (x + 1023) / 1024 * 1024; }

template <int WP, int D>
struct CbRowsSmem {
  static constexpr int AT = atoms_of<D>(), BN = CbKeys<WP>::BN, KHT = CbKeys<WP>::KHT, KS = 4;
  static constexpr int kQ = 0, kDO = AT * kTileBytes, kRing = 2 * AT * kTileBytes;
  static constexpr int kKV = AT * BN * kRowBytes;              // K or V of a step
  static constexpr int kHl = 2 * kKV;                          // within a stage: hl of the step, by 64 queries
  static constexpr int kHlBlock = KHT * kCbRow * 4;
  static constexpr int kStage = kHl + cb_align(2 * kHlBlock);
  static constexpr int kBars = kRing + KS * kStage;
  static constexpr int kMisc = kBars + kCbBars * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static_assert(kAlloc <= 232448, "shared memory");
  static_assert(KS * kStage >= kBlockM * (WP + 1) * 4, "the drel_w sums are joined in the ring");
};

template <int D>
struct CbColsSmem {
  static constexpr int AT = atoms_of<D>(), KS = D == 64 ? 4 : 3;
  static constexpr int kK = 0, kV = AT * kTileBytes, kRing = 2 * AT * kTileBytes;
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

template <class SM>
__device__ __forceinline__ CbCta cb_setup(uint8_t* smem_raw, int warp) {
  CbCta c;
  const uint32_t raw = smem_u32(smem_raw);
  c.smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  c.bars = reinterpret_cast<uint64_t*>(c.smem + SM::kBars);
  uint32_t* slot = reinterpret_cast<uint32_t*>(c.smem + SM::kMisc);
  c.abort_flag = reinterpret_cast<volatile int*>(c.smem + SM::kMisc + 4);
  if (threadIdx.x == 0) {
    *c.abort_flag = 0;
    for (int i = 0; i < kCbBars; ++i) {
      const int n = (i >= kCbPFull && i < kCbPFull + 2) ? kBlockM : (i == kCbJoin ? 2 * kBlockM : 1);
      mbar_init(&c.bars[i], n);
    }
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
// 4 D of out and dO per query and writes 4.25 (H + W): bound by memory.
constexpr int kCbPrepThreads = 256;

template <bool BF16, int D>
__global__ void __launch_bounds__(kCbPrepThreads) relpos_cb_prep_kernel(const CbArgs a) {
  constexpr int fmt = BF16 ? kBF16 : kF16, LANES = D / 8, WARPS = kCbPrepThreads / 32;
  __shared__ float tr[64][kBlockM + 1];
  __shared__ float s_lse[kBlockM];
  const int bh = blockIdx.y, n0 = blockIdx.x * kBlockM;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = min(kBlockM, a.N - n0);
  const float inf = __int_as_float(0x7f800000);
  const size_t row0 = static_cast<size_t>(bh) * a.N + n0;
  if (threadIdx.x < kBlockM) {
    // a row without keys (lse = -inf) takes +inf, so that its P is exactly 0, and so does a row past N
    const float l = threadIdx.x < rows ? a.lse[row0 + threadIdx.x] : inf;
    s_lse[threadIdx.x] = l == -inf ? inf : l;
  }
  #pragma unroll 2
  for (int r = threadIdx.x / LANES; r < kBlockM; r += kCbPrepThreads / LANES) {
    const int c = threadIdx.x % LANES;
    float s = 0.f;
    if (r < rows) {
      const size_t at = (row0 + r) * D + 8 * c;
      const uint4 g = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.dout) + at));
      const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
      float o[8];
      if (a.out_fmt == kF32) {
        const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.out) + at);
        const float4 lo = __ldg(p), hi = __ldg(p + 1);
        o[0] = lo.x, o[1] = lo.y, o[2] = lo.z, o[3] = lo.w, o[4] = hi.x, o[5] = hi.y, o[6] = hi.z, o[7] = hi.w;
      } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.out) + at));
        const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 t = unpack_in(uw[i], fmt);
          o[2 * i] = t.x;
          o[2 * i + 1] = t.y;
        }
      }
      #pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = unpack_in(gw[i], fmt);
        s = fmaf(t.x, o[2 * i], s);
        s = fmaf(t.y, o[2 * i + 1], s);
      }
    }
    #pragma unroll
    for (int o = 1; o < LANES; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (c == 0) a.nD[static_cast<size_t>(bh) * a.n_blocks * 64 + n0 + r] = -s;
  }
  #pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int L = part == 0 ? a.H : a.W;
    const void* src = part == 0 ? a.rel_h : a.rel_w;
    float* dst = (part == 0 ? a.hl : a.rw) + (static_cast<size_t>(bh) * a.n_blocks + 2 * blockIdx.x) * L * kCbRow;
    __syncthreads();   // s_lse is written; the other part's rows are read
    #pragma unroll 4
    for (int r = warp; r < rows; r += WARPS)
      for (int c = lane; c < L; c += 32) tr[c][r] = load_elem(src, (row0 + r) * L + c, a.bias_fmt);
    __syncthreads();
    for (int c = warp; c < L; c += WARPS)
      #pragma unroll
      for (int r = lane; r < kBlockM; r += 32) {
        float v;
        if (part == 0) v = r < rows ? kLog2e * tr[c][r] - s_lse[r] : -inf;
        else v = r < rows ? kLog2e * tr[c][r] : 0.f;
        dst[(static_cast<size_t>(r >> 6) * L + c) * kCbRow + (r & 63)] = v;
      }
  }
}

// ---------------------------------------------------------------------------
// rows.  TMEM columns: S_b [128 b, 128 b + 64), dP_b 64 further, dZ_b [256 + 32 b, ...) as packed
// pairs, dq [320, 320 + D).
template <int WP, bool BF16, int D>
__global__ void __launch_bounds__(kCbThreads, 1)
relpos_cb_rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const CbArgs a) {
  using SM = CbRowsSmem<WP, D>;
  constexpr int KHT = SM::KHT, BN = SM::BN, KS = SM::KS, AT = SM::AT;
  constexpr int fmt = BF16 ? kBF16 : kF16;
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CbCta cta = cb_setup<SM>(smem_raw, warp);
  uint8_t* smem = cta.smem;
  uint64_t* bars = cta.bars;
  volatile int* abort_flag = cta.abort_flag;
  const uint32_t tbase = cta.tbase;
  int* status = a.status;
  const int n_kv = (a.H + KHT - 1) / KHT;
  const CbUnit unit(blockIdx.x, a.rows_full, a.rows_split, a.n_tiles, n_kv);
  const int bh = unit.bh, steps = unit.i1 - unit.i0;
  auto stage = [&](int i) { return smem + SM::kRing + (i % KS) * SM::kStage; };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      mbar_arrive_expect_tx(&bars[kCbAFull], 2 * AT * kTileBytes);
      #pragma unroll
      for (int t = 0; t < AT; ++t) {
        tma_load_3d(smem + SM::kQ + t * kTileBytes, &tm_q, &bars[kCbAFull], 64 * t, unit.tile * kBlockM, bh);
        tma_load_3d(smem + SM::kDO + t * kTileBytes, &tm_do, &bars[kCbAFull], 64 * t, unit.tile * kBlockM, bh);
      }
      const float* hl = a.hl + (static_cast<size_t>(bh) * a.n_blocks + 2 * unit.tile) * a.H * kCbRow;
      for (int i = 0; i < steps; ++i) {
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
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t id_s = idesc_f16(kBlockM, BN, fmt, fmt, 0, 0);   // S, dP: both K-major
    constexpr uint32_t id_n = idesc_f16(kBlockM, 64, fmt, fmt, 0, 1);   // dZ k: k N-major, 64 columns at a time
    const uint64_t d_q = sdesc_sw128(smem_u32(smem + SM::kQ), 16, 1024);
    const uint64_t d_do = sdesc_sw128(smem_u32(smem + SM::kDO), 16, 1024);
    const uint64_t d_ring = sdesc_sw128(smem_u32(smem + SM::kRing), 16, 1024);
    constexpr uint32_t kStep = SM::kStage >> 4, kV = SM::kKV >> 4, kA = kTileBytes >> 4, kB = (BN * kRowBytes) >> 4;
    auto issue_s = [&](int i) {
      const uint64_t k = d_ring + (i % KS) * kStep;
      const uint32_t t = tbase + 128u * (i & 1);
      #pragma unroll
      for (int c = 0; c < D / 16; ++c)
        umma_ss_w(t, d_q + (c / 4) * kA + 2 * (c % 4), k + (c / 4) * kB + 2 * (c % 4), id_s, c > 0);
      #pragma unroll
      for (int c = 0; c < D / 16; ++c)
        umma_ss_w(t + 64, d_do + (c / 4) * kA + 2 * (c % 4), k + kV + (c / 4) * kB + 2 * (c % 4), id_s, c > 0);
      umma_commit_w(&bars[kCbSFull + (i & 1)]);
    };
    bool ok = warp_all(mbar_wait(&bars[kCbAFull], 0, abort_flag, status));
    for (int i = 0; ok && i < min(2, steps); ++i) {
      ok = warp_all(mbar_wait(&bars[kCbRingFull + i % KS], 0, abort_flag, status));
      if (!ok) break;
      tc_fence_after();
      issue_s(i);
    }
    for (int i = 0; ok && i < steps; ++i) {
      ok = warp_all(mbar_wait(&bars[kCbPFull + (i & 1)], (i >> 1) & 1, abort_flag, status));
      if (!ok) break;
      if (i + 2 < steps) {   // first what the warpgroup that has just finished waits for next
        ok = warp_all(mbar_wait(&bars[kCbRingFull + (i + 2) % KS], ((i + 2) / KS) & 1, abort_flag, status));
        if (!ok) break;
        tc_fence_after();
        issue_s(i + 2);
      }
      tc_fence_after();
      #pragma unroll
      for (int t = 0; t < AT; ++t)
        #pragma unroll
        for (int c = 0; c < BN / 16; ++c)
          umma_ts_w(tbase + 320 + 64 * t, tbase + 256 + 32 * (i & 1) + 8 * c, d_ring + (i % KS) * kStep + t * kB + 128 * c,
                    id_n, (i > 0 || c > 0) ? 1u : 0u);
      umma_commit_w(&bars[kCbAccDone + (i & 1)]);
      umma_commit_w(&bars[kCbRingEmpty + i % KS]);
    }
    // every product issued above completes before TMEM is read at the end or released
    umma_commit_w(&bars[kCbAllDone]);
    mbar_wait_budget(&bars[kCbAllDone], 0, kWaitBudgetCycles);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax threads
    const int H = a.H, W = a.W, N = a.N;
    const int wg = (warp - 2) >> 2, wq = warp & 3, r = wq * 32 + lane;
    const int n = unit.tile * kBlockM + r;
    const bool row_valid = n < N;
    const size_t row = static_cast<size_t>(bh) * N + n;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tbase + lanes + 128 * wg, tdP = tS + 64, tdZ = tbase + lanes + 256 + 32 * wg;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
    float bw[WP], dRW[WP];
    {
      const float* src = a.rw + (static_cast<size_t>(bh) * a.n_blocks + 2 * unit.tile + (r >> 6)) * W * kCbRow + (r & 63);
      #pragma unroll
      for (int kw = 0; kw < WP; ++kw) {
        bw[kw] = kw < W ? __ldg(src + kw * kCbRow) : NEG_INF;
        dRW[kw] = 0.f;
      }
    }
    const float nDn = __ldg(a.nD + static_cast<size_t>(bh) * a.n_blocks * 64 + n);
    const float2 nD = make_float2(nDn, nDn);
    bool ok = true;
    for (int i = wg; ok && i < steps; i += 2) {
      const int kh0 = (unit.i0 + i) * KHT;
      ok = warp_all(mbar_wait(&bars[kCbRingFull + i % KS], (i / KS) & 1, abort_flag, status));
      if (!ok) break;
      float bh_[KHT];
      {
        const float* hl = reinterpret_cast<const float*>(stage(i) + SM::kHl + (r >> 6) * SM::kHlBlock) + (r & 63);
        #pragma unroll
        for (int g = 0; g < KHT; ++g) bh_[g] = (KHT == 1 || kh0 + g < H) ? hl[g * kCbRow] : NEG_INF;
      }
      ok = warp_all(mbar_wait(&bars[kCbSFull + wg], (i >> 1) & 1, abort_flag, status));
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
        for (int k = 0; k < 16; k += 2) {
          const int col = cb + k, g = col / WP, kw = col % WP;
          const float2 s2 = make_float2(__uint_as_float(us[cur][k]), __uint_as_float(us[cur][k + 1]));
          const float2 dp = make_float2(__uint_as_float(up[cur][k]), __uint_as_float(up[cur][k + 1]));
          const float2 b2 = fadd2(make_float2(bw[kw], bw[kw + 1]), make_float2(bh_[g], bh_[g]));
          const float2 x = ffma2(s2, sl2, b2);
          const float2 d = __fmul2_rn(make_float2(ex2_approx(x.x), ex2_approx(x.y)), fadd2(dp, nD));
          const float2 acc = fadd2(make_float2(dRW[kw], dRW[kw + 1]), d);
          dRW[kw] = acc.x;
          dRW[kw + 1] = acc.y;
          dRH[g] = fadd2(dRH[g], d);
          pk[k / 2] = pack_in(d.x, d.y, fmt);
        }
        if (bb == 0 && i >= 2) {   // this group's last dZ has been read before it is overwritten
          ok = warp_all(mbar_wait(&bars[kCbAccDone + wg], ((i >> 1) - 1) & 1, abort_flag, status));
          if (!ok) {
            tmem_wait_ld();
            break;
          }
          tc_fence_after();
        }
        tmem_st8(tdZ + cb / 2, pk);
      }
      if (!ok) break;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars[kCbPFull + wg]);
      if (row_valid) {
        #pragma unroll
        for (int g = 0; g < KHT; ++g)
          if (KHT == 1 || kh0 + g < H) a.drel_h[row * H + kh0 + g] = dRH[g].x + dRH[g].y;
      }
    }
    if (ok) ok = warp_all(mbar_wait(&bars[kCbAllDone], 0, abort_flag, status));
    // drel_w: the two groups' sums, added in the (now idle) ring and stored row by row
    float* sum = reinterpret_cast<float*>(smem + SM::kRing);
    auto join = [&](int phase) {
      mbar_arrive(&bars[kCbJoin]);
      return warp_all(mbar_wait(&bars[kCbJoin], phase, abort_flag, status));
    };
    if (ok && wg == 1) {
      #pragma unroll
      for (int kw = 0; kw < WP; ++kw) sum[r * (WP + 1) + kw] = dRW[kw];
    }
    if (ok) ok = join(0);
    if (ok && wg == 0) {
      #pragma unroll
      for (int kw = 0; kw < WP; ++kw) sum[r * (WP + 1) + kw] += dRW[kw];
    }
    if (ok) ok = join(1);
    if (ok) {
      const int n0 = unit.tile * kBlockM, rows = min(kBlockM, N - n0);
      float* part = unit.piece < 0 ? nullptr : a.parts_rows + static_cast<size_t>(unit.piece) * kBlockM * (D + W);
      float* dst = part ? part + kBlockM * D : a.drel_w + (static_cast<size_t>(bh) * N + n0) * W;
      for (int rr = warp - 2; rr < rows; rr += 8)
        for (int c = lane; c < W; c += 32) dst[rr * W + c] = sum[rr * (WP + 1) + c];
      // dq: each group half of the columns
      tc_fence_after();
      #pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        const int c0 = wg * (D / 2) + 32 * h;
        uint32_t u[32];
        tmem_ld32(tbase + lanes + 320 + c0, u);
        tmem_wait_ld();
        if (part) {   // column chunks of four, chunk by chunk: a warp's rows lie together
          #pragma unroll
          for (int c = 0; c < 8; ++c)
            reinterpret_cast<float4*>(part)[(c0 / 4 + c) * kBlockM + r] =
                make_float4(__uint_as_float(u[4 * c]), __uint_as_float(u[4 * c + 1]), __uint_as_float(u[4 * c + 2]),
                            __uint_as_float(u[4 * c + 3]));
        } else if (row_valid) {
          #pragma unroll
          for (int c = 0; c < 8; ++c)
            st_grad4(a.dq, row * D + c0 + 4 * c, a.scale * __uint_as_float(u[4 * c]),
                     a.scale * __uint_as_float(u[4 * c + 1]), a.scale * __uint_as_float(u[4 * c + 2]),
                     a.scale * __uint_as_float(u[4 * c + 3]), a.grad_fmt);
        }
      }
    }
  }
  cb_teardown(tbase, warp);
}

// ---------------------------------------------------------------------------
// cols.  128 consecutive keys of a head, whatever its grid, one per TMEM lane.  TMEM columns:
// S^T_b [128 b, 128 b + 64), dP^T_b 64 further.  head_dim 64: P^T_b [256 + 64 b, ...), dZ^T_b 32
// further, dv [384, 448), dk [448, 512).  head_dim 128: dv [256, 384), dk [384, 512), and P^T_b and
// dZ^T_b lie over the columns of S^T_b and dP^T_b that the threads have read, so the next step of
// a buffer waits until its products are complete.
template <bool BF16, int D>
__global__ void __launch_bounds__(kCbThreads, 1)
relpos_cb_cols_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const CbArgs a) {
  using SM = CbColsSmem<D>;
  constexpr int KS = SM::KS, AT = SM::AT;
  constexpr bool kOver = D == 128;   // P^T and dZ^T over S^T and dP^T
  constexpr uint32_t tmP = kOver ? 0 : 256, tmZ = kOver ? 64 : 288, kPStep = kOver ? 128 : 64;
  constexpr uint32_t tmDV = kOver ? 256 : 384, tmDK = tmDV + D;
  constexpr int fmt = BF16 ? kBF16 : kF16;
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CbCta cta = cb_setup<SM>(smem_raw, warp);
  uint8_t* smem = cta.smem;
  uint64_t* bars = cta.bars;
  volatile int* abort_flag = cta.abort_flag;
  const uint32_t tbase = cta.tbase;
  int* status = a.status;
  const int n_steps = (a.N + 63) / 64;
  const CbUnit unit(blockIdx.x, a.cols_full, a.cols_split, a.n_tiles, n_steps);
  const int bh = unit.bh, steps = unit.i1 - unit.i0;
  auto stage = [&](int i) { return smem + SM::kRing + (i % KS) * SM::kStage; };
  // grid rows of the tile's keys
  const int m0 = unit.tile * kBlockM, kh_first = m0 / a.W;
  const int kh_count = (min(m0 + kBlockM, a.N) - 1) / a.W - kh_first + 1;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_do);
      mbar_arrive_expect_tx(&bars[kCbAFull], 2 * AT * kTileBytes);
      #pragma unroll
      for (int t = 0; t < AT; ++t) {
        tma_load_3d(smem + SM::kK + t * kTileBytes, &tm_k, &bars[kCbAFull], 64 * t, m0, bh);
        tma_load_3d(smem + SM::kV + t * kTileBytes, &tm_v, &bars[kCbAFull], 64 * t, m0, bh);
      }
      const uint32_t wb = static_cast<uint32_t>(a.W) * kCbRow * 4, hb = static_cast<uint32_t>(kh_count) * kCbRow * 4;
      for (int i = 0; i < steps; ++i) {
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
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t id_s = idesc_f16(kBlockM, 64, fmt, fmt, 0, 0);   // S^T, dP^T: both K-major
    constexpr uint32_t id_n = idesc_f16(kBlockM, 64, fmt, fmt, 0, 1);   // q, dO N-major, 64 columns at a time
    const uint64_t d_k = sdesc_sw128(smem_u32(smem + SM::kK), 16, 1024);
    const uint64_t d_v = sdesc_sw128(smem_u32(smem + SM::kV), 16, 1024);
    const uint64_t d_ring = sdesc_sw128(smem_u32(smem + SM::kRing), 16, 1024);
    constexpr uint32_t kStep = SM::kStage >> 4, kDO = SM::kQ >> 4, kA = kTileBytes >> 4, kB = (64 * kRowBytes) >> 4;
    auto issue_s = [&](int i) {
      const uint64_t q = d_ring + (i % KS) * kStep;
      const uint32_t t = tbase + 128u * (i & 1);
      #pragma unroll
      for (int c = 0; c < D / 16; ++c)
        umma_ss_w(t, d_k + (c / 4) * kA + 2 * (c % 4), q + (c / 4) * kB + 2 * (c % 4), id_s, c > 0);
      #pragma unroll
      for (int c = 0; c < D / 16; ++c)
        umma_ss_w(t + 64, d_v + (c / 4) * kA + 2 * (c % 4), q + kDO + (c / 4) * kB + 2 * (c % 4), id_s, c > 0);
      umma_commit_w(&bars[kCbSFull + (i & 1)]);
    };
    auto next_s = [&](int i) -> bool {
      if (!warp_all(mbar_wait(&bars[kCbRingFull + i % KS], (i / KS) & 1, abort_flag, status))) return false;
      tc_fence_after();
      issue_s(i);
      return true;
    };
    bool ok = warp_all(mbar_wait(&bars[kCbAFull], 0, abort_flag, status));
    for (int i = 0; ok && i < min(2, steps); ++i) ok = next_s(i);
    for (int i = 0; ok && i < steps; ++i) {
      ok = warp_all(mbar_wait(&bars[kCbPFull + (i & 1)], (i >> 1) & 1, abort_flag, status));
      if (!ok) break;
      if (!kOver && i + 2 < steps && !(ok = next_s(i + 2))) break;
      tc_fence_after();
      const uint64_t q = d_ring + (i % KS) * kStep;
      const uint32_t p = tbase + tmP + kPStep * (i & 1), z = tbase + tmZ + kPStep * (i & 1);
      #pragma unroll
      for (int t = 0; t < AT; ++t)
        #pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t acc = (i > 0 || c > 0) ? 1u : 0u;
          umma_ts_w(tbase + tmDV + 64 * t, p + 8 * c, q + kDO + t * kB + 128 * c, id_n, acc);
          umma_ts_w(tbase + tmDK + 64 * t, z + 8 * c, q + t * kB + 128 * c, id_n, acc);
        }
      umma_commit_w(&bars[kCbAccDone + (i & 1)]);
      umma_commit_w(&bars[kCbRingEmpty + i % KS]);
      if (kOver && i + 2 < steps) {
        ok = warp_all(mbar_wait(&bars[kCbAccDone + (i & 1)], (i >> 1) & 1, abort_flag, status)) && next_s(i + 2);
      }
    }
    umma_commit_w(&bars[kCbAllDone]);
    mbar_wait_budget(&bars[kCbAllDone], 0, kWaitBudgetCycles);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax threads
    const int wg = (warp - 2) >> 2, wq = warp & 3, m = wq * 32 + lane;
    const bool key_valid = m0 + m < a.N;
    const int key = min(m0 + m, a.N - 1);   // lanes without a key compute what nobody stores
    const int kh = key / a.W, kw = key - kh * a.W;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tbase + lanes + 128 * wg, tdP = tS + 64;
    const uint32_t tP = tbase + lanes + tmP + kPStep * wg, tZ = tbase + lanes + tmZ + kPStep * wg;
    const int rw_at = kw * kCbRow, hl_at = (a.W + kh - kh_first) * kCbRow;
    const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
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
      tmem_ld16(tS, us[0]);
      tmem_ld16(tdP, up[0]);
      #pragma unroll
      for (int bb = 0; bb < 4; ++bb) {
        const int cb = 16 * bb, cur = bb & 1;
        tmem_wait_ld();
        if (bb < 3) {
          tmem_ld16(tS + cb + 16, us[cur ^ 1]);
          tmem_ld16(tdP + cb + 16, up[cur ^ 1]);
        }
        uint32_t pp[8], pz[8];
        #pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const float4 w4 = *reinterpret_cast<const float4*>(bias + rw_at + cb + k);
          const float4 h4 = *reinterpret_cast<const float4*>(bias + hl_at + cb + k);
          const float4 d4 = *reinterpret_cast<const float4*>(nDs + cb + k);
          #pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 w2 = e == 0 ? make_float2(w4.x, w4.y) : make_float2(w4.z, w4.w);
            const float2 h2 = e == 0 ? make_float2(h4.x, h4.y) : make_float2(h4.z, h4.w);
            const float2 d2 = e == 0 ? make_float2(d4.x, d4.y) : make_float2(d4.z, d4.w);
            const float2 s2 = make_float2(__uint_as_float(us[cur][k + e]), __uint_as_float(us[cur][k + e + 1]));
            const float2 dp = make_float2(__uint_as_float(up[cur][k + e]), __uint_as_float(up[cur][k + e + 1]));
            const float2 x = ffma2(s2, sl2, fadd2(w2, h2));
            const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            const float2 z = __fmul2_rn(p, fadd2(dp, d2));
            pp[(k + e) / 2] = pack_in(p.x, p.y, fmt);
            pz[(k + e) / 2] = pack_in(z.x, z.y, fmt);
          }
        }
        if (!kOver && bb == 0 && i >= 2) {   // this group's last P^T and dZ^T have been read
          ok = warp_all(mbar_wait(&bars[kCbAccDone + wg], ((i >> 1) - 1) & 1, abort_flag, status));
          if (!ok) {
            tmem_wait_ld();
            break;
          }
          tc_fence_after();
        }
        tmem_st8(tP + cb / 2, pp);
        tmem_st8(tZ + cb / 2, pz);
      }
      if (!ok) break;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars[kCbPFull + wg]);
    }
    if (ok) ok = warp_all(mbar_wait(&bars[kCbAllDone], 0, abort_flag, status));
    if (ok) {
      // group 0 stores dv, group 1 dk (tcgen05.ld is warp-collective: every lane loads)
      tc_fence_after();
      const size_t row = static_cast<size_t>(bh) * a.N + m0 + m;
      float* part = unit.piece < 0 ? nullptr : a.parts_cols + static_cast<size_t>(unit.piece) * kBlockM * 2 * D + wg * kBlockM * D;
      void* dst = wg == 0 ? a.dv : a.dk;
      const float mul = wg == 0 ? 1.f : a.scale;
      #pragma unroll
      for (int h = 0; h < D / 32; ++h) {
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
          for (int c = 0; c < 8; ++c)
            st_grad4(dst, row * D + 32 * h + 4 * c, mul * __uint_as_float(u[4 * c]), mul * __uint_as_float(u[4 * c + 1]),
                     mul * __uint_as_float(u[4 * c + 2]), mul * __uint_as_float(u[4 * c + 3]), a.grad_fmt);
        }
      }
    }
  }
  cb_teardown(tbase, warp);
}

// ---------------------------------------------------------------------------
// join: the pieces of a split unit added in order.  Blocks [0, rows_tail) take the rows kernel's
// units, the rest the cols kernel's; thread (r, y) takes the chunks y, y + 4, ... of row r.
template <int D>
__global__ void __launch_bounds__(512) relpos_cb_join_kernel(const CbArgs a, int rows_tail) {
  const int r = threadIdx.x & 127, y = threadIdx.x >> 7;
  const bool rows = static_cast<int>(blockIdx.x) < rows_tail;
  const int t = rows ? blockIdx.x : blockIdx.x - rows_tail;
  const int split = rows ? a.rows_split : a.cols_split;
  const int u = (rows ? a.rows_full : a.cols_full) + t;
  const int bh = u / a.n_tiles, n0 = (u - bh * a.n_tiles) * kBlockM;
  const int per = kBlockM * (rows ? D + a.W : 2 * D);
  const float* part = (rows ? a.parts_rows : a.parts_cols) + static_cast<size_t>(t) * split * per;
  const size_t row0 = static_cast<size_t>(bh) * a.N + n0;
  const bool valid = n0 + r < a.N;
  const int chunks = rows ? D / 4 : D / 2;
  for (int c = y; c < chunks; c += 4) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
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
    if (valid) st_grad4(dst, (row0 + r) * D + 4 * (first ? c : c - D / 4), mul * s.x, mul * s.y, mul * s.z, mul * s.w, a.grad_fmt);
  }
  if (!rows) return;
  const int n = min(kBlockM, a.N - n0) * a.W;
  for (int e = threadIdx.x; e < n; e += 512) {
    float s = 0.f;
    for (int p = 0; p < split; ++p) s += part[static_cast<size_t>(p) * per + kBlockM * D + e];
    a.drel_w[row0 * a.W + e] = s;
  }
}

}  // namespace dera
