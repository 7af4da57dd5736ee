// Backward of the decomposed rel-pos projection, on tcgen05.
//
// With G[r][i] = drel[r][coord(r) - i + L - 1] (0 outside the row; coord is qh or qw), which
// holds a token's bias gradient by table row,
//   dq[r] = dq_in[r] + G_h[r] T_h + G_w[r] T_w,   dT = G^T q,
// so both are plain products once G is formed.  What a pass cannot do without is its memory traffic: 4 (H + W)
// bytes of drel, and q, dq_in and dq, per token.
//
// A CTA takes every gridDim.x-th tile of 128 tokens (of any heads: a token's coordinates are
// all that matters) and 64 columns of head_dim.  drel comes by bulk copies, 64 tokens of one table at a
// time and ahead of its use; sixteen warps form G in shared memory, K-major (tokens by table rows); the same G,
// read M-major, serves dT.  G's two halves of 64 tokens are formed in turn, each while the products of the other
// run (dq's have M = 64 for this; dT's sum over tokens, 64 at a time).
//
// Measured on 96 heads of 64 x 64 tokens, head_dim 64, bf16 (337 MB): 150 us, 2.2 TB/s; 157 us with both halves
// formed together before the products.  No one part bounds it: without its products it takes 133 us, without forming
// G 119, without either 81 (timings only).  Forming G is some 1300 issue slots a scheduler and half, in
// chains of loads, conversions and stores that 48 registers a thread do not overlap further; splitting by truncation
// (fewer conversions), whole sectors of dq per store, one arrival a warp and G held in registers ahead
// of its buffer measured the same or slower.
//
// Precision: tensor-core operands have 16 bits, drel has 32.  G is split into three bf16 terms
// (what is left is 2^-24 of a value: the tables' gradients are fp32 sums over all tokens), of which the first two
// serve a 16-bit dq (2^-16; one term would leave 2^-8).  With two terms the tables' gradients were 2.5e-6 off
// (relative, the case above), with three 4e-7.  bf16 and not fp16, because a gradient may have any size; fp16
// q and tables are split into two bf16 terms as well, exactly (11 bits = 8 + 3); products of terms
// below 2^-16 of the whole are left out.  dT leaves TMEM after every tile and is summed in fp32 registers, where
// sums are rounded to nearest; the CTAs' partial sums are added in a fixed order by relpos_pb_tables_kernel.
#pragma once
#include "common.cuh"
#include "train.cuh"

namespace dera {

// warpgroups: control (warp 0 copies, warp 1 products), four that form G, two that take dq and dT
constexpr int kPbBuilders = 512, kPbThreads = 128 + kPbBuilders + 256;
constexpr int kPbLaunchRegs = 72, kPbRegsCtl = 64, kPbRegsBuild = 48, kPbRegsOut = 120;
static_assert(kPbRegsCtl + 4 * kPbRegsBuild + 2 * kPbRegsOut <= 7 * kPbLaunchRegs, "register split exceeds the launch pool");
constexpr int kPbAtoms = 2 * kTileBytes;   // a 128 x 128 operand of 16-bit values: two atoms of 64 columns

template <bool BF16>
struct PbSmem {
  static constexpr int kTerms = BF16 ? 1 : 2;                 // bf16 terms of q and the tables
  static constexpr int NS = BF16 ? 5 : 2;                     // staged halves of drel
  static constexpr int kT = 0;                                // [term][table] 128 rows x 64 columns
  static constexpr int kQ = kT + 2 * kTerms * kTileBytes;     // [term]
  static constexpr int kG = kQ + kTerms * kTileBytes;         // [three terms] two atoms
  static constexpr int kStg = kG + 3 * kPbAtoms;              // [NS] 64 rows of drel_h or drel_w, fp32
  static constexpr int kStgBytes = 64 * 64 * 4;
  static constexpr int kBars = kStg + NS * kStgBytes;
  static constexpr int kMisc = kBars + 28 * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static_assert(kAlloc <= 232448, "shared memory");
};

enum : int {
  kPbStgFull = 0,   // [5] a half of drel landed
  kPbStgFree = 5,   // [5] and has been read
  kPbGFull = 10,    // [half] 64 rows of G (and with the first table of q) written
  kPbMmaDone = 12,  // [half] their products are complete
  kPbDqFull = 14,   // [2] dq of a tile is in TMEM
  kPbDqFree = 16,   // [2] and has been read
  kPbDtFull = 18,   // [table][2] dT of a tile
  kPbDtFree = 22,   // [table][2]
  kPbAllDone = 26,  // every product is complete
  kPbBars = 27
};

// 16-bit operand element (row, i) of a K-major 128 x 128 tile, 128-byte swizzled.
__device__ __forceinline__ uint32_t pb_off(int row, int i) {
  return static_cast<uint32_t>((i >> 6) * kTileBytes + row * 128 + (((((i & 63) >> 3) ^ (row & 7))) << 4) + ((i & 7) << 1));
}

// Eight 16-bit values as bf16 terms: the value itself (bf16), or its two terms (fp16).
template <bool BF16>
__device__ __forceinline__ void pb_terms(const uint4& u, uint4& t1, uint4& t2) {
  if (BF16) {
    t1 = u;
    return;
  }
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t a[4], b[4];
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack_in(w[i], kF16);
    a[i] = pack_bf16x2(x.x, x.y);
    const float2 h = unpack_in(a[i], kBF16);
    b[i] = pack_bf16x2(x.x - h.x, x.y - h.y);
  }
  t1 = make_uint4(a[0], a[1], a[2], a[3]);
  t2 = make_uint4(b[0], b[1], b[2], b[3]);
}

// 4 rows of G (its three terms) from their staged drel rows of L floats: LPR lanes a row, a pair of columns
// (i, i + 1) each, ATOMS times 2 LPR columns.  The first is row r8 (0 or 4) of a swizzle
// group.  Lane l < 4 holds row l's coordinate, or one so large that the row comes out as zeros.
template <int LPR, int ATOMS>
__device__ __forceinline__ void pb_rows(const float* stg, uint8_t* g, int r8, int coord, int L, int lane) {
  constexpr int RPI = 32 / LPR;
  const int sub = lane / LPR, p = lane % LPR;
  const uint32_t n = static_cast<uint32_t>(L);
  // a row's values lie two apart from lane to lane: the lower lanes read their even one first, the
  // upper lanes their odd one, and the warp's 32 words are in different banks
  const int odd = LPR == 32 ? p >> 4 : 0;
  stg += L - 1 - 2 * p;
  g += (p & 3) * 4;
  #pragma unroll
  for (int it = 0; it < 4 / RPI; ++it) {
    const int rl = it * RPI + sub;
    const int c = __shfl_sync(0xffffffffu, coord, rl);
    const int k0 = c + L - 1 - 2 * p;
    const float* src = stg + rl * L + c;
    uint8_t* at = g + rl * 128 + (((p >> 2) ^ (r8 + rl)) << 4);
    #pragma unroll
    for (int a = 0; a < ATOMS; ++a) {
      const int k1 = 64 * a + odd, k2 = 64 * a + (odd ^ 1);
      const float x1 = static_cast<uint32_t>(k0 - k1) < n ? src[-k1] : 0.f;
      const float x2 = static_cast<uint32_t>(k0 - k2) < n ? src[-k2] : 0.f;
      const float v0 = odd ? x2 : x1, v1 = odd ? x1 : x2;
      const uint32_t g1 = pack_bf16x2(v0, v1);
      const float2 h = unpack_in(g1, kBF16);
      const float r0 = v0 - h.x, r1 = v1 - h.y;   // exact
      const uint32_t g2 = pack_bf16x2(r0, r1);
      const float2 m = unpack_in(g2, kBF16);
      *reinterpret_cast<uint32_t*>(at + a * kTileBytes) = g1;
      *reinterpret_cast<uint32_t*>(at + a * kTileBytes + kPbAtoms) = g2;
      *reinterpret_cast<uint32_t*>(at + a * kTileBytes + 2 * kPbAtoms) = pack_bf16x2(r0 - m.x, r1 - m.y);
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kPbThreads, 1) relpos_pb_kernel(const PbArgs a) {
  using SM = PbSmem<BF16>;
  constexpr int TERMS = SM::kTerms, NS = SM::NS;
  extern __shared__ uint8_t smem_raw[];
  grid_launch_dependents();   // relpos_pb_tables_kernel starts as these blocks run out
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM::kBars);
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + SM::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* status = a.status;
  const int c0 = 64 * blockIdx.y;   // this CTA's columns of head_dim
  const int T = static_cast<int>((a.n_tiles - 1 - blockIdx.x) / gridDim.x) + 1;
  auto tile_of = [&](int t) { return static_cast<long long>(blockIdx.x) + static_cast<long long>(t) * gridDim.x; };
  auto rows_of = [&](long long tile) {
    const long long left = a.tokens - tile * kBlockM;
    return static_cast<int>(left < kBlockM ? left : kBlockM);
  };
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kPbBars; ++i) {
      int n = 1;
      if (i >= kPbStgFree && i < kPbGFull + 2) n = kPbBuilders;
      else if (i == kPbDqFree || i == kPbDqFree + 1) n = 256;
      else if (i >= kPbDtFree && i < kPbDtFree + 4) n = 128;
      mbar_init(&bars[i], n);
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
  const uint32_t tbase = *slot;   // dq [128 parity + 64 half, + 64), dT [256 + 128 table + 64 parity, + 64)

  if (warp < 4) {
    regs_release<kPbRegsCtl>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------------- drel, half a tile of a table at a time
      bool ok = true;
      int j = 0;
      for (; j < 4 * T; ++j) {
        const long long tile = tile_of(j >> 2);
        const int tb = (j >> 1) & 1, half = j & 1, L = tb == 0 ? a.H : a.W;
        const int rows = max(0, min(64, rows_of(tile) - 64 * half));
        ok = mbar_wait(&bars[kPbStgFree + j % NS], ((j / NS) & 1) ^ 1, abort_flag, status);
        if (!ok) break;
        const float* src = (tb == 0 ? a.drel_h : a.drel_w) + (static_cast<size_t>(tile) * kBlockM + 64 * half) * L;
        float* dst = reinterpret_cast<float*>(smem + SM::kStg + (j % NS) * SM::kStgBytes);
        // bulk copies go by 16 bytes; the last rows may end up to three floats further
        const int n = rows * L, whole = n & ~3;
        for (int e = whole; e < n; ++e) dst[e] = src[e];
        mbar_arrive_expect_tx(&bars[kPbStgFull + j % NS], static_cast<uint32_t>(whole) * 4);
        if (whole > 0) bulk_load(dst, src, static_cast<uint32_t>(whole) * 4, &bars[kPbStgFull + j % NS]);
      }
      // the copies have landed: at once after a whole run, and with a limit if some role gave up
      for (int i = max(0, j - NS); i < j; ++i)
        mbar_wait_budget(&bars[kPbStgFull + i % NS], (i / NS) & 1, kWaitBudgetCycles);
    } else if (warp == 1) {
      // -------------------------------------------------------------- products
      constexpr uint32_t id_dq = idesc_f16(64, 64, kBF16, kBF16, 0, 1);          // G K-major, T N-major
      constexpr uint32_t id_dt = idesc_f16(kBlockM, 64, kBF16, kBF16, 1, 1);   // G^T M-major, q N-major
      constexpr uint32_t kGTerm = kPbAtoms >> 4, kAtom = kTileBytes >> 4, kHalf = kAtom / 2;
      const uint64_t d_g = sdesc_sw128(smem_u32(smem + SM::kG), 16, 1024);
      const uint64_t d_gt = sdesc_sw128(smem_u32(smem + SM::kG), kTileBytes, 1024);   // its two atoms lie along M
      const uint64_t d_q = sdesc_sw128(smem_u32(smem + SM::kQ), 16, 1024);
      for (int s = 0; s < 4 * T; ++s) {
        const int t = s >> 2, tb = (s >> 1) & 1, half = s & 1, buf = t & 1;
        bool ok = mbar_wait(&bars[kPbGFull + half], (s >> 1) & 1, abort_flag, status);
        if (t >= 2 && half == 0) {   // tile t - 2's dq and dT have been read
          const uint32_t ph = ((t >> 1) - 1) & 1;
          ok = ok && (tb == 1 || mbar_wait(&bars[kPbDqFree + buf], ph, abort_flag, status)) &&
               mbar_wait(&bars[kPbDtFree + 2 * tb + buf], ph, abort_flag, status);
        }
        if (!warp_all(ok)) break;
        tc_fence_after();
        const uint64_t d_t = sdesc_sw128(smem_u32(smem + SM::kT + tb * kTileBytes), 16, 1024);
        const uint32_t dq = tbase + 128 * buf + 64 * half, dt = tbase + 256 + 128 * tb + 64 * buf;
        const int ks = (2 * (tb == 0 ? a.H : a.W) + 14) / 16;   // 16-row steps over the table's 2L - 1 rows
        // dq and dT: G1 X1 + G2 X1 + G3 X1 (+ G1 X2 + G2 X2); a 16-bit dq does without G3 T1 and G2 T2
        #pragma unroll
        for (int p = 0; p < (TERMS == 1 ? 3 : 5); ++p) {
          if ((p == 2 || p == 4) && a.grad_fmt != kF32) continue;
          const uint32_t g = (p < 3 ? p : p - 3) * kGTerm + half * kHalf, x = p < 3 ? 0 : 2 * kAtom;
          for (int k = 0; k < ks; ++k)
            umma_ss_w(dq, d_g + g + (k / 4) * kAtom + 2 * (k % 4), d_t + x + 128 * k, id_dq,
                      (tb > 0 || p > 0 || k > 0) ? 1u : 0u);
        }
        if (tb == 1 && half == 1) umma_commit_w(&bars[kPbDqFull + buf]);
        #pragma unroll
        for (int p = 0; p < (TERMS == 1 ? 3 : 5); ++p) {
          const uint32_t g = (p < 3 ? p : p - 3) * kGTerm + half * kHalf, x = (p < 3 ? 0 : kAtom) + half * kHalf;
          #pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_ss_w(dt, d_gt + g + 128 * k, d_q + x + 128 * k, id_dt, (half > 0 || p > 0 || k > 0) ? 1u : 0u);
        }
        umma_commit_w(&bars[kPbMmaDone + half]);
        if (half == 1) umma_commit_w(&bars[kPbDtFull + 2 * tb + buf]);
      }
      // every product issued above completes before TMEM is released
      umma_commit_w(&bars[kPbAllDone]);
      mbar_wait_budget(&bars[kPbAllDone], 0, kWaitBudgetCycles);
      __syncwarp();
    }
  } else if (warp < 4 + kPbBuilders / 32) {
    // ---------------------------------------------------------------- builders
    regs_release<kPbRegsBuild>();
    const int tid = threadIdx.x - 128;
    const int row0 = 4 * (warp - 4);   // a warp forms 4 rows of each half of G
    // the tables' columns [c0, c0 + 64), rows past 2L - 1 as zeros
    for (int e = tid; e < 2 * kBlockM * 8; e += kPbBuilders) {
      const int tb = e >> 10, row = (e >> 3) & 127, ch = e & 7;
      const int L = tb == 0 ? a.H : a.W;
      uint4 u = make_uint4(0u, 0u, 0u, 0u), t1, t2;
      if (row < 2 * L - 1)
        u = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(tb == 0 ? a.th : a.tw) +
                                                 static_cast<size_t>(row) * a.D + c0 + 8 * ch));
      pb_terms<BF16>(u, t1, t2);
      uint8_t* at = smem + SM::kT + tb * kTileBytes + pb_off(row, 8 * ch);
      *reinterpret_cast<uint4*>(at) = t1;
      if (TERMS == 2) *reinterpret_cast<uint4*>(at + 2 * kTileBytes) = t2;
    }
    // this thread's 16-byte chunk of either half of a tile's q
    uint4 qv[2];
    auto load_q = [&](int t) {
      const long long tile = tile_of(t);
      const int rows = rows_of(tile);
      #pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int e = tid + i * kPbBuilders, row = e >> 3, ch = e & 7;
        qv[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows)
          qv[i] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) +
                                                       (static_cast<size_t>(tile) * kBlockM + row) * a.D + c0 + 8 * ch));
      }
    };
    load_q(0);
    bool ok = true;
    int qh[2] = {0, 0}, qw[2] = {0, 0};
    for (int t = 0; ok && t < T; ++t) {
      #pragma unroll
      for (int half = 0; half < 2; ++half) {
        const long long g = tile_of(t) * kBlockM + 64 * half + row0 + (lane & 3);
        const int n = static_cast<int>(g % a.N);
        qh[half] = n / a.W;
        qw[half] = n - qh[half] * a.W;
        if (g >= a.tokens) qh[half] = qw[half] = 1 << 20;   // a row past the last token: zeros
      }
      #pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const int s = 4 * t + i, tb = i >> 1, half = i & 1, L = tb == 0 ? a.H : a.W;
        // the last products of these 64 rows have read G (and q), and the half has landed
        ok = (s < 2 || mbar_wait(&bars[kPbMmaDone + half], ((s >> 1) - 1) & 1, abort_flag, status)) &&
             mbar_wait(&bars[kPbStgFull + s % NS], (s / NS) & 1, abort_flag, status);
        ok = warp_all(ok);
        if (!ok) break;
        const float* stg = reinterpret_cast<const float*>(smem + SM::kStg + (s % NS) * SM::kStgBytes) + row0 * L;
        uint8_t* g = smem + SM::kG + (64 * half + row0) * 128;
        const int c = tb == 0 ? (half == 0 ? qh[0] : qh[1]) : (half == 0 ? qw[0] : qw[1]), r8 = row0 & 7;
        if (L <= 8) pb_rows<8, 1>(stg, g, r8, c, L, lane);         // 15 table rows at most: 16 columns of G
        else if (L <= 16) pb_rows<16, 1>(stg, g, r8, c, L, lane);  // 31: 32
        else if (L <= 32) pb_rows<32, 1>(stg, g, r8, c, L, lane);  // 63: 64
        else pb_rows<32, 2>(stg, g, r8, c, L, lane);
        mbar_arrive(&bars[kPbStgFree + s % NS]);   // after the stores, which need every staged value in a register
        if (tb == 0) {
          const int e = tid + half * kPbBuilders;
          uint4 t1, t2;
          pb_terms<BF16>(half == 0 ? qv[0] : qv[1], t1, t2);
          uint8_t* at = smem + SM::kQ + pb_off(e >> 3, 8 * (e & 7));
          *reinterpret_cast<uint4*>(at) = t1;
          if (TERMS == 2) *reinterpret_cast<uint4*>(at + kTileBytes) = t2;
          if (half == 1 && t + 1 < T) load_q(t + 1);
        }
        fence_proxy_async_smem();
        mbar_arrive(&bars[kPbGFull + half]);
      }
    }
  } else {
    // ---------------------------------------------------------------- dq, half of the columns each, and one table's dT
    regs_claim<kPbRegsOut>();
    const int tb = (warp - 4 - kPbBuilders / 32) >> 2, wq = warp & 3, r = wq * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    float acc[64];
    #pragma unroll
    for (int e = 0; e < 64; ++e) acc[e] = 0.f;
    bool ok = true;
    for (int t = 0; ok && t < T; ++t) {
      const int buf = t & 1;
      const uint32_t ph = (t >> 1) & 1;
      const long long tile = tile_of(t);
      // a half's 64 rows lie in the first 16 lanes of each warp's 32; every other eight columns of a row are the
      // other lanes', so that a row's two threads touch whole 32-byte sectors
      const int row0 = 16 * wq + (lane & 15), rows = rows_of(tile);
      const size_t at = (static_cast<size_t>(tile) * kBlockM + row0) * a.D + c0 + 32 * tb + (lane & 16) / 2;
      const size_t at_half = 64 * static_cast<size_t>(a.D);
      // 16-bit dq_in: on its way while the products run
      const bool early = a.dq_in && a.grad_fmt != kF32;
      uint4 x[2][2] = {};
      if (early) {
        #pragma unroll
        for (int h = 0; h < 2; ++h)
          if (row0 + 64 * h < rows) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dq_in) + at + h * at_half);
            x[h][0] = p[0];
            x[h][1] = p[2];
          }
      }
      ok = warp_all(mbar_wait(&bars[kPbDqFull + buf], ph, abort_flag, status));
      if (!ok) break;
      tc_fence_after();
      #pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool valid = row0 + 64 * h < rows;
        #pragma unroll
        for (int c = 0; c < 32; c += 16) {
          const uint32_t from = tbase + lanes + 128 * buf + 64 * h + 32 * tb + c;
          uint32_t lo[8], hi[8];
          tmem_ld8(from, lo);
          tmem_ld8(from + 8, hi);
          tmem_wait_ld();
          if (h == 1 && c == 16) {
            tc_fence_before();
            mbar_arrive(&bars[kPbDqFree + buf]);
          }
          float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          if (early) unpack8(x[h][c / 16], v, a.grad_fmt);
          else if (a.dq_in && valid) load8(a.dq_in, at + h * at_half + c, v, a.grad_fmt);
          #pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t far = __shfl_sync(0xffffffffu, hi[e], lane & 15);
            v[e] += __uint_as_float(lane < 16 ? lo[e] : far);
          }
          if (valid) store8(a.dq, at + h * at_half + c, v, a.grad_fmt);
        }
      }
      ok = warp_all(mbar_wait(&bars[kPbDtFull + 2 * tb + buf], ph, abort_flag, status));
      if (!ok) break;
      tc_fence_after();
      #pragma unroll
      for (int h = 0; h < 64; h += 16) {
        uint32_t u[16];
        tmem_ld16(tbase + lanes + 256 + 128 * tb + 64 * buf + h, u);
        tmem_wait_ld();
        #pragma unroll
        for (int e = 0; e < 16; ++e) acc[h + e] += __uint_as_float(u[e]);
      }
      tc_fence_before();
      mbar_arrive(&bars[kPbDtFree + 2 * tb + buf]);
    }
    const int LH = 2 * a.H - 1, LW = 2 * a.W - 1;
    if (ok && r < (tb == 0 ? LH : LW)) {
      float* dst = a.parts + (static_cast<size_t>(blockIdx.x) * (LH + LW) + (tb == 0 ? 0 : LH) + r) * a.D + c0;
      #pragma unroll
      for (int e = 0; e < 64; e += 4)
        *reinterpret_cast<float4*>(dst + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// The tables' gradients: the CTAs' partials added in a fixed order (thread (o, c) takes partials
// c, c + 8, ..., then the eight sums one after another).
__global__ void __launch_bounds__(256) relpos_pb_tables_kernel(const PbArgs a, int n_parts) {
  __shared__ float red[8][32];
  const int LH = 2 * a.H - 1, LW = 2 * a.W - 1, total = (LH + LW) * a.D;
  const int ol = threadIdx.x & 31, chunk = threadIdx.x >> 5, o = blockIdx.x * 32 + ol;   // total is a multiple of 32
  float acc = 0.f;
  grid_wait_prerequisites();   // every partial is written
  #pragma unroll 8
  for (int p = chunk; p < n_parts; p += 8) acc += a.parts[static_cast<size_t>(p) * total + o];
  red[chunk][ol] = acc;
  __syncthreads();
  if (chunk == 0) {
    float v = red[0][ol];
    #pragma unroll
    for (int c = 1; c < 8; ++c) v += red[c][ol];
    if (o < LH * a.D) a.dth[o] = v;
    else a.dtw[o - LH * a.D] = v;
  }
}

}  // namespace dera
