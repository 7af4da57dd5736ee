// Backward of the decomposed rel-pos projection, on tcgen05.
//
// With G[r][i] = drel[r][coord(r) - i + L - 1] (0 outside the row; coord is qh or qw), which
// holds a token's bias gradient by table row,
//   dq[r] = dq_in[r] + G_h[r] T_h + G_w[r] T_w,   dT = G^T q,
// so both are plain products once G is formed.  What bounds the pass is memory (4 (H + W)
// bytes of drel, and q, dq_in and dq, per token); the products take half as long.
//
// A CTA takes every gridDim.x-th tile of 128 tokens (of any heads: a token's coordinates are
// all that matters) and 64 columns of head_dim.  drel comes by bulk copies one tile ahead;
// eight warps form G in shared memory; one set of G serves both products, K-major (tokens by table rows) for dq
// and M-major for dT.  dT stays in TMEM over all of the CTA's tiles and leaves once, as a partial
// that relpos_pb_tables_kernel adds in a fixed order.
//
// Precision: tensor-core operands have 16 bits, drel has 32.  G is split into two bf16 terms,
// G = G1 + G2 to 2^-16 (a single one would leave 2^-8 in the tables' gradients, which
// are fp32 sums over all tokens).  bf16 and not fp16, because a gradient may have any size; fp16
// q and tables are split into two bf16 terms as well, exactly (11 bits = 8 + 3), and the product
// of the two small terms, 2^-16 of the whole, is left out.
#pragma once
#include "common.cuh"
#include "train.cuh"

namespace dera {

constexpr int kPbBuilders = 256, kPbThreads = 64 + kPbBuilders + 128;
constexpr int kPbAtoms = 2 * kTileBytes;   // a 128 x 128 operand of 16-bit values: two atoms of 64 columns

template <bool BF16>
struct PbSmem {
  static constexpr int kTerms = BF16 ? 1 : 2;                 // bf16 terms of q and the tables
  static constexpr int kT = 0;                                // [term][table] 128 rows x 64 columns
  static constexpr int kQ = kT + 2 * kTerms * kTileBytes;     // [term]
  static constexpr int kG = kQ + kTerms * kTileBytes;         // [term of G] two atoms
  static constexpr int kStg = kG + 2 * kPbAtoms;              // [table] drel of a tile, fp32
  static constexpr int kStgBytes = kBlockM * 64 * 4;
  static constexpr int kBars = kStg + 2 * kStgBytes;
  static constexpr int kMisc = kBars + 12 * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static_assert(kAlloc <= 232448, "shared memory");
};

enum : int {
  kPbStgFull = 0,   // [2] drel_h, drel_w of a tile landed
  kPbStgFree = 2,   // [2] the builders have read them
  kPbGFull = 4,     // G (and q) of one table written
  kPbMmaDone = 5,   // its products are complete
  kPbDqFull = 6,    // [2] dq of a tile is in TMEM
  kPbDqFree = 8,    // [2] and has been read
  kPbAllDone = 10,
  kPbBars = 11
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

template <bool BF16>
__global__ void __launch_bounds__(kPbThreads, 1) relpos_pb_kernel(const PbArgs a) {
  using SM = PbSmem<BF16>;
  constexpr int TERMS = SM::kTerms;
  extern __shared__ uint8_t smem_raw[];
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
      const int n = (i == kPbStgFree || i == kPbStgFree + 1 || i == kPbGFull)
                        ? kPbBuilders
                        : ((i == kPbDqFree || i == kPbDqFree + 1) ? kBlockM : 1);
      mbar_init(&bars[i], n);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *slot;   // dq of even and odd tiles [0, 64), [64, 128), dT_h [128, 192), dT_w [192, 256)

  if (warp == 0) {
    // ---------------------------------------------------------------- drel, one tile ahead
    if (lane == 0) {
      bool ok = true;
      for (int t = 0; ok && t < T; ++t) {
        const long long tile = tile_of(t);
        const int rows = rows_of(tile);
        for (int tb = 0; tb < 2; ++tb) {
          ok = mbar_wait(&bars[kPbStgFree + tb], (t & 1) ^ 1, abort_flag, status);
          if (!ok) break;
          const int L = tb == 0 ? a.H : a.W;
          const float* src = (tb == 0 ? a.drel_h : a.drel_w) + static_cast<size_t>(tile) * kBlockM * L;
          float* dst = reinterpret_cast<float*>(smem + SM::kStg + tb * SM::kStgBytes);
          // bulk copies go by 16 bytes; the last tile may end up to three floats further
          const int n = rows * L, whole = n & ~3;
          for (int e = whole; e < n; ++e) dst[e] = src[e];
          mbar_arrive_expect_tx(&bars[kPbStgFull + tb], static_cast<uint32_t>(whole) * 4);
          if (whole > 0) bulk_load(dst, src, static_cast<uint32_t>(whole) * 4, &bars[kPbStgFull + tb]);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t id_dq = idesc_f16(kBlockM, 64, kBF16, kBF16, 0, 1);   // G K-major, T N-major
    constexpr uint32_t id_dt = idesc_f16(kBlockM, 64, kBF16, kBF16, 1, 1);   // G^T M-major, q N-major
    constexpr uint32_t kG2 = kPbAtoms >> 4, kAtom = kTileBytes >> 4;
    const uint64_t d_g = sdesc_sw128(smem_u32(smem + SM::kG), 16, 1024);
    const uint64_t d_gt = sdesc_sw128(smem_u32(smem + SM::kG), kTileBytes, 1024);   // its two atoms lie along M
    const uint64_t d_q = sdesc_sw128(smem_u32(smem + SM::kQ), 16, 1024);
    bool ok = true;
    for (int s = 0; ok && s < 2 * T; ++s) {
      const int t = s >> 1, tb = s & 1;
      ok = warp_all(mbar_wait(&bars[kPbGFull], s & 1, abort_flag, status));
      if (ok && tb == 0 && t >= 2) ok = warp_all(mbar_wait(&bars[kPbDqFree + (t & 1)], ((t >> 1) - 1) & 1, abort_flag, status));
      if (!ok) break;
      tc_fence_after();
      const uint64_t d_t = sdesc_sw128(smem_u32(smem + SM::kT + tb * kTileBytes), 16, 1024);
      const uint32_t dq = tbase + 64 * (t & 1), dt = tbase + 128 + 64 * tb;
      const int ks = (2 * (tb == 0 ? a.H : a.W) + 14) / 16;   // 16-row steps over the table's 2L - 1 rows
      // G1 X1 + G2 X1 (+ G1 X2)
      for (int p = 0; p < 1 + TERMS; ++p) {
        const uint32_t g = p == 1 ? kG2 : 0, x = p == 2 ? 2 * kAtom : 0;
        for (int k = 0; k < ks; ++k)
          umma_ss_w(dq, d_g + g + (k / 4) * kAtom + 2 * (k % 4), d_t + x + 128 * k, id_dq, (tb > 0 || p > 0 || k > 0) ? 1u : 0u);
      }
      if (tb == 1) umma_commit_w(&bars[kPbDqFull + (t & 1)]);
      for (int p = 0; p < 1 + TERMS; ++p) {
        const uint32_t g = p == 1 ? kG2 : 0, x = p == 2 ? kAtom : 0;
        #pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_ss_w(dt, d_gt + g + 128 * k, d_q + x + 128 * k, id_dt, (t > 0 || p > 0 || k > 0) ? 1u : 0u);
      }
      umma_commit_w(&bars[kPbMmaDone]);
    }
    umma_commit_w(&bars[kPbAllDone]);
    mbar_wait_budget(&bars[kPbAllDone], 0, kWaitBudgetCycles);
    __syncwarp();
  } else if (warp < 2 + kPbBuilders / 32) {
    // ---------------------------------------------------------------- builders
    const int tid = threadIdx.x - 64;
    const int row0 = 16 * (warp - 2);   // a warp forms 16 rows of G, whose coordinates its lanes hold
    int qh = 0, qw = 0;
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
    // this thread's four 16-byte chunks of a tile's q
    uint4 qv[4];
    auto load_q = [&](int t) {
      const long long tile = tile_of(t);
      const int rows = rows_of(tile);
      #pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = tid + i * kPbBuilders, row = e >> 3, ch = e & 7;
        qv[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows)
          qv[i] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) +
                                                       (static_cast<size_t>(tile) * kBlockM + row) * a.D + c0 + 8 * ch));
      }
    };
    load_q(0);
    bool ok = true;
    for (int s = 0; ok && s < 2 * T; ++s) {
      const int t = s >> 1, tb = s & 1;
      const long long tile = tile_of(t);
      const int rows = rows_of(tile), L = tb == 0 ? a.H : a.W;
      // the previous table's products have read G, and its tile's q
      if (s > 0) ok = warp_all(mbar_wait(&bars[kPbMmaDone], (s - 1) & 1, abort_flag, status));
      if (ok) ok = warp_all(mbar_wait(&bars[kPbStgFull + tb], t & 1, abort_flag, status));
      if (!ok) break;
      if (tb == 0) {
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = tid + i * kPbBuilders;
          uint4 t1, t2;
          pb_terms<BF16>(qv[i], t1, t2);
          uint8_t* at = smem + SM::kQ + pb_off(e >> 3, 8 * (e & 7));
          *reinterpret_cast<uint4*>(at) = t1;
          if (TERMS == 2) *reinterpret_cast<uint4*>(at + kTileBytes) = t2;
        }
        if (t + 1 < T) load_q(t + 1);
      }
      if (tb == 0) {
        const long long g = tile * kBlockM + row0 + (lane & 15);
        const int n = static_cast<int>(g % a.N);
        qh = n / a.W;
        qw = n - qh * a.W;
      }
      const float* stg = reinterpret_cast<const float*>(smem + SM::kStg + tb * SM::kStgBytes);
      // pairs (i, i + 1) of the first 16 ks columns of this warp's 16 rows of G, row by row
      const int pairs = 8 * ((2 * L + 14) / 16);
      const uint32_t magic = 0xffffffffu / pairs + 1;   // e / pairs = umulhi(e, magic) for these e
      #pragma unroll 4
      for (int e = lane; e < 16 * pairs; e += 32) {
        const int rl = static_cast<int>(__umulhi(e, magic)), i = 2 * (e - rl * pairs), row = row0 + rl;
        const int k0 = __shfl_sync(0xffffffffu, tb == 0 ? qh : qw, rl) + L - 1 - i, k1 = k0 - 1;
        const float v0 = (row < rows && k0 >= 0 && k0 < L) ? stg[row * L + k0] : 0.f;
        const float v1 = (row < rows && k1 >= 0 && k1 < L) ? stg[row * L + k1] : 0.f;
        const uint32_t g1 = pack_bf16x2(v0, v1);
        const float2 h = unpack_in(g1, kBF16);
        uint8_t* at = smem + SM::kG + pb_off(row, i);
        *reinterpret_cast<uint32_t*>(at) = g1;
        *reinterpret_cast<uint32_t*>(at + kPbAtoms) = pack_bf16x2(v0 - h.x, v1 - h.y);
      }
      fence_proxy_async_smem();
      mbar_arrive(&bars[kPbGFull]);
      mbar_arrive(&bars[kPbStgFree + tb]);
    }
  } else {
    // ---------------------------------------------------------------- dq, and the tables at the end
    const int wq = warp & 3, r = wq * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    bool ok = true;
    for (int t = 0; ok && t < T; ++t) {
      const long long tile = tile_of(t);
      const bool valid = r < rows_of(tile);
      const size_t at = (static_cast<size_t>(tile) * kBlockM + r) * a.D + c0;
      ok = warp_all(mbar_wait(&bars[kPbDqFull + (t & 1)], (t >> 1) & 1, abort_flag, status));
      if (!ok) break;
      tc_fence_after();
      uint32_t u[2][32];
      tmem_ld32(tbase + lanes + 64 * (t & 1), u[0]);
      tmem_ld32(tbase + lanes + 64 * (t & 1) + 32, u[1]);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(&bars[kPbDqFree + (t & 1)]);
      if (valid) {
        #pragma unroll
        for (int h = 0; h < 2; ++h)
          #pragma unroll
          for (int c = 0; c < 32; c += 8) {
            float v[8];
            #pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(u[h][c + e]);
            if (a.dq_in) {
              float x[8];
              load8(a.dq_in, at + 32 * h + c, x, a.grad_fmt);
              #pragma unroll
              for (int e = 0; e < 8; ++e) v[e] += x[e];
            }
            store8(a.dq, at + 32 * h + c, v, a.grad_fmt);
          }
      }
    }
    if (ok) ok = warp_all(mbar_wait(&bars[kPbAllDone], 0, abort_flag, status));
    if (ok) {
      tc_fence_after();
      const int LH = 2 * a.H - 1, LW = 2 * a.W - 1;
      float* part = a.parts + static_cast<size_t>(blockIdx.x) * (LH + LW) * a.D + c0;
      #pragma unroll
      for (int tb = 0; tb < 2; ++tb)
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t u[32];
          tmem_ld32(tbase + lanes + 128 + 64 * tb + 32 * h, u);
          tmem_wait_ld();
          if (r < (tb == 0 ? LH : LW)) {
            float4* dst = reinterpret_cast<float4*>(part + static_cast<size_t>((tb == 0 ? 0 : LH) + r) * a.D + 32 * h);
            #pragma unroll
            for (int c = 0; c < 8; ++c)
              dst[c] = make_float4(__uint_as_float(u[4 * c]), __uint_as_float(u[4 * c + 1]), __uint_as_float(u[4 * c + 2]),
                                   __uint_as_float(u[4 * c + 3]));
          }
        }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 256);
  }
}

// The tables' gradients: the CTAs' partials added in a fixed order (thread (o, c) takes partials
// c, c + 8, ..., then the eight sums one after another).
__global__ void __launch_bounds__(256) relpos_pb_tables_kernel(const PbArgs a, int n_parts) {
  __shared__ float red[8][32];
  const int LH = 2 * a.H - 1, LW = 2 * a.W - 1, total = (LH + LW) * a.D;
  const int ol = threadIdx.x & 31, chunk = threadIdx.x >> 5, o = blockIdx.x * 32 + ol;   // total is a multiple of 32
  float acc = 0.f;
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
