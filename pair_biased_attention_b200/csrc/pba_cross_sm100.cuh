// pba_cross_sm100.cuh -- cross attention on the sm_100a tensor cores: queries
// of one sequence against an encoder's keys and values of another length,
// without a pair bias.
//
//     O_i = sum_j softmax_j( tau q_i.k_j ) v_j   over the keys j < k_len[b]
//                                                with key_mask[b][j] != 0
//
// Heads are grouped: head h reads the keys and values of head h / (H / Hkv).
// Beside pair-biased attention this is the second attention of a layer that
// conditions one sequence on another.
//
// Persistent: one CTA per SM walks the units u = blockIdx.x, + gridDim.x, ...;
// a unit is two 128-row query tiles of one (b, h), its keys come 128 at a time.
//   warps 0-3   softmax warpgroup of query tile 0 (thread t owns row t)
//   warps 4-7   softmax warpgroup of query tile 1
//   warp 8      TMA producer of Q (per unit) and of K and V
//   warps 9, 11 issue the tcgen05.mma of query tile 0 and 1 (9 allocates
//               Tensor Memory)
//   warp 10     takes out the keys that do not take part
// Without a bias nothing streams from HBM while a unit runs (K and V of a head
// stay in L2), so what bounds the kernel is the exponentials: per key tile and
// SM 2 x 128 x 128 of them, 2048 cycles of the exp2 unit, against 1050 cycles
// of products at D = 64.
//
// Tensor Memory (512 columns x 128 lanes of fp32), D <= 64:
//   [0,128) S0  [128,256) S1  [256,320) P0  [320,384) P1  [384,+D) O0  [448,+D) O1
// so that the next score tile is computed while the softmax warps work on this
// one.  D = 128: O0 and O1 take [256,512) and P lies over its own S, whose next
// tile then waits for the product with V; the two query tiles alternate.
//
// With fewer units than SMs a thread-block cluster shares a unit: each of its
// CTAs takes a share of the keys, leaves its O (not yet divided), maximum and
// sum in shared memory, and the cluster joins them row by row through
// distributed shared memory, always in the same order.
//
// Keys that do not take part cost the softmax nothing: warp 10 zeroes their
// rows of K and V in shared memory, so that what lies there, NaN included, does
// not matter, and in a tile that has any it fills one more column of K, 0 or
// -inf per key, which meets a column of ones beside Q in one more MMA of the
// score tile (K = 16).  Selecting among the 128 scores of a row in registers
// instead took 35 of 93 us at 2048 x 2048 keys, 32 heads, one key in ten masked.
//
// P is rounded to bf16, half a step of 2^-8 of each probability, because both
// operands of the product with V have one type; the sum l is taken over the
// unrounded fp32 values.  The output is then off by 1.3 to 1.4 times what its own
// rounding alone leaves.
//
// Measured at D = 64: 2 x 16 heads, 2048 queries on 8192 keys of which padding
// leaves four fifths, 165 us, 0.68 PFLOP/s, where the exponentials alone would
// take 100 us and the products 68; 256 units on 148 SMs, two waves for 1.73,
// account for most of the rest.  2 x 16 heads, 2048 x 2048, masked: D = 32 55 us,
// D = 64 59, D = 128 88 (0.78 PFLOP/s); on 8192 keys D = 128 287 us, 0.96 PFLOP/s.
// 4 heads, 256 x 8192, clusters of eight: 23 us, a CTA to a unit took 98.
#pragma once

#include <cooperative_groups.h>
#include <cuda.h>

#include "pba_ptx_more.cuh"

namespace pba {

constexpr int kXTile = 128;      // query rows and keys per tile
constexpr int kXQTiles = 2;      // query tiles per unit
constexpr int kXThreads = 384;
constexpr int kXWarpProducer = 8;
constexpr int kXWarpMma = 9;
constexpr int kXWarpFix = 10;
constexpr int kXWarpMma1 = 11;
constexpr int kXRegsSoftmax = 224;
constexpr int kXRegsOther = 56;
constexpr int kXRegSplitTotal = 256 * kXRegsSoftmax + 128 * kXRegsOther;
constexpr int kXMaxSplits = 8;  // CTAs of a cluster (the portable limit)
constexpr float kXLog2e = 1.4426950408889634f;
constexpr float kXLn2 = 0.6931471805599453f;

// Shared-memory tile of [kRows][D] bf16 as TMA and the tensor core see it: one
// or two slabs of at most 64 features (128 bytes) per row.
template <int D, int kRows = kXTile>
struct XTileLayout {
  static_assert(D == 32 || D == 64 || D == 128, "head dimension");
  static constexpr int kSlabs = D == 128 ? 2 : 1;
  static constexpr int kSlabCols = D / kSlabs;
  static constexpr int kRowBytes = kSlabCols * 2;
  static constexpr int kSwizzleMode = kRowBytes == 128 ? 2 : 4;  // 128- / 64-byte swizzle
  static constexpr int kAtomBytes = 8 * kRowBytes;
  static constexpr int kSlabBytes = kRows * kRowBytes;
  static constexpr int kBytes = kSlabs * kSlabBytes;
  static constexpr uint32_t kDescHi = smem_desc_hi(kAtomBytes, kSwizzleMode);
  // address step (16-byte units) of the K = 16 slice kk of a K-major operand
  static constexpr __host__ __device__ uint32_t k_step(int kk) {
    return uint32_t((kk / (kSlabCols / 16)) * kSlabBytes + (kk % (kSlabCols / 16)) * 32) / 16;
  }
  // and of an MN-major one (16 rows down)
  static constexpr __host__ __device__ uint32_t mn_step(int kk) { return uint32_t(kk * 16 * kRowBytes) / 16; }
  static __device__ __forceinline__ void zero_row(uint8_t *tile, int r) {
    // a row is the same 16-byte chunks whatever their swizzled order
#pragma unroll
    for (int i = 0; i < kSlabs * (kRowBytes / 16); ++i) {
      const int slab = i / (kRowBytes / 16), chunk = i % (kRowBytes / 16);
      *reinterpret_cast<uint4 *>(tile + slab * kSlabBytes + r * kRowBytes + chunk * 16) = make_uint4(0, 0, 0, 0);
    }
  }
  // The part-th kBox rows of the tile, from a map whose boxes have that many.
  template <int kBox>
  static __device__ __forceinline__ void load(void *dst, int part, const void *map, uint64_t *bar, int row, int h,
                                              int b, uint64_t policy) {
#pragma unroll
    for (int s = 0; s < kSlabs; ++s)
      tma_load_4d(static_cast<uint8_t *>(dst) + s * kSlabBytes + part * kBox * kRowBytes, map, bar, s * kSlabCols,
                  row + part * kBox, h, b, policy);
  }
};

struct CrossParams {
  CUtensorMap tm_q, tm_k, tm_v;  // (D, n, heads, B) bf16, box {min(D, 64), 128, 1, 1}
  int32_t B, H, group, Nq, Nk;   // group = H / Hkv
  int32_t n_qblocks, n_units;
  int32_t splits;                // CTAs of a cluster that share a unit (1: none does, and the grid is persistent)
  float tau;
  const int32_t *k_len;          // [B] or null
  const uint8_t *mask;           // [B][Nk] or null
  int64_t mask_sb;
  int32_t mask_vec4;             // mask rows readable as aligned 4-byte words
  uint16_t *out;
  int64_t out_sb, out_sh, out_sn;
  float *lse;
  int64_t lse_sb, lse_sh, lse_sn;
  int *err;
  uint64_t timeout_ns;
};

// Waits of a whole warp, which end as one: the phases of one barrier, or of two
// at once (both are asked before the first answer is used, which is what it
// takes when both are usually there).
__device__ __forceinline__ bool warp_wait(uint64_t *bar, int parity, const WaitCtl &wc) {
  return __all_sync(0xffffffffu, mbar_wait<false>(bar, parity & 1, wc));
}
__device__ __forceinline__ bool warp_wait2(uint64_t *a, int pa, uint64_t *b, int pb, const WaitCtl &wc) {
  const bool ra = mbar_try_wait(a, pa & 1), rb = mbar_try_wait(b, pb & 1);
  if (__all_sync(0xffffffffu, ra && rb)) return true;
  return warp_wait(a, pa, wc) && warp_wait(b, pb, wc);
}

// Keys of batch b that may take part: k_len, kept inside [0, Nk].
__device__ __forceinline__ int cross_keys(const int32_t *k_len, int b, int Nk) {
  return k_len == nullptr ? Nk : min(max(__ldg(k_len + b), 0), Nk);
}

// Which of the 32 kPer keys of the tile at key0 take part, asked by a whole
// warp: bit l of word e is key kPer l + e.  `bytes` is what cross_mask_bytes read
// (without a mask all keys before the end take part).
template <int kPer>
__device__ __forceinline__ uint32_t cross_mask_bytes(const uint8_t *row, bool vec4, int key0, int keys, int lane) {
  const int k = key0 + kPer * lane;
  uint32_t v = 0;
  if (row == nullptr) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) v |= uint32_t(k + e < keys) << (8 * e);
    return v;
  }
  if (kPer == 4 && vec4 && k + 3 < keys) return __ldg(reinterpret_cast<const uint32_t *>(row + k));
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    if (k + e < keys) v |= uint32_t(__ldg(row + k + e)) << (8 * e);
  return v;
}
template <int kPer>
struct KeepWords {
  uint32_t w[kPer];
  __device__ __forceinline__ bool all() const {
    uint32_t a = w[0];
#pragma unroll
    for (int e = 1; e < kPer; ++e) a &= w[e];
    return a == 0xFFFFFFFFu;
  }
};
template <int kPer>
__device__ __forceinline__ KeepWords<kPer> cross_keep(uint32_t bytes) {
  KeepWords<kPer> k;
#pragma unroll
  for (int e = 0; e < kPer; ++e) k.w[e] = __ballot_sync(0xffffffffu, ((bytes >> (8 * e)) & 0xFFu) != 0);
  return k;
}

// The column of ones beside Q and the columns of 0 and -inf beside K: [rows][16]
// bf16 tiles, K-major, 32-byte swizzle, of which only feature 0 is not 0.
struct XMaskTile {
  static constexpr int kRowBytes = 32;
  static constexpr uint32_t kDescHi = smem_desc_hi(256, 6);
  // feature 0 of row r: the 16-byte chunk's place in the row follows bit 2 of r
  static __device__ __forceinline__ uint16_t *at(uint8_t *tile, int r) {
    return reinterpret_cast<uint16_t *>(tile + r * kRowBytes + ((r >> 2) & 1) * 16);
  }
};
// By one warp: zeroes the rows of `tile` (of D features) whose keys do not take
// part, each lane its own.
template <int D, int kPer>
__device__ __forceinline__ void cross_zero_rows(uint8_t *tile, const KeepWords<kPer> &keep, int lane) {
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    if (!((keep.w[e] >> lane) & 1u)) XTileLayout<D, 32 * kPer>::zero_row(tile, kPer * lane + e);
}
// By one warp: the column of a tile's keys.
template <int kPer>
__device__ __forceinline__ void cross_mask_column(uint8_t *tile, const KeepWords<kPer> &keep, int lane) {
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    *XMaskTile::at(tile, kPer * lane + e) = (keep.w[e] >> lane) & 1u ? 0x0000u : 0xFF80u;
}

template <int D>
struct CrossLayout {
  using T = XTileLayout<D>;
  static constexpr bool kAlias = D == 128;  // P over S
  static constexpr int kKVStages = D == 128 ? 2 : 4;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kXQTiles * T::kBytes;
  static constexpr int kOffV = kOffK + kKVStages * T::kBytes;
  static constexpr int kOffOnes = kOffV + kKVStages * T::kBytes;
  static constexpr int kMaskBytes = kXTile * XMaskTile::kRowBytes;
  static constexpr int kOffMask = kOffOnes + kMaskBytes;                // [K stage]
  static constexpr int kOffPartial = kOffMask + kKVStages * kMaskBytes;  // [K stage]: the tile needs its column
  static constexpr int kOffBar = kOffPartial + 16;
  static_assert(kKVStages * 4 <= 16, "flags");
  static constexpr int kBarQFull = 0;
  static constexpr int kBarQEmpty = 1;
  static constexpr int kBarKFull = 2;
  static constexpr int kBarVFull = kBarKFull + kKVStages;
  static constexpr int kBarKEmpty = kBarVFull + kKVStages;
  static constexpr int kBarVEmpty = kBarKEmpty + kKVStages;
  static constexpr int kBarKReady = kBarVEmpty + kKVStages;  // keys that do not take part are out
  static constexpr int kBarVReady = kBarKReady + kKVStages;
  static constexpr int kBarSFull = kBarVReady + kKVStages;   // [w]
  static constexpr int kBarSFree = kBarSFull + kXQTiles;
  static constexpr int kBarPFull = kBarSFree + kXQTiles;
  static constexpr int kBarODone = kBarPFull + kXQTiles;
  static constexpr int kBarOFree = kBarODone + kXQTiles;
  static constexpr int kBarTurn = kBarOFree + kXQTiles;  // [w][warp of the warpgroup]
  static constexpr int kBarDrain = kBarTurn + kXQTiles * 4;
  static constexpr int kNumBars = kBarDrain + kXQTiles;
  static constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
  static constexpr int kOffAbort = kOffTmemSlot + 4;
  static constexpr int kBytes = kOffAbort + 4;
  static constexpr int kSmemAlloc = kBytes + 1024;  // room to align the base to 1024
  static_assert(kSmemAlloc <= 232448, "shared memory budget");
  // A unit's O and (maximum, sum) for the join, where K, V and the mask columns
  // were; the 16-byte chunks of a row in an order that spreads over the banks.
  static constexpr int kOffJoinMl = kOffK + kXQTiles * kXTile * D * 4;
  static_assert(kOffJoinMl + kXQTiles * kXTile * 8 <= kOffPartial, "join");
  static __device__ __forceinline__ float4 *join_o(uint8_t *base, int r, int chunk) {
    return reinterpret_cast<float4 *>(base + kOffK + (r * (D / 4) + (chunk ^ (r & 7))) * 16);
  }
  static __device__ __forceinline__ float2 *join_ml(uint8_t *base, int r) {
    return reinterpret_cast<float2 *>(base + kOffJoinMl + r * 8);
  }
  static constexpr __host__ __device__ uint32_t col_s(int w) { return uint32_t(w * kXTile); }
  static constexpr __host__ __device__ uint32_t col_p(int w) { return kAlias ? col_s(w) : 256u + w * 64; }
  static constexpr __host__ __device__ uint32_t col_o(int w) { return kAlias ? 256u + w * 128 : 384u + w * 64; }
};

// A CTA's part of a unit: nt key tiles from key0 on, of keys that end at `keys`.
struct CrossUnit {
  int b, h, q0, keys, key0, nt;
};
template <bool kShared>
__device__ __forceinline__ CrossUnit cross_unit(const CrossParams &p, int u) {
  const int qblk = u % p.n_qblocks, bh = u / p.n_qblocks;
  CrossUnit x;
  x.b = bh / p.H;
  x.h = bh - x.b * p.H;
  x.q0 = qblk * (kXQTiles * kXTile);
  x.keys = cross_keys(p.k_len, x.b, p.Nk);
  const int tiles = (x.keys + kXTile - 1) / kXTile;
  x.key0 = 0;
  x.nt = tiles;
  if (kShared) {
    const int per = (tiles + p.splits - 1) / p.splits, part = int(blockIdx.x) % p.splits;
    x.nt = max(0, min(per, tiles - part * per));
    x.key0 = part * per * kXTile;
  }
  return x;
}

// kShared: a cluster of p.splits CTAs shares each unit; otherwise the grid is
// persistent and p.splits is 1.
template <int D, bool kShared>
__global__ void __launch_bounds__(kXThreads, 1) pba_cross_sm100_kernel(const __grid_constant__ CrossParams p) {
  using L = CrossLayout<D>;
  using T = typename L::T;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffTmemSlot);
  int *abort_flag = reinterpret_cast<int *>(smem + L::kOffAbort);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int u_begin = kShared ? blockIdx.x / p.splits : blockIdx.x, u_step = kShared ? p.n_units : gridDim.x;
  // whole tiles of keys that all take part: nothing for warp 10 to do
  const bool fix = p.mask != nullptr || p.k_len != nullptr || p.Nk % kXTile != 0;
  volatile int *partial = reinterpret_cast<volatile int *>(smem + L::kOffPartial);

  if (threadIdx.x == 0) {
    mbar_init(&bars[L::kBarQFull], 1);
    mbar_init(&bars[L::kBarQEmpty], kXQTiles);  // a commit of each issuer, as for the tiles
    for (int s = 0; s < L::kKVStages; ++s) {
      mbar_init(&bars[L::kBarKFull + s], 1);
      mbar_init(&bars[L::kBarVFull + s], 1);
      mbar_init(&bars[L::kBarKEmpty + s], kXQTiles);
      mbar_init(&bars[L::kBarVEmpty + s], kXQTiles);
      mbar_init(&bars[L::kBarKReady + s], 32);
      mbar_init(&bars[L::kBarVReady + s], 32);
    }
    for (int w = 0; w < kXQTiles; ++w) {
      mbar_init(&bars[L::kBarSFull + w], 1);
      mbar_init(&bars[L::kBarSFree + w], kXTile);
      mbar_init(&bars[L::kBarPFull + w], kXTile);
      mbar_init(&bars[L::kBarODone + w], 1);
      mbar_init(&bars[L::kBarOFree + w], kXTile);
      mbar_init(&bars[L::kBarDrain + w], 1);
      for (int i = 0; i < 4; ++i) mbar_init(&bars[L::kBarTurn + w * 4 + i], 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  // zeros but for the ones
  for (int i = threadIdx.x; i < (1 + L::kKVStages) * L::kMaskBytes / 16; i += kXThreads)
    reinterpret_cast<uint4 *>(smem + L::kOffOnes)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  if (threadIdx.x < kXTile) *XMaskTile::at(smem + L::kOffOnes, threadIdx.x) = 0x3F80u;
  fence_proxy_async_smem();
  if (warp == kXWarpMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == kXWarpProducer && lane == 0) {
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl wc{abort_flag, p.err, p.timeout_ns};
  WaitCtl wc_drain = wc;  // clean-up waits: ignore the abort word, keep the time limit
  int drain_abort = 0;
  wc_drain.abort_flag = &drain_abort;

  if (warp >= 8) {
    setmaxnreg_dec<kXRegsOther>();
    if (warp == kXWarpProducer) {
      // ============================================================== Q/K/V TMA producer
      if (lane == 0) {
        const uint64_t pol_stream = l2_policy_evict_first();
        const uint64_t pol_keep = l2_policy_evict_last();
        bool ok = true;
        int kc = 0, vc = 0, uc = 0;  // K tiles, V tiles, Q loads issued
        auto load_k = [&](const CrossUnit &un, int j) -> bool {
          const int s = kc % L::kKVStages;
          if (kc >= L::kKVStages && !mbar_wait(&bars[L::kBarKEmpty + s], ((kc / L::kKVStages) - 1) & 1, wc))
            return false;
          mbar_arrive_expect_tx(&bars[L::kBarKFull + s], T::kBytes);
          T::template load<kXTile>(smem + L::kOffK + s * T::kBytes, 0, &p.tm_k, &bars[L::kBarKFull + s],
                                   un.key0 + j * kXTile, un.h / p.group, un.b, pol_keep);
          ++kc;
          return true;
        };
        auto load_v = [&](const CrossUnit &un, int j) -> bool {
          const int s = vc % L::kKVStages;
          if (vc >= L::kKVStages && !mbar_wait(&bars[L::kBarVEmpty + s], ((vc / L::kKVStages) - 1) & 1, wc))
            return false;
          mbar_arrive_expect_tx(&bars[L::kBarVFull + s], T::kBytes);
          T::template load<kXTile>(smem + L::kOffV + s * T::kBytes, 0, &p.tm_v, &bars[L::kBarVFull + s],
                                   un.key0 + j * kXTile, un.h / p.group, un.b, pol_keep);
          ++vc;
          return true;
        };
        for (int u = u_begin; u < p.n_units && ok; u += u_step) {
          const CrossUnit un = cross_unit<kShared>(p, u);
          if (un.nt == 0) continue;
          // Q slot: free once the last score MMAs of the previous unit are done
          if (uc > 0) ok = mbar_wait(&bars[L::kBarQEmpty], (uc - 1) & 1, wc);
          if (!ok) break;
          mbar_arrive_expect_tx(&bars[L::kBarQFull], kXQTiles * T::kBytes);
          for (int w = 0; w < kXQTiles; ++w)
            T::template load<kXTile>(smem + L::kOffQ + w * T::kBytes, 0, &p.tm_q, &bars[L::kBarQFull],
                                     un.q0 + w * kXTile, un.h, un.b, pol_stream);
          ++uc;
          ok = load_k(un, 0);
          for (int j = 0; j < un.nt && ok; ++j) {
            if (j + 1 < un.nt) ok = load_k(un, j + 1);
            if (ok) ok = load_v(un, j);
          }
        }
        if (!ok) {
          // every copy already issued lands before the CTA exits; slot s was
          // armed (n - s + stages - 1) / stages times after n issues
          if (uc) mbar_wait(&bars[L::kBarQFull], (uc - 1) & 1, wc_drain);
          for (int s = 0; s < L::kKVStages; ++s) {
            const int ak = (kc - s + L::kKVStages - 1) / L::kKVStages, av = (vc - s + L::kKVStages - 1) / L::kKVStages;
            if (ak > 0) mbar_wait(&bars[L::kBarKFull + s], (ak - 1) & 1, wc_drain);
            if (av > 0) mbar_wait(&bars[L::kBarVFull + s], (av - 1) & 1, wc_drain);
          }
        }
      }
    } else if (warp == kXWarpMma || warp == kXWarpMma1) {
      // ============================================================== MMA issuers
      // One warp per query tile: a single one that served both in turn made
      // each tile's products wait for the other's softmax.  The whole warp
      // walks through the loop and one lane issues, which keeps the operand
      // descriptors in uniform registers; under a branch for one lane every
      // instruction took some 85 cycles to issue.
      const int w = __shfl_sync(0xffffffffu, int(warp == kXWarpMma1), 0);
      constexpr uint32_t idesc_s = idesc_bf16_f32(kXTile, kXTile, false);
      constexpr uint32_t idesc_o = idesc_bf16_f32(kXTile, D, true);
      const uint32_t tbase = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t tS = tbase + L::col_s(w), tP = tbase + L::col_p(w), tO = tbase + L::col_o(w);
      const uint32_t smem0 = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
      const uint32_t q_lo = smem_desc_lo(smem0 + L::kOffQ + w * T::kBytes, 16);
      bool ok = true;
      int kc = 0, vc = 0;  // K and V tiles consumed (= score and P V tiles issued)
      int uc = 0;
      auto wait = [&](int bar, int parity) -> bool { return warp_wait(&bars[bar], parity, wc); };
      auto wait2 = [&](int a, int pa, int b, int pb) -> bool { return warp_wait2(&bars[a], pa, &bars[b], pb, wc); };
      auto issue_s = [&](int s) {
        const uint32_t k_lo = smem_desc_lo(smem0 + L::kOffK + s * T::kBytes, 16);
        const uint32_t ones_lo = smem_desc_lo(smem0 + L::kOffOnes, 16);
        const uint32_t mask_lo = smem_desc_lo(smem0 + L::kOffMask + s * L::kMaskBytes, 16);
        const bool masked = fix && partial[s] != 0;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_ss(tS, desc_join(q_lo + T::k_step(kk), T::kDescHi), desc_join(k_lo + T::k_step(kk), T::kDescHi),
                        idesc_s, kk > 0 ? 1u : 0u);
          if (masked)
            mma_bf16_ss(tS, desc_join(ones_lo, XMaskTile::kDescHi), desc_join(mask_lo, XMaskTile::kDescHi), idesc_s,
                        1u);
          tc_commit(&bars[L::kBarSFull + w]);
          tc_commit(&bars[L::kBarKEmpty + s]);
        }
        __syncwarp();
      };
      auto issue_pv = [&](int s, bool first) {
        const uint32_t v_lo = smem_desc_lo(smem0 + L::kOffV + s * T::kBytes, T::kSlabBytes);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kXTile / 16; ++kk)
            mma_bf16_ts(tO, tP + kk * 8, desc_join(v_lo + T::mn_step(kk), T::kDescHi), idesc_o,
                        (!first || kk > 0) ? 1u : 0u);
          tc_commit(&bars[L::kBarODone + w]);
          tc_commit(&bars[L::kBarVEmpty + s]);
        }
        __syncwarp();
      };
      // the next score tile, once its keys are there and S (at D = 128: P
      // over it) has been read
      auto next_s = [&]() -> bool {
        const int s = kc % L::kKVStages;
        const int full = (fix ? L::kBarKReady : L::kBarKFull) + s;
        if (kc > 0 ? !wait2(full, kc / L::kKVStages, L::kBarSFree + w, kc - 1) : !wait(full, kc / L::kKVStages))
          return false;
        if (L::kAlias && vc > 0 && !wait(L::kBarODone + w, vc - 1)) return false;
        tc_fence_after_sync();
        issue_s(s);
        ++kc;
        return true;
      };
      auto q_done = [&]() {
        if (elect_one()) tc_commit(&bars[L::kBarQEmpty]);
        __syncwarp();
      };
      // D <= 64: S(j+1) before P V(j), so that the next scores are there when
      // the softmax has written P(j).  D = 128 (P over S): after it.
      for (int u = u_begin; u < p.n_units && ok; u += u_step) {
        const int nt = cross_unit<kShared>(p, u).nt;
        if (nt == 0) continue;
        ok = wait(L::kBarQFull, uc) && next_s();
        if (!ok) break;
        if (nt == 1) q_done();
        for (int j = 0; j < nt && ok; ++j) {
          const bool has_next = j + 1 < nt;
          const int sv = vc % L::kKVStages;
          if (!L::kAlias && has_next) {
            if (!(ok = next_s())) break;
            // after the unit's last score MMAs the Q slot can be refilled
            if (j + 2 == nt) q_done();
          }
          if (!(ok = wait2((fix ? L::kBarVReady : L::kBarVFull) + sv, vc / L::kKVStages, L::kBarPFull + w, vc))) break;
          // the first P V of a unit overwrites O: the epilogue of the
          // previous unit must have read it
          if (j == 0 && uc > 0 && !(ok = wait(L::kBarOFree + w, uc - 1))) break;
          tc_fence_after_sync();
          issue_pv(sv, j == 0);
          ++vc;
          if (L::kAlias && has_next) {
            if (!(ok = next_s())) break;
            if (j + 2 == nt) q_done();
          }
        }
        ++uc;
      }
      // every MMA issued above completes before Tensor Memory is released
      if (elect_one()) tc_commit(&bars[L::kBarDrain + w]);
      __syncwarp();
      mbar_wait<false>(&bars[L::kBarDrain + w], 0, wc_drain);
    } else if (warp == kXWarpFix && fix) {
      // ============================================================== keys that do not take part
      bool ok = true;
      int kc = 0, vc = 0;
      auto wait = [&](int bar, int parity) -> bool { return warp_wait(&bars[bar], parity, wc); };
      auto fix_k = [&](const KeepWords<4> &keep) -> bool {
        const int s = kc % L::kKVStages;
        if (!wait(L::kBarKFull + s, kc / L::kKVStages)) return false;
        const bool any = !keep.all();
        if (any) {
          cross_zero_rows<D>(smem + L::kOffK + s * T::kBytes, keep, lane);
          cross_mask_column(smem + L::kOffMask + s * L::kMaskBytes, keep, lane);
          fence_proxy_async_smem();
        }
        if (lane == 0) partial[s] = any;
        __syncwarp();
        mbar_arrive(&bars[L::kBarKReady + s]);
        ++kc;
        return true;
      };
      auto fix_v = [&](const KeepWords<4> &keep) -> bool {
        const int s = vc % L::kKVStages;
        if (!wait(L::kBarVFull + s, vc / L::kKVStages)) return false;
        if (!keep.all()) {
          cross_zero_rows<D>(smem + L::kOffV + s * T::kBytes, keep, lane);
          fence_proxy_async_smem();
        }
        mbar_arrive(&bars[L::kBarVReady + s]);
        ++vc;
        return true;
      };
      // in the order of the loads: K runs one tile ahead of V
      for (int u = u_begin; u < p.n_units && ok; u += u_step) {
        const CrossUnit un = cross_unit<kShared>(p, u);
        if (un.nt == 0) continue;
        const uint8_t *mrow = p.mask != nullptr ? p.mask + int64_t(un.b) * p.mask_sb : nullptr;
        auto bytes = [&](int j) { return cross_mask_bytes<4>(mrow, p.mask_vec4, un.key0 + j * kXTile, un.keys, lane); };
        KeepWords<4> keep = cross_keep<4>(bytes(0));
        uint32_t next = un.nt > 1 ? bytes(1) : 0u;
        ok = fix_k(keep);
        for (int j = 0; j < un.nt && ok; ++j) {
          const KeepWords<4> v_keep = keep;
          if (j + 1 < un.nt) {
            keep = cross_keep<4>(next);
            if (j + 2 < un.nt) next = bytes(j + 2);
            ok = fix_k(keep);
          }
          if (ok) ok = fix_v(v_keep);
        }
      }
    }
  } else {
    // ================================================================ softmax warpgroups
    setmaxnreg_inc<kXRegsSoftmax>();
    const int w = warp >> 2;          // query tile
    const int t = threadIdx.x & 127;  // row inside the tile
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + L::col_s(w);
    const uint32_t tP = tmem + lane_base + L::col_p(w);
    const uint32_t tO = tmem + lane_base + L::col_o(w);
    const float c_s = p.tau * kXLog2e;  // scores to log2 units
    // A row keeps its running maximum until a tile's exceeds it by more than 8
    // in log2 units, so most tiles skip the rescale of O; the kept maximum is
    // used for P and l alike, so the result is unchanged.
    const float slack = fminf(8.f / c_s, 1e30f);
    uint64_t *my_turn = &bars[L::kBarTurn + w * 4 + (warp & 3)];
    uint64_t *other_turn = &bars[L::kBarTurn + (1 - w) * 4 + (warp & 3)];
    bool ok = true;
    int gt = 0;  // key tiles processed (all units)
    for (int u = u_begin; u < p.n_units && ok; u += u_step) {
      const CrossUnit un = cross_unit<kShared>(p, u);
      float m_cur = -INFINITY;  // maximum used for P and l (raw scores)
      float neg_m = 0.f;        // -m_cur in log2 units (0 while there is none)
      float l = 0.f;
      for (int j = 0; j < un.nt && ok; ++j, ++gt) {
        // the loads below are warp-collective: a warp leaves its waits as one
        ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars[L::kBarSFull + w], gt & 1, wc));
        if (!ok) break;
        tc_fence_after_sync();
        uint32_t sreg[kXTile];
#pragma unroll
        for (int c = 0; c < kXTile / 32; ++c)
          tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sreg[c * 32]));
        tmem_wait_ld();
        reg_fence(sreg);
        tc_fence_before_sync();
        mbar_arrive(&bars[L::kBarSFree + w]);

        // tile maximum: eight independent chains
        float m8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) m8[i] = fmaxf(__uint_as_float(sreg[2 * i]), __uint_as_float(sreg[2 * i + 1]));
#pragma unroll
        for (int i = 8; i < kXTile / 2; ++i)
          m8[i & 7] = max3f(m8[i & 7], __uint_as_float(sreg[2 * i]), __uint_as_float(sreg[2 * i + 1]));
        const float mx = max3f(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
        const bool need = mx > m_cur + slack;
        float alpha = 1.f;
        if (need) {
          alpha = (m_cur == -INFINITY) ? 0.f : ex2_approx((m_cur - mx) * c_s);
          l *= alpha;
          m_cur = mx;
          neg_m = -mx * c_s;
        }
        // The exponentials' turn.  Warps w and w + 4 share a scheduler and its
        // exp2 unit; left alone they fall into step, both in their exponentials
        // and then both out of them.  Taking turns, one loads, masks and finds
        // maxima while the other keeps the unit busy.
        if (w == 1 || gt > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait<false>(my_turn, w == 1 ? (gt & 1) : ((gt - 1) & 1), wc));
          if (!ok) break;
        }
        const float2 cs2 = make_float2(c_s, c_s), negm2 = make_float2(neg_m, neg_m);
        uint32_t pk[kXTile / 2];
        float2 ls[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < kXTile / 2; ++i) {
          const float2 a = ffma2(make_float2(__uint_as_float(sreg[2 * i]), __uint_as_float(sreg[2 * i + 1])), cs2,
                                 negm2);
          const float2 pv = make_float2(ex2_approx(a.x), ex2_approx(a.y));
          ls[i & 3] = fadd2(ls[i & 3], pv);
          pk[i] = pack_bf16x2(pv.x, pv.y);
        }
        if (lane == 0) mbar_arrive(other_turn);
        const float2 lsum2 = fadd2(fadd2(ls[0], ls[1]), fadd2(ls[2], ls[3]));
        l += lsum2.x + lsum2.y;

        // P(j) overwrites what P V(j-1) read, possibly the last one of the
        // previous unit, and the rescale needs its sum
        if (gt > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars[L::kBarODone + w], (gt - 1) & 1, wc));
          if (!ok) break;
          tc_fence_after_sync();
          if (j > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(tO + c, o);
              tmem_wait_ld();
              reg_fence(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tO + c, o);
            }
          }
        }
#pragma unroll
        for (int c = 0; c < kXTile / 2; c += 32) tmem_st32(tP + c, *reinterpret_cast<uint32_t(*)[32]>(&pk[c]));
        tmem_wait_st();
        tc_fence_before_sync();
        mbar_arrive(&bars[L::kBarPFull + w]);
      }

      // -------------------------------------------------------------- epilogue
      if (un.nt > 0 && ok) {
        ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars[L::kBarODone + w], (gt - 1) & 1, wc));
        tc_fence_after_sync();
      }
      if (kShared) {
        // the unit's only one of this CTA: K and V are done with once both
        // warpgroups are here, and their memory takes O for the join.  A warp
        // that gave up a wait comes here too, and leaves nothing.
        named_bar_sync(1, 2 * kXTile);
        if (!ok) break;
        const int r = w * kXTile + t;
        if (un.nt > 0) {
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(tO + c, o);
            tmem_wait_ld();
            reg_fence(o);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *L::join_o(smem, r, c / 4 + q) =
                  make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]), __uint_as_float(o[4 * q + 2]),
                              __uint_as_float(o[4 * q + 3]));
          }
        }
        *L::join_ml(smem, r) = make_float2(m_cur, l);
        break;
      }
      if (!ok) break;
      const float inv_l = l == 0.f ? 0.f : 1.f / l;  // 0: no key
      const int row = un.q0 + w * kXTile + t;
      uint4 *op = reinterpret_cast<uint4 *>(p.out + un.b * p.out_sb + un.h * p.out_sh + int64_t(row) * p.out_sn);
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t r[32] = {};
        if (un.nt > 0) {
          tmem_ld32(tO + c, r);
          tmem_wait_ld();
          reg_fence(r);
        }
        if (row < p.Nq) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t wv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              wv[e] = pack_bf16x2(__uint_as_float(r[8 * q + 2 * e]) * inv_l,
                                  __uint_as_float(r[8 * q + 2 * e + 1]) * inv_l);
            op[c / 8 + q] = make_uint4(wv[0], wv[1], wv[2], wv[3]);
          }
        }
      }
      if (un.nt > 0) {
        // O has been read: the next unit's first P V may overwrite it
        tc_fence_before_sync();
        mbar_arrive(&bars[L::kBarOFree + w]);
      }
      if (row < p.Nq && p.lse != nullptr)
        p.lse[un.b * p.lse_sb + un.h * p.lse_sh + int64_t(row) * p.lse_sn] =
            l == 0.f ? -INFINITY : fmaf(neg_m, -kXLn2, logf(l));
    }
  }

  if (kShared) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const CrossUnit un = cross_unit<kShared>(p, u_begin);
    const float c_s = p.tau * kXLog2e;
    const int rows = kXQTiles * kXTile / p.splits, row0 = int(cluster.block_rank()) * rows;
    for (int at = threadIdx.x; at < rows * (D / 4); at += kXThreads) {
      const int r = row0 + at / (D / 4), c = at % (D / 4), row = un.q0 + r;
      if (row >= p.Nq) continue;
      float2 ml[kXMaxSplits];
      float mm = -INFINITY, ll = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int s = 0; s < kXMaxSplits; ++s) {
        ml[s] = make_float2(-INFINITY, 0.f);
        if (s < p.splits) ml[s] = *L::join_ml(cluster.map_shared_rank(smem, s), r);
        mm = fmaxf(mm, ml[s].x);
      }
#pragma unroll
      for (int s = 0; s < kXMaxSplits; ++s) {
        if (ml[s].y != 0.f) {  // otherwise the part had no key, and left no O
          const float a = ex2_approx((ml[s].x - mm) * c_s);
          const float4 o = *L::join_o(cluster.map_shared_rank(smem, s), r, c);
          ll = fmaf(a, ml[s].y, ll);
          acc.x = fmaf(a, o.x, acc.x);
          acc.y = fmaf(a, o.y, acc.y);
          acc.z = fmaf(a, o.z, acc.z);
          acc.w = fmaf(a, o.w, acc.w);
        }
      }
      const float inv = ll == 0.f ? 0.f : 1.f / ll;
      *reinterpret_cast<uint2 *>(p.out + un.b * p.out_sb + un.h * p.out_sh + int64_t(row) * p.out_sn + 4 * c) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (c == 0 && p.lse != nullptr)
        p.lse[un.b * p.lse_sb + un.h * p.lse_sh + int64_t(row) * p.lse_sn] =
            ll == 0.f ? -INFINITY : fmaf(mm, p.tau, logf(ll));
    }
    cluster.sync();  // no CTA leaves while another reads its shared memory
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kXWarpMma) tmem_dealloc(tmem, 512);
}

}  // namespace pba
