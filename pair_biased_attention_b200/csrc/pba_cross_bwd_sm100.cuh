// pba_cross_bwd_sm100.cuh -- gradients of cross attention on the sm_100a tensor
// cores.  With the forward's log-sum-exp and P_ij = exp(tau q_i.k_j - lse_i)
// over the keys that take part,
//     Delta_i = sum_d dO_id O_id                         (pba_cross_delta_kernel)
//     dS_ij   = P_ij (dO_i . v_j - Delta_i)
//     dq_i = tau sum_j dS_ij k_j                          (kind A)
//     dk_j = tau sum dS_ij q_i,  dv_j = sum P_ij dO_i     (kind B, over the
//                                 queries of every head that shares key head)
//
// A unit of kind A walks the keys of one 128-row query tile: S = Q K^T and dP = dO V^T
// into Tensor Memory, dS in registers and back to Tensor Memory as bf16,
// dQ += dS K.  One of kind B walks the queries, head by head of the group, of one
// 128-row key tile: S^T = K Q^T, dP^T = V dO^T, then dV += P^T dO and
// dK += dS^T Q.  No atomics and nothing of size Nq Nk in memory: each gradient
// is summed in one accumulator in one order.
//
// One CTA per unit, 384 threads: warps 0-7 two compute warpgroups (row =
// thread = Tensor Memory lane), warp 8 the TMA producer, warps 9 and 11 the
// MMAs, warp 10 in kind A takes out the keys that do not take part, as in the
// forward (their rows of K and V are zeros, their scores -inf).
//   D <= 64: a step is 128 columns, 64 for each warpgroup; its successor's S
//     and dP are issued as soon as both have read theirs.
//   D = 128: Tensor Memory holds no second copy of P and dS, so they lie over S
//     and dP and the next ones wait for the products that read them.  A step is
//     64 columns there, with S and dP of its own for each warpgroup, which take
//     the steps in turn: one computes while the other's products run.
// Both kinds are one launch, so that their last waves overlap.  Measured at
// 2 x 16 heads x 2048 x 2048 with Delta, a key mask / none: D = 64 166 / 162 us
// (in two launches 189 / 184; 64-wide steps in turn instead of shared ones 8 us
// more with the mask), D = 32 157 / 154, D = 128 238 / 235 (275 / 270).  At
// D = 64 that is 0.53 PFLOP/s counting each product of the formulas once, 0.74
// with the scores and dP that B computes again; what is left is the
// exponentials' and the conversions' instructions between the products.  Delta
// summed by kind A's threads for their rows, without its launch of 7 us, was
// slower (D = 128 by 13 us): their rows are read in 16-byte pieces.
#pragma once

#include "pba_cross_sm100.cuh"

namespace pba {

constexpr int kXBox = 64;  // rows of a tile load

struct CrossBwdParams {
  CUtensorMap tm_q, tm_k, tm_v, tm_do;  // (D, n, heads, B) bf16, box {min(D, 64), kXBox, 1, 1}
  int32_t B, H, Hkv, group, Nq, Nk;
  int32_t q_tiles;      // A: units per (b, h), ceil(Nq / 128)
  int32_t k_tiles;      // B: units per (b, hkv), ceil(Nk / 128)
  int32_t units_a, units_b, b_first;
  float tau;
  const int32_t *k_len;
  const uint8_t *mask;
  int64_t mask_sb;
  const float *lse;     // [B][H][Nq] with strides
  int64_t lse_sb, lse_sh, lse_sn;
  const float *delta;   // [B][H][Nq] contiguous
  uint16_t *dq, *dk, *dv;  // bf16, contiguous [B][heads][n][D]
  int *err;
  uint64_t timeout_ns;
};

template <int D>
struct CrossBwdLayout {
  static constexpr bool kAlias = D == 128;
  static constexpr int kTurns = kAlias ? 2 : 1;   // warpgroups that take steps in turn (1: they share each)
  static constexpr int kStep = kAlias ? 64 : 128;  // keys (A) or queries (B) of a step
  static constexpr int kPer = kStep / 32;
  using T = XTileLayout<D>;         // the unit's rows
  using S = XTileLayout<D, kStep>;  // a step's
  static constexpr int kStages = 4;
  static constexpr int kOffFix0 = 0;
  static constexpr int kOffFix1 = kOffFix0 + T::kBytes;
  static constexpr int kOffStep0 = kOffFix1 + T::kBytes;             // [stage]
  static constexpr int kOffStep1 = kOffStep0 + kStages * S::kBytes;  // [stage]
  // B: per compute warp -lse log2(e) and -Delta of its 64 query columns of a
  // step, double-buffered by the parity of the warpgroup's steps
  static constexpr int kRowvFloats = 2 * 64;
  static constexpr int kOffRowv = kOffStep1 + kStages * S::kBytes;
  static constexpr int kMaskBytes = kStep * XMaskTile::kRowBytes;
  static constexpr int kOffOnes = kOffRowv + 2 * 8 * kRowvFloats * 4;
  static constexpr int kOffMask = kOffOnes + kXTile * XMaskTile::kRowBytes;  // [stage]
  static constexpr int kOffPartial = kOffMask + kStages * kMaskBytes;        // [stage]: the tile needs its column
  static constexpr int kOffBar = kOffPartial + 32;
  static_assert(kStages * 4 <= 32, "flags");
  static constexpr int kBarFixFull = 0;
  static constexpr int kBarStepFull = 1;
  static constexpr int kBarStepEmpty = kBarStepFull + kStages;
  static constexpr int kBarStepReady = kBarStepEmpty + kStages;  // A: keys that do not take part are out
  static constexpr int kBarSFull = kBarStepReady + kStages;  // [turn], and so on
  static constexpr int kBarSFree = kBarSFull + kTurns;
  static constexpr int kBarGFull = kBarSFree + kTurns;  // P / dS written to Tensor Memory
  static constexpr int kBarGDone = kBarGFull + kTurns;  // the accumulating MMAs of a step are done
  static constexpr int kBarDrain = kBarGDone + kTurns;
  static constexpr int kNumBars = kBarDrain + 2;
  static constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
  static constexpr int kOffAbort = kOffTmemSlot + 4;
  static constexpr int kBytes = kOffAbort + 4;
  static constexpr int kSmemAlloc = kBytes + 1024;
  static_assert(kSmemAlloc <= 232448, "shared memory budget");
  // Tensor Memory columns of warpgroup g: 64 each of S and dP, 32 each of P and
  // dS as bf16; then the accumulators.  Shared steps have S, dP, P and dS of
  // both warpgroups next to each other.
  static constexpr __host__ __device__ uint32_t col_s(int g) { return (kAlias ? 128u : 64u) * g; }
  static constexpr __host__ __device__ uint32_t col_dp(int g) { return kAlias ? 128u * g + 64 : 128u + 64 * g; }
  static constexpr __host__ __device__ uint32_t col_p(int g) { return kAlias ? col_s(g) : 256u + 32 * g; }
  static constexpr __host__ __device__ uint32_t col_ds(int g) { return kAlias ? col_dp(g) : 320u + 32 * g; }
  static constexpr uint32_t kColAcc0 = kAlias ? 256 : 384, kColAcc1 = kColAcc0 + D;
  static_assert(kColAcc1 + D <= 512, "Tensor Memory budget");
};

// kB = false: a unit of kind A (dq); kB = true: of kind B (dk, dv).
template <int D, bool kB>
__device__ __forceinline__ void cross_bwd_unit(const CrossBwdParams &p, int unit) {
  using L = CrossBwdLayout<D>;
  using T = typename L::T;
  using S = typename L::S;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffTmemSlot);
  int *abort_flag = reinterpret_cast<int *>(smem + L::kOffAbort);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int n_tiles = kB ? p.k_tiles : p.q_tiles;
  const int tile = unit % n_tiles;
  const int bh = unit / n_tiles;
  const int heads = kB ? p.Hkv : p.H;
  const int h = bh % heads, b = bh / heads;  // A: query head; B: key head
  const int row0 = tile * kXTile;
  const int keys = cross_keys(p.k_len, b, p.Nk);
  const int q_tiles = (p.Nq + L::kStep - 1) / L::kStep;
  // B: a key tile with no key that counts has no steps (its gradients are 0)
  const int nsteps = kB ? (row0 < keys ? p.group * q_tiles : 0) : (keys + L::kStep - 1) / L::kStep;
  const bool fix = !kB && (p.mask != nullptr || p.k_len != nullptr || p.Nk % L::kStep != 0);
  volatile int *partial = reinterpret_cast<volatile int *>(smem + L::kOffPartial);

  if (threadIdx.x == 0) {
    mbar_init(&bars[L::kBarFixFull], 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&bars[L::kBarStepFull + s], 1);
      mbar_init(&bars[L::kBarStepEmpty + s], 1);  // the commit after the step's last MMAs
      mbar_init(&bars[L::kBarStepReady + s], 32);
    }
    for (int g = 0; g < L::kTurns; ++g) {
      mbar_init(&bars[L::kBarSFull + g], 1);
      mbar_init(&bars[L::kBarSFree + g], 2 * kXTile / L::kTurns);
      mbar_init(&bars[L::kBarGFull + g], 2 * kXTile / L::kTurns);
      mbar_init(&bars[L::kBarGDone + g], 1);
    }
    mbar_init(&bars[L::kBarDrain], 1);
    mbar_init(&bars[L::kBarDrain + 1], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (!kB) {  // zeros but for the ones
    for (int i = threadIdx.x; i < (L::kOffPartial - L::kOffOnes) / 16; i += kXThreads)
      reinterpret_cast<uint4 *>(smem + L::kOffOnes)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (threadIdx.x < kXTile) *XMaskTile::at(smem + L::kOffOnes, threadIdx.x) = 0x3F80u;
    fence_proxy_async_smem();
  }
  if (warp == kXWarpMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl wc{abort_flag, p.err, p.timeout_ns};
  WaitCtl wc_drain = wc;
  int drain_abort = 0;
  wc_drain.abort_flag = &drain_abort;

  if (warp >= 8) {
    setmaxnreg_dec<kXRegsOther>();
    if (warp == kXWarpProducer) {
      // ================================================================ TMA producer
      if (lane == 0 && nsteps > 0) {
        const uint64_t pol = l2_policy_evict_last();
        // fixed tiles of the unit: A: Q, dO rows; B: K, V rows
        mbar_arrive_expect_tx(&bars[L::kBarFixFull], 2 * T::kBytes);
        const CUtensorMap *fix0 = kB ? &p.tm_k : &p.tm_q, *fix1 = kB ? &p.tm_v : &p.tm_do;
        const CUtensorMap *step0 = kB ? &p.tm_q : &p.tm_k, *step1 = kB ? &p.tm_do : &p.tm_v;
        for (int half = 0; half < 2; ++half) {
          T::template load<kXBox>(smem + L::kOffFix0, half, fix0, &bars[L::kBarFixFull], row0, h, b, pol);
          T::template load<kXBox>(smem + L::kOffFix1, half, fix1, &bars[L::kBarFixFull], row0, h, b, pol);
        }
        bool ok = true;
        int it = 0;
        for (; it < nsteps && ok; ++it) {
          const int s = it % L::kStages;
          if (it >= L::kStages) ok = mbar_wait(&bars[L::kBarStepEmpty + s], ((it / L::kStages) - 1) & 1, wc);
          if (!ok) break;
          const int o0 = (kB ? it % q_tiles : it) * L::kStep;
          const int oh = kB ? h * p.group + it / q_tiles : h / p.group;
          uint64_t *full = &bars[L::kBarStepFull + s];
          mbar_arrive_expect_tx(full, 2 * S::kBytes);
          for (int part = 0; part < L::kStep / kXBox; ++part) {
            S::template load<kXBox>(smem + L::kOffStep0 + s * S::kBytes, part, step0, full, o0, oh, b, pol);
            S::template load<kXBox>(smem + L::kOffStep1 + s * S::kBytes, part, step1, full, o0, oh, b, pol);
          }
        }
        // every copy issued lands before the CTA exits
        mbar_wait(&bars[L::kBarFixFull], 0, wc_drain);
        if (!ok)
          for (int s = 0; s < L::kStages; ++s) {
            const int a = (it - s + L::kStages - 1) / L::kStages;
            if (a > 0) mbar_wait(&bars[L::kBarStepFull + s], (a - 1) & 1, wc_drain);
          }
      }
    } else if (warp == kXWarpMma || warp == kXWarpMma1) {
      // ================================================================ MMA issuers
      // One warp for the scores, one for the products over them: neither's
      // waits hold up the other, and the accumulators see one order.  The whole
      // warp walks through the loop and one lane issues: the operand
      // descriptors then stay in uniform registers.
      constexpr uint32_t idesc_s = idesc_bf16_f32(kXTile, L::kStep, false);  // both operands K-major
      constexpr uint32_t idesc_g = idesc_bf16_f32(kXTile, D, true);        // B MN-major
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t smem0 = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
      auto wait = [&](int bar, int parity) -> bool { return warp_wait(&bars[bar], parity, wc); };
      bool ok = nsteps > 0;
      if (warp == kXWarpMma) {
        // S, dP (A: Q K^T, dO V^T; B: K Q^T, V dO^T) once the tiles have landed
        // and the warpgroup has read those of its last step (at D = 128: and
        // the products over them are done)
        const uint32_t a0 = smem_desc_lo(smem0 + L::kOffFix0, 16), a1 = smem_desc_lo(smem0 + L::kOffFix1, 16);
        const uint32_t ones_lo = smem_desc_lo(smem0 + L::kOffOnes, 16);
        if (ok) ok = wait(L::kBarFixFull, 0);
        for (int it = 0; it < nsteps && ok; ++it) {
          const int s = it % L::kStages, g = it % L::kTurns, n = it / L::kTurns;
          const int full = (fix ? L::kBarStepReady : L::kBarStepFull) + s;
          const int read = (L::kAlias ? L::kBarGDone : L::kBarSFree) + g;
          ok = n > 0 ? warp_wait2(&bars[full], it / L::kStages, &bars[read], n - 1, wc) : wait(full, it / L::kStages);
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t b0 = smem_desc_lo(smem0 + L::kOffStep0 + s * S::kBytes, 16);
          const uint32_t b1 = smem_desc_lo(smem0 + L::kOffStep1 + s * S::kBytes, 16);
          const uint32_t mask_lo = smem_desc_lo(smem0 + L::kOffMask + s * L::kMaskBytes, 16);
          const uint32_t ts = tm + L::col_s(g), tdp = tm + L::col_dp(g);
          const bool masked = fix && partial[s] != 0;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_ss(ts, desc_join(a0 + T::k_step(kk), T::kDescHi), desc_join(b0 + S::k_step(kk), S::kDescHi),
                          idesc_s, kk > 0);
            if (masked)
              mma_bf16_ss(ts, desc_join(ones_lo, XMaskTile::kDescHi), desc_join(mask_lo, XMaskTile::kDescHi), idesc_s,
                          1u);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_ss(tdp, desc_join(a1 + T::k_step(kk), T::kDescHi), desc_join(b1 + S::k_step(kk), S::kDescHi),
                          idesc_s, kk > 0);
            tc_commit(&bars[L::kBarSFull + g]);
          }
          __syncwarp();
        }
      } else {
        // acc += G X with G (bf16, in Tensor Memory) and X an MN-major tile
        auto issue_g = [&](uint32_t acc, uint32_t gcol, uint32_t x_lo, bool more) {
#pragma unroll
          for (int kk = 0; kk < L::kStep / 16; ++kk)
            mma_bf16_ts(acc, gcol + kk * 8, desc_join(x_lo + S::mn_step(kk), S::kDescHi), idesc_g,
                        (more || kk > 0) ? 1u : 0u);
        };
        for (int it = 0; it < nsteps && ok; ++it) {
          const int s = it % L::kStages, g = it % L::kTurns, n = it / L::kTurns;
          // the step's tiles are there: its scores came from them
          if (!(ok = wait(L::kBarGFull + g, n))) break;
          tc_fence_after_sync();
          const uint32_t x0 = smem_desc_lo(smem0 + L::kOffStep0 + s * S::kBytes, S::kSlabBytes);
          const uint32_t x1 = smem_desc_lo(smem0 + L::kOffStep1 + s * S::kBytes, S::kSlabBytes);
          const uint32_t tp = tm + L::col_p(g), tds = tm + L::col_ds(g);
          if (elect_one()) {
            if (kB) issue_g(tm + L::kColAcc1, tp, x1, it > 0);  // dV += P^T dO
            issue_g(tm + L::kColAcc0, tds, x0, it > 0);         // A: dQ += dS K; B: dK += dS^T Q
            tc_commit(&bars[L::kBarGDone + g]);
            tc_commit(&bars[L::kBarStepEmpty + s]);
          }
          __syncwarp();
        }
      }
      // every MMA issued above completes before Tensor Memory is released; the
      // second issuer's end is also the sums'
      const int drain = L::kBarDrain + (warp == kXWarpMma1);
      if (elect_one()) tc_commit(&bars[drain]);
      __syncwarp();
      mbar_wait<false>(&bars[drain], 0, wc_drain);
    } else if (warp == kXWarpFix && fix) {
      // ================================================================ A: keys that do not take part
      const uint8_t *mrow = p.mask != nullptr ? p.mask + int64_t(b) * p.mask_sb : nullptr;
      bool ok = true;
      uint32_t next = nsteps > 0 ? cross_mask_bytes<L::kPer>(mrow, false, 0, keys, lane) : 0u;
      for (int it = 0; it < nsteps && ok; ++it) {
        const int s = it % L::kStages;
        const KeepWords<L::kPer> keep = cross_keep<L::kPer>(next);
        if (it + 1 < nsteps) next = cross_mask_bytes<L::kPer>(mrow, false, (it + 1) * L::kStep, keys, lane);
        ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars[L::kBarStepFull + s], (it / L::kStages) & 1, wc));
        if (!ok) break;
        const bool any = !keep.all();
        if (any) {
          cross_zero_rows<D>(smem + L::kOffStep0 + s * S::kBytes, keep, lane);
          cross_zero_rows<D>(smem + L::kOffStep1 + s * S::kBytes, keep, lane);
          cross_mask_column(smem + L::kOffMask + s * L::kMaskBytes, keep, lane);
          fence_proxy_async_smem();
        }
        if (lane == 0) partial[s] = any;
        __syncwarp();
        mbar_arrive(&bars[L::kBarStepReady + s]);
      }
    }
  } else {
    // ================================================================ compute warpgroups
    setmaxnreg_inc<kXRegsSoftmax>();
    const int g = warp >> 2;           // shared steps: takes 64 columns; in turn: the steps g, g + 2, ...
    constexpr bool kShare = L::kTurns == 1;
    const int turn = kShare ? 0 : g, col0 = kShare ? 64 * g : 0;
    const int t = threadIdx.x & 127;   // row of the unit's tile = Tensor Memory lane
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const int r = row0 + t;            // A: query row; B: key row
    const uint32_t tS = tmem + lane_base + L::col_s(g), tDP = tmem + lane_base + L::col_dp(g);
    const float c_s = p.tau * kXLog2e;
    float lse2 = 0.f, delta = 0.f;     // A: this row's
    bool key_ok = true;                // B: this row's key takes part
    if (!kB) {
      if (r < p.Nq) {
        // a row without a key (lse = -inf) gets a finite stand-in: its scores
        // are all -inf already
        const float lse = p.lse[b * p.lse_sb + h * p.lse_sh + int64_t(r) * p.lse_sn];
        lse2 = (lse == -INFINITY) ? 0.f : lse * kXLog2e;
        delta = p.delta[(int64_t(b) * p.H + h) * p.Nq + r];
      }
    } else {
      // a key that does not take part keeps its row to itself: what the row
      // sums up to, NaN included, is dropped at the end
      key_ok = r < keys && (p.mask == nullptr || p.mask[int64_t(b) * p.mask_sb + r] != 0);
    }
    // B: lse and Delta of a step's query columns `lane` and `lane + 32`, loaded
    // a step ahead
    float nlse[2] = {0.f, 0.f}, ndelta[2] = {0.f, 0.f};
    auto load_cols = [&](int step) {
      if (kB) {
        const int qh = h * p.group + step / q_tiles;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int qi = (step % q_tiles) * L::kStep + col0 + lane + 32 * e;
          if (qi < p.Nq) {
            nlse[e] = p.lse[b * p.lse_sb + qh * p.lse_sh + int64_t(qi) * p.lse_sn];
            ndelta[e] = p.delta[(int64_t(b) * p.H + qh) * p.Nq + qi];
          }
        }
      }
    };
    if (turn < nsteps) load_cols(turn);
    bool ok = true;
    int n = 0;  // steps of this warpgroup so far
    for (int it = turn; it < nsteps && ok; it += L::kTurns, ++n) {
      const float clse[2] = {nlse[0], nlse[1]}, cdelta[2] = {ndelta[0], ndelta[1]};
      if (it + L::kTurns < nsteps) load_cols(it + L::kTurns);
      float *rv = reinterpret_cast<float *>(smem + L::kOffRowv) + ((n & 1) * 8 + warp) * L::kRowvFloats;
      if (kB) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = lane + 32 * e;
          const int qi = (it % q_tiles) * L::kStep + col0 + col;
          rv[col] = qi >= p.Nq ? -INFINITY : (clse[e] == -INFINITY ? 0.f : -clse[e] * kXLog2e);
          rv[64 + col] = qi < p.Nq ? -cdelta[e] : 0.f;
        }
        __syncwarp();
      }
      ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars[L::kBarSFull + turn], n & 1, wc));
      if (!ok) break;
      tc_fence_after_sync();
      const float2 cs2 = make_float2(c_s, c_s);
      const float2 rowl2 = make_float2(-lse2, -lse2), rowd2 = make_float2(-delta, -delta);
      uint32_t sv[64], dpv[64];
      tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
      tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
      tmem_ld32(tDP, *reinterpret_cast<uint32_t(*)[32]>(&dpv[0]));
      tmem_ld32(tDP + 32, *reinterpret_cast<uint32_t(*)[32]>(&dpv[32]));
      tmem_wait_ld();
      reg_fence(sv);
      reg_fence(dpv);
      // the warpgroup's next S and dP may overwrite these columns
      tc_fence_before_sync();
      if (!L::kAlias) mbar_arrive(&bars[L::kBarSFree + turn]);
      // two quarters of 32 columns, each stored to Tensor Memory before the next is formed
#pragma unroll
      for (int qt = 0; qt < 2; ++qt) {
        uint32_t pk[16], dk[16];
#pragma unroll
        for (int j4 = 0; j4 < 8; ++j4) {  // four columns at a time
          const int c = qt * 32 + j4 * 4;
          float2 nl[2] = {rowl2, rowl2}, nd[2] = {rowd2, rowd2};
          if (kB) {
            const float4 la = *reinterpret_cast<const float4 *>(rv + c);
            const float4 da = *reinterpret_cast<const float4 *>(rv + 64 + c);
            nl[0] = make_float2(la.x, la.y), nl[1] = make_float2(la.z, la.w);
            nd[0] = make_float2(da.x, da.y), nd[1] = make_float2(da.z, da.w);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = c + 2 * e;
            const float2 a = ffma2(make_float2(__uint_as_float(sv[i]), __uint_as_float(sv[i + 1])), cs2, nl[e]);
            const float2 pe = make_float2(ex2_approx(a.x), ex2_approx(a.y));
            const float2 dp = make_float2(__uint_as_float(dpv[i]), __uint_as_float(dpv[i + 1]));
            const float2 ds = fmul2(pe, fadd2(dp, nd[e]));
            if (kB) pk[j4 * 2 + e] = pack_bf16x2(pe.x, pe.y);
            dk[j4 * 2 + e] = pack_bf16x2(ds.x, ds.y);
          }
        }
        if (!L::kAlias && qt == 0 && n > 0) {
          // the accumulating MMAs of its last step read what the stores below overwrite
          ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars[L::kBarGDone + turn], (n - 1) & 1, wc));
          if (!ok) break;
          tc_fence_after_sync();
        }
        if (kB) tmem_st16(tmem + lane_base + L::col_p(g) + qt * 16, pk);
        tmem_st16(tmem + lane_base + L::col_ds(g) + qt * 16, dk);
      }
      if (!ok) break;
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(&bars[L::kBarGFull + turn]);
    }
    // -------------------------------------------------------------- epilogue
    // all steps, the other warpgroup's too, are in the accumulators
    if (ok && nsteps > 0) ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars[L::kBarDrain + 1], 0, wc));
    if (ok) {
      tc_fence_after_sync();
      const int nrows = kB ? p.Nk : p.Nq;
      // A: dQ (acc0), the warpgroups take 32 columns in turn.  B: warpgroup 0
      // dK (acc0), warpgroup 1 dV (acc1), all D columns.
      const bool second = kB && g == 1;
      const uint32_t col = second ? L::kColAcc1 : L::kColAcc0;
      const float scale = second ? 1.f : p.tau;
      uint16_t *dst = !kB ? p.dq : (second ? p.dv : p.dk);
      const int c_begin = kB ? 0 : 32 * g, c_step = kB ? 32 : 64;
#pragma unroll 1
      for (int c = c_begin; c < D; c += c_step) {
        uint32_t v[32] = {};
        if (nsteps > 0) {
          tmem_ld32(tmem + lane_base + col + c, v);
          tmem_wait_ld();
          reg_fence(v);
        }
        if (r < nrows) {
          uint4 *o = reinterpret_cast<uint4 *>(dst + ((int64_t(b) * heads + h) * nrows + r) * D + c);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = key_ok ? pack_bf16x2(__uint_as_float(v[8 * q + 2 * e]) * scale,
                                          __uint_as_float(v[8 * q + 2 * e + 1]) * scale)
                            : 0u;
            o[q] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kXWarpMma) tmem_dealloc(tmem, 512);
}

// One launch for both kinds: neither reads what the other writes, and their last
// waves fill up with each other's units.  The kind with the longer units goes
// first.
template <int D>
__global__ void __launch_bounds__(kXThreads, 1) pba_cross_bwd_sm100_kernel(const __grid_constant__ CrossBwdParams p) {
  const int at = blockIdx.x, first = p.b_first ? p.units_b : p.units_a;
  const int unit = at < first ? at : at - first;
  if ((at < first) == (p.b_first != 0))
    cross_bwd_unit<D, true>(p, unit);
  else
    cross_bwd_unit<D, false>(p, unit);
}

struct CrossDeltaParams {
  const uint16_t *dout, *out;
  int64_t do_sb, do_sh, do_sn, o_sb, o_sh, o_sn;
  float *delta;
  int64_t rows;
  int32_t H, Nq;
};

// Delta_i = sum_d dO_id O_id, fp32: D / 8 lanes per row, one 16-byte load of
// each tensor per lane, the lanes of a row joined by shuffles.
template <int D>
__global__ void pba_cross_delta_kernel(const __grid_constant__ CrossDeltaParams p) {
  constexpr int kLanes = D / 8;
  const int64_t at = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t row = at / kLanes;
  const int c = int(at % kLanes) * 8;
  float acc = 0.f;
  if (row < p.rows) {
    const int64_t bh = row / p.Nq, i = row - bh * p.Nq;
    const int64_t b = bh / p.H, h = bh - b * p.H;
    const uint4 x = *reinterpret_cast<const uint4 *>(p.dout + b * p.do_sb + h * p.do_sh + i * p.do_sn + c);
    const uint4 y = *reinterpret_cast<const uint4 *>(p.out + b * p.o_sb + h * p.o_sh + i * p.o_sn + c);
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc = fmaf(bf16lo_to_f32(xw[e]), bf16lo_to_f32(yw[e]), acc);
      acc = fmaf(bf16hi_to_f32(xw[e]), bf16hi_to_f32(yw[e]), acc);
    }
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (row < p.rows && c == 0) p.delta[row] = acc;
}

}  // namespace pba
