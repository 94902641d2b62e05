// pba_cross_bwd_sm100.cuh -- gradients of cross attention on the sm_100a tensor
// cores.  With the forward's log-sum-exp and P_ij = exp(tau q_i.k_j - lse_i)
// over the keys that take part,
//     Delta_i = sum_d dO_id O_id                         (pba_cross_delta_kernel)
//     dS_ij   = P_ij (dO_i . v_j - Delta_i)
//     dq_i = tau sum_j dS_ij k_j                          (kernel A)
//     dk_j = tau sum dS_ij q_i,  dv_j = sum P_ij dO_i     (kernel B, over the
//                                 queries of every head that shares key head)
//
// Kernel A walks the key tiles of one 128-row query tile: S = Q K^T and dP =
// dO V^T into Tensor Memory, dS in registers and back to Tensor Memory as
// bf16, dQ += dS K.  Kernel B walks the query tiles, head by head of the group,
// of one 128-row key tile: S^T = K Q^T, dP^T = V dO^T, then dV += P^T dO and
// dK += dS^T Q.  No atomics and nothing of size Nq Nk in memory: each gradient
// is summed in one accumulator in one order.
//
// One CTA per unit, 384 threads: warps 0-7 two compute warpgroups (row =
// thread = Tensor Memory lane; warpgroup g takes columns 64g .. 64g+63 of
// every step), warp 8 the TMA producer, warp 9 Tensor Memory and the MMAs,
// warp 10 in kernel A takes out the keys that do not take part, as in the forward
// (their rows of K and V are zeros, their scores -inf).  For
// D <= 64 the next step's S and dP are issued as soon as this step's have been
// read; at D = 128 P and dS lie over S and dP, so they wait for the products
// that read them.
#pragma once

#include "pba_cross_sm100.cuh"

namespace pba {

struct CrossBwdParams {
  CUtensorMap tm_q, tm_k, tm_v, tm_do;  // (D, n, heads, B) bf16, box {min(D, 64), 128, 1, 1}
  int32_t B, H, Hkv, group, Nq, Nk;
  int32_t n_tiles;      // A: ceil(Nq / 128) per (b, h); B: ceil(Nk / 128) per (b, hkv)
  float tau;
  const int32_t *k_len;
  const uint8_t *mask;
  int64_t mask_sb;
  int32_t mask_vec4;
  const float *lse;     // [B][H][Nq] with strides
  int64_t lse_sb, lse_sh, lse_sn;
  const float *delta;   // [B][H][Nq] contiguous
  uint16_t *dq, *dk, *dv;  // bf16, contiguous [B][heads][n][D]
  int *err;
  uint64_t timeout_ns;
};

template <int D>
struct CrossBwdLayout {
  using T = XTileLayout<D>;
  static constexpr bool kAlias = D == 128;
  static constexpr int kStages = D == 128 ? 2 : 3;
  static constexpr int kOffFix0 = 0;
  static constexpr int kOffFix1 = kOffFix0 + T::kBytes;
  static constexpr int kOffStep0 = kOffFix1 + T::kBytes;             // [stage]
  static constexpr int kOffStep1 = kOffStep0 + kStages * T::kBytes;  // [stage]
  // B: per compute warp -lse log2(e) and -Delta of its 64 query columns,
  // double-buffered by step parity
  static constexpr int kRowvFloats = kXTile;
  static constexpr int kOffRowv = kOffStep1 + kStages * T::kBytes;
  static constexpr int kOffOnes = kOffRowv + 2 * 8 * kRowvFloats * 4;
  static constexpr int kOffMask = kOffOnes + XMaskTile::kBytes;              // [stage]
  static constexpr int kOffPartial = kOffMask + kStages * XMaskTile::kBytes;  // [stage]: the tile needs its column
  static constexpr int kOffBar = kOffPartial + 16;
  static constexpr int kBarFixFull = 0;
  static constexpr int kBarStepFull = 1;
  static constexpr int kBarStepEmpty = kBarStepFull + kStages;
  static constexpr int kBarStepReady = kBarStepEmpty + kStages;  // A: keys that do not take part are out
  static constexpr int kBarSFull = kBarStepReady + kStages;
  static constexpr int kBarSFree = kBarSFull + 1;
  static constexpr int kBarGFull = kBarSFree + 1;  // P / dS written to Tensor Memory
  static constexpr int kBarGDone = kBarGFull + 1;  // the accumulating MMAs of a step are done
  static constexpr int kBarDrain = kBarGDone + 1;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
  static constexpr int kOffAbort = kOffTmemSlot + 4;
  static constexpr int kBytes = kOffAbort + 4;
  static constexpr int kSmemAlloc = kBytes + 1024;
  static_assert(kSmemAlloc <= 232448, "shared memory budget");
  // Tensor Memory columns.  The 128 columns of P^T / dS as bf16 are two halves
  // of 32 words, one per warpgroup; over S and dP each half lies in the columns
  // that its own warpgroup has read.
  static constexpr uint32_t kColS = 0, kColDP = 128;
  static constexpr uint32_t kColAcc0 = kAlias ? 256 : 384, kColAcc1 = kColAcc0 + D;
  static_assert(kColAcc1 + D <= 512, "Tensor Memory budget");
  static constexpr __host__ __device__ uint32_t col_p(int half) { return kAlias ? kColS + half * 64 : 256u + half * 32; }
  static constexpr __host__ __device__ uint32_t col_ds(int half) { return kAlias ? kColDP + half * 64 : 320u + half * 32; }
};

// kB = false: kernel A (dq); kB = true: kernel B (dk, dv).
template <int D, bool kB>
__global__ void __launch_bounds__(kXThreads, 1) pba_cross_bwd_sm100_kernel(const __grid_constant__ CrossBwdParams p) {
  using L = CrossBwdLayout<D>;
  using T = typename L::T;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffTmemSlot);
  int *abort_flag = reinterpret_cast<int *>(smem + L::kOffAbort);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int tile = blockIdx.x % p.n_tiles;
  const int bh = blockIdx.x / p.n_tiles;
  const int heads = kB ? p.Hkv : p.H;
  const int h = bh % heads, b = bh / heads;  // A: query head; B: key head
  const int row0 = tile * kXTile;
  const int keys = cross_keys(p.k_len, b, p.Nk);
  const int q_tiles = (p.Nq + kXTile - 1) / kXTile;
  // B: a key tile with no key that counts has no steps (its gradients are 0)
  const int nsteps = kB ? (row0 < keys ? p.group * q_tiles : 0) : (keys + kXTile - 1) / kXTile;
  const bool fix = !kB && (p.mask != nullptr || p.k_len != nullptr || p.Nk % kXTile != 0);
  volatile int *partial = reinterpret_cast<volatile int *>(smem + L::kOffPartial);

  if (threadIdx.x == 0) {
    mbar_init(&bars[L::kBarFixFull], 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&bars[L::kBarStepFull + s], 1);
      mbar_init(&bars[L::kBarStepEmpty + s], 1);  // the commit after the step's last MMAs
      mbar_init(&bars[L::kBarStepReady + s], 32);
    }
    mbar_init(&bars[L::kBarSFull], 1);
    mbar_init(&bars[L::kBarSFree], 2 * kXTile);
    mbar_init(&bars[L::kBarGFull], 2 * kXTile);
    mbar_init(&bars[L::kBarGDone], 1);
    mbar_init(&bars[L::kBarDrain], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (!kB) {  // zeros but for the ones
    for (int i = threadIdx.x; i < (1 + L::kStages) * XMaskTile::kBytes / 16; i += kXThreads)
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
        T::load(smem + L::kOffFix0, kB ? &p.tm_k : &p.tm_q, &bars[L::kBarFixFull], row0, h, b, pol);
        T::load(smem + L::kOffFix1, kB ? &p.tm_v : &p.tm_do, &bars[L::kBarFixFull], row0, h, b, pol);
        bool ok = true;
        int it = 0;
        for (; it < nsteps && ok; ++it) {
          const int s = it % L::kStages;
          if (it >= L::kStages) ok = mbar_wait(&bars[L::kBarStepEmpty + s], ((it / L::kStages) - 1) & 1, wc);
          if (!ok) break;
          const int o0 = (kB ? it % q_tiles : it) * kXTile;
          const int oh = kB ? h * p.group + it / q_tiles : h / p.group;
          uint64_t *full = &bars[L::kBarStepFull + s];
          mbar_arrive_expect_tx(full, 2 * T::kBytes);
          T::load(smem + L::kOffStep0 + s * T::kBytes, kB ? &p.tm_q : &p.tm_k, full, o0, oh, b, pol);
          T::load(smem + L::kOffStep1 + s * T::kBytes, kB ? &p.tm_do : &p.tm_v, full, o0, oh, b, pol);
        }
        // every copy issued lands before the CTA exits
        mbar_wait(&bars[L::kBarFixFull], 0, wc_drain);
        if (!ok)
          for (int s = 0; s < L::kStages; ++s) {
            const int a = (it - s + L::kStages - 1) / L::kStages;
            if (a > 0) mbar_wait(&bars[L::kBarStepFull + s], (a - 1) & 1, wc_drain);
          }
      }
    } else if (warp == kXWarpMma) {
      // ================================================================ MMA issuer
      // The whole warp walks through the loop and one lane issues: the operand
      // descriptors then stay in uniform registers.
      if (nsteps > 0) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(kXTile, kXTile, false);  // both operands K-major
        constexpr uint32_t idesc_g = idesc_bf16_f32(kXTile, D, true);        // B MN-major
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t smem0 = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
        const uint32_t a0 = smem_desc_lo(smem0 + L::kOffFix0, 16), a1 = smem_desc_lo(smem0 + L::kOffFix1, 16);
        // a warp's waits end as one
        auto wait = [&](int bar, int parity) -> bool {
          return __all_sync(0xffffffffu, mbar_wait<false>(&bars[bar], parity & 1, wc));
        };
        // S, dP of step `it` (A: Q K^T, dO V^T; B: K Q^T, V dO^T) once its
        // tiles have landed and the previous step's S and dP have been read
        // (at D = 128: and the products over them are done)
        auto issue_s = [&](int it) -> bool {
          const int s = it % L::kStages;
          if (!wait(fix ? L::kBarStepReady + s : L::kBarStepFull + s, it / L::kStages)) return false;
          if (it > 0 && !wait(L::kAlias ? L::kBarGDone : L::kBarSFree, it - 1)) return false;
          tc_fence_after_sync();
          const uint32_t b0 = smem_desc_lo(smem0 + L::kOffStep0 + s * T::kBytes, 16);
          const uint32_t b1 = smem_desc_lo(smem0 + L::kOffStep1 + s * T::kBytes, 16);
          const uint32_t ones_lo = smem_desc_lo(smem0 + L::kOffOnes, 16);
          const uint32_t mask_lo = smem_desc_lo(smem0 + L::kOffMask + s * XMaskTile::kBytes, 16);
          const bool masked = fix && partial[s] != 0;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_ss(tm + L::kColS, desc_join(a0 + T::k_step(kk), T::kDescHi),
                          desc_join(b0 + T::k_step(kk), T::kDescHi), idesc_s, kk > 0);
            if (masked)
              mma_bf16_ss(tm + L::kColS, desc_join(ones_lo, XMaskTile::kDescHi),
                          desc_join(mask_lo, XMaskTile::kDescHi), idesc_s, 1u);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_ss(tm + L::kColDP, desc_join(a1 + T::k_step(kk), T::kDescHi),
                          desc_join(b1 + T::k_step(kk), T::kDescHi), idesc_s, kk > 0);
            tc_commit(&bars[L::kBarSFull]);
          }
          __syncwarp();
          return true;
        };
        // acc += G X with G (bf16, in Tensor Memory) and X an MN-major tile; by one lane
        auto issue_g = [&](uint32_t acc, bool ds, uint32_t x_lo, bool more) {
#pragma unroll
          for (int kk = 0; kk < kXTile / 16; ++kk)
            mma_bf16_ts(tm + acc, tm + (ds ? L::col_ds(kk >> 2) : L::col_p(kk >> 2)) + (kk & 3) * 8,
                        desc_join(x_lo + T::mn_step(kk), T::kDescHi), idesc_g, (more || kk > 0) ? 1u : 0u);
        };
        bool ok = wait(L::kBarFixFull, 0) && issue_s(0);
        for (int it = 0; it < nsteps && ok; ++it) {
          const int s = it % L::kStages;
          if (!L::kAlias && it + 1 < nsteps && !(ok = issue_s(it + 1))) break;
          ok = wait(L::kBarGFull, it);
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t x0 = smem_desc_lo(smem0 + L::kOffStep0 + s * T::kBytes, T::kSlabBytes);
          const uint32_t x1 = smem_desc_lo(smem0 + L::kOffStep1 + s * T::kBytes, T::kSlabBytes);
          if (elect_one()) {
            if (kB) issue_g(L::kColAcc1, false, x1, it > 0);  // dV += P^T dO
            issue_g(L::kColAcc0, true, x0, it > 0);           // A: dQ += dS K; B: dK += dS^T Q
            tc_commit(&bars[L::kBarGDone]);
            tc_commit(&bars[L::kBarStepEmpty + s]);
          }
          __syncwarp();
          if (L::kAlias && it + 1 < nsteps && !(ok = issue_s(it + 1))) break;
        }
        if (elect_one()) tc_commit(&bars[L::kBarDrain]);
        __syncwarp();
        mbar_wait<false>(&bars[L::kBarDrain], 0, wc_drain);
      }
    } else if (warp == kXWarpFix && fix) {
      // ================================================================ A: keys that do not take part
      const uint8_t *mrow = p.mask != nullptr ? p.mask + int64_t(b) * p.mask_sb : nullptr;
      bool ok = true;
      uint32_t next = nsteps > 0 ? cross_mask_bytes(mrow, p.mask_vec4, 0, keys, lane) : 0u;
      for (int it = 0; it < nsteps && ok; ++it) {
        const int s = it % L::kStages;
        const KeepWords keep = cross_keep(next);
        if (it + 1 < nsteps) next = cross_mask_bytes(mrow, p.mask_vec4, (it + 1) * kXTile, keys, lane);
        ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars[L::kBarStepFull + s], (it / L::kStages) & 1, wc));
        if (!ok) break;
        const bool any = !keep.all();
        if (any) {
          cross_zero_rows<D>(smem + L::kOffStep0 + s * T::kBytes, keep, lane);
          cross_zero_rows<D>(smem + L::kOffStep1 + s * T::kBytes, keep, lane);
          cross_mask_column(smem + L::kOffMask + s * XMaskTile::kBytes, keep, lane);
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
    const int g = warp >> 2;           // column half of each step
    const int t = threadIdx.x & 127;   // row of the unit's tile = Tensor Memory lane
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const int r = row0 + t;            // A: query row; B: key row
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
          const int qi = (step % q_tiles) * kXTile + g * 64 + lane + 32 * e;
          if (qi < p.Nq) {
            nlse[e] = p.lse[b * p.lse_sb + qh * p.lse_sh + int64_t(qi) * p.lse_sn];
            ndelta[e] = p.delta[(int64_t(b) * p.H + qh) * p.Nq + qi];
          }
        }
      }
    };
    if (nsteps > 0) load_cols(0);
    bool ok = true;
    for (int it = 0; it < nsteps && ok; ++it) {
      const float clse[2] = {nlse[0], nlse[1]}, cdelta[2] = {ndelta[0], ndelta[1]};
      if (it + 1 < nsteps) load_cols(it + 1);
      float *rv = reinterpret_cast<float *>(smem + L::kOffRowv) + ((it & 1) * 8 + warp) * L::kRowvFloats;
      if (kB) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = lane + 32 * e;
          const int qi = (it % q_tiles) * kXTile + g * 64 + col;
          rv[col] = qi >= p.Nq ? -INFINITY : (clse[e] == -INFINITY ? 0.f : -clse[e] * kXLog2e);
          rv[64 + col] = qi < p.Nq ? -cdelta[e] : 0.f;
        }
        __syncwarp();
      }
      ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars[L::kBarSFull], it & 1, wc));
      if (!ok) break;
      tc_fence_after_sync();
      const float2 cs2 = make_float2(c_s, c_s);
      const float2 rowl2 = make_float2(-lse2, -lse2), rowd2 = make_float2(-delta, -delta);
      uint32_t sv[64], dpv[64];
      tmem_ld32(tmem + lane_base + L::kColS + g * 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
      tmem_ld32(tmem + lane_base + L::kColS + g * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
      tmem_ld32(tmem + lane_base + L::kColDP + g * 64, *reinterpret_cast<uint32_t(*)[32]>(&dpv[0]));
      tmem_ld32(tmem + lane_base + L::kColDP + g * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&dpv[32]));
      tmem_wait_ld();
      reg_fence(sv);
      reg_fence(dpv);
      // the next step's S and dP may overwrite these columns
      tc_fence_before_sync();
      if (!L::kAlias) mbar_arrive(&bars[L::kBarSFree]);
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
            const float2 ds = fmul2(pe, fadd2(make_float2(__uint_as_float(dpv[i]), __uint_as_float(dpv[i + 1])), nd[e]));
            if (kB) pk[j4 * 2 + e] = pack_bf16x2(pe.x, pe.y);
            dk[j4 * 2 + e] = pack_bf16x2(ds.x, ds.y);
          }
        }
        if (!L::kAlias && qt == 0 && it > 0) {
          // the previous step's accumulating MMAs read what the stores below overwrite
          ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars[L::kBarGDone], (it - 1) & 1, wc));
          if (!ok) break;
          tc_fence_after_sync();
        }
        if (kB) tmem_st16(tmem + lane_base + L::col_p(g) + qt * 16, pk);
        tmem_st16(tmem + lane_base + L::col_ds(g) + qt * 16, dk);
      }
      if (!ok) break;
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(&bars[L::kBarGFull]);
    }
    // -------------------------------------------------------------- epilogue
    if (ok && nsteps > 0) ok = __all_sync(0xffffffffu, mbar_wait<false>(&bars[L::kBarGDone], (nsteps - 1) & 1, wc));
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
