// pba_cross_split.cuh -- cross attention for few query rows (a decoder's new
// tokens): the same sums as pba_cross_sm100.cuh, arranged for reading the keys
// and values once at full bandwidth.
//
// The query rows of the heads that share a key head (H / Hkv x Nq of them) are
// one matrix; a block takes 16 of its rows and a share of the keys, and each
// warp works on keys of its own, 32 at a time.  16 rows are one warp-level
// matrix instruction high, which suits: the products are a small part of the
// time, and the instruction takes its operands from registers, so keys and
// values go from global memory to the registers that use them and never
// through shared memory.  Two orders are chosen freely to make that so:
//   - scores: the feature axis is summed over, so lane (g, t) of eight rows
//     by four takes the 16-byte chunks t, t + 4, ... of key row g whole, and
//     the query operand is loaded in the same order;
//   - output: lane (g, t) loads chunk g of the four key rows whose
//     probabilities it holds, and feature e of every chunk goes to the e-th
//     accumulator, so pairs of rows are interleaved in registers.
//
// Each warp keeps its own maximum and sum.  They are joined over the block's
// warps in shared memory, and over the blocks that share the rows, one
// thread-block cluster, through distributed shared memory: one launch, no
// workspace, always in the same order.
#pragma once

#include <cooperative_groups.h>

#include "pba_cross_sm100.cuh"

namespace pba {

constexpr int kXsWarps = 4;
constexpr int kXsThreads = 32 * kXsWarps;
constexpr int kXsRows = 16;        // query rows of a block
constexpr int kXsKeys = 32;        // keys of a warp's step
constexpr int kXsMaxSplits = 8;    // blocks of a cluster (the portable limit)

struct CrossSplitParams {
  int32_t B, H, Hkv, group, Nq, Nk;
  int32_t row_tiles;  // ceil(group * Nq / 16)
  float tau;
  const uint16_t *q, *k, *v;
  int64_t q_sb, q_sh, q_sn, k_sb, k_sh, k_sn, v_sb, v_sh, v_sn;
  const int32_t *k_len;
  const uint8_t *mask;
  int64_t mask_sb;
  uint16_t *out;
  int64_t out_sb, out_sh, out_sn;
  float *lse;
  int64_t lse_sb, lse_sh, lse_sn;
};

// C[16 x 8] += A[16 x 16] B[16 x 8], bf16 with fp32 sums.
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld_keep16(const void *p) {  // read once by this SM
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_keep8(const void *p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

template <int D>
struct CrossSplitSmem {
  // partial sums of the warps, then (in warp 0's place) of the block
  float o[kXsWarps][kXsRows][D + 4];
  float m[kXsWarps][kXsRows];
  float l[kXsWarps][kXsRows];
};

template <int D>
__global__ void __launch_bounds__(kXsThreads) pba_cross_split_kernel(const __grid_constant__ CrossSplitParams p) {
  constexpr int kChunks = D / 32;            // 16-byte chunks of a key row per lane
  constexpr int kSteps = D / 16;             // matrix instructions along the features
  constexpr int kCols = D / 8;               // output accumulators: feature = kCols * column + accumulator, column 0..7
  constexpr int kWords = kCols / 2;          // 4-byte words of a value row per lane
  __shared__ CrossSplitSmem<D> sm;
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int splits = int(cluster.num_blocks()), split = int(cluster.block_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int unit = blockIdx.x / splits;
  const int tile = unit % p.row_tiles, bh = unit / p.row_tiles;
  const int hk = bh % p.Hkv, b = bh / p.Hkv;
  const int rows = p.group * p.Nq;
  const int keys = cross_keys(p.k_len, b, p.Nk);

  // query rows g and g + 8 of the tile as the first operand of every step
  uint32_t qa[kSteps][4];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = tile * kXsRows + g + 8 * half;
    const int hr = r / p.Nq;
    const uint16_t *src = p.q + b * p.q_sb + (int64_t(hk) * p.group + hr) * p.q_sh + int64_t(r - hr * p.Nq) * p.q_sn;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < rows) v = __ldg(reinterpret_cast<const uint4 *>(src + 8 * (t + 4 * i)));
      qa[2 * i][half] = v.x;
      qa[2 * i][2 + half] = v.y;
      qa[2 * i + 1][half] = v.z;
      qa[2 * i + 1][2 + half] = v.w;
    }
  }

  // this block's keys, and within them every kXsWarps-th step for the warp
  const int steps = (keys + kXsKeys - 1) / kXsKeys;
  const int per = (steps + splits - 1) / splits;
  const int s_end = min(steps, (split + 1) * per);
  const uint16_t *kb = p.k + b * p.k_sb + hk * p.k_sh, *vb = p.v + b * p.v_sb + hk * p.v_sh;
  const uint8_t *mrow = p.mask == nullptr ? nullptr : p.mask + b * p.mask_sb;
  const float c_s = p.tau * kXLog2e;
  float o[kCols][4] = {};
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  for (int s = split * per + warp; s < s_end; s += kXsWarps) {
    const int key0 = s * kXsKeys;
    // bit i: key key0 + i takes part; the others are neither read nor used
    uint32_t keep = keys - key0 >= 32 ? 0xFFFFFFFFu : (1u << (keys - key0)) - 1u;
    if (mrow != nullptr) {
      const bool on = key0 + lane < keys && __ldg(mrow + key0 + lane) != 0;
      keep &= __ballot_sync(0xffffffffu, on);
    }
    uint4 kr[4][kChunks];
    uint32_t vr[4][4][kWords];  // [16-key half and pair][row of the pair ...]: rows 2t, 2t+1, 2t+8, 2t+9 of each 16
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int key = 8 * n + g;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        kr[n][i] = make_uint4(0, 0, 0, 0);
        if ((keep >> key) & 1u) kr[n][i] = ld_keep16(kb + int64_t(key0 + key) * p.k_sn + 8 * (t + 4 * i));
      }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = 8 * n + 2 * t + e;
        uint32_t *w = vr[n][e];
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
        if ((keep >> key) & 1u) {
          const uint16_t *src = vb + int64_t(key0 + key) * p.v_sn + kCols * g;
          if (kWords == 2) {
            const uint2 x = ld_keep8(src);
            w[0] = x.x, w[1] = x.y;
          } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
              const uint4 x = ld_keep16(src + 2 * i);
              w[i] = x.x, w[i + 1 < kWords ? i + 1 : 0] = x.y, w[i + 2 < kWords ? i + 2 : 0] = x.z,
              w[i + 3 < kWords ? i + 3 : 0] = x.w;
            }
          }
        }
      }
    }
    // scores of 16 rows by 32 keys
    float sc[4][4] = {};
#pragma unroll
    for (int n = 0; n < 4; ++n) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        mma_16816(sc[n], qa[2 * i], kr[n][i].x, kr[n][i].y);
        mma_16816(sc[n], qa[2 * i + 1], kr[n][i].z, kr[n][i].w);
      }
    }
    if (keep != 0xFFFFFFFFu) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!((keep >> (8 * n + 2 * t + (e & 1))) & 1u)) sc[n][e] = -INFINITY;
    }
    uint32_t pa[2][4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float mx = fmaxf(sc[0][2 * half], sc[0][2 * half + 1]);
#pragma unroll
      for (int n = 1; n < 4; ++n) mx = max3f(mx, sc[n][2 * half], sc[n][2 * half + 1]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float m_new = fmaxf(m[half], mx);
      const float neg = m_new == -INFINITY ? 0.f : -m_new * c_s;
      const float alpha = m[half] == -INFINITY ? 0.f : ex2_approx(fmaf(m[half], c_s, neg));
      m[half] = m_new;
      l[half] *= alpha;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        o[c][2 * half] *= alpha;
        o[c][2 * half + 1] *= alpha;
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float a = ex2_approx(fmaf(sc[n][2 * half], c_s, neg));
        const float d = ex2_approx(fmaf(sc[n][2 * half + 1], c_s, neg));
        l[half] += a + d;
        pa[n >> 1][(n & 1) * 2 + half] = pack_bf16x2(a, d);
      }
    }
    // output: 16 keys at a time, rows 2t and 2t+1 of each eight interleaved
#pragma unroll
    for (int h16 = 0; h16 < 2; ++h16) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint32_t a0 = vr[2 * h16][0][i], a1 = vr[2 * h16][1][i];
        const uint32_t b0 = vr[2 * h16 + 1][0][i], b1 = vr[2 * h16 + 1][1][i];
        mma_16816(o[2 * i], pa[h16], __byte_perm(a0, a1, 0x5410), __byte_perm(b0, b1, 0x5410));
        mma_16816(o[2 * i + 1], pa[h16], __byte_perm(a0, a1, 0x7632), __byte_perm(b0, b1, 0x7632));
      }
    }
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
    const int r = g + 8 * half;
    if (t == 0) {
      sm.m[warp][r] = m[half];
      sm.l[warp][r] = l[half];
    }
    // column 2t (+1) of accumulator c is feature kCols * column + c
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      sm.o[warp][r][kCols * (2 * t) + c] = o[c][2 * half];
      sm.o[warp][r][kCols * (2 * t + 1) + c] = o[c][2 * half + 1];
    }
  }
  cluster.sync();
  // join: the cluster's blocks share out the rows, each row's partials taken
  // in the order of block and warp
  for (int at = split * kXsThreads + threadIdx.x; at < kXsRows * (D / 4); at += splits * kXsThreads) {
    const int r = at / (D / 4), c = (at - r * (D / 4)) * 4;
    float mm = -INFINITY;
    for (int s = 0; s < splits; ++s) {
      const CrossSplitSmem<D> *o_sm = cluster.map_shared_rank(&sm, s);
#pragma unroll
      for (int w = 0; w < kXsWarps; ++w) mm = fmaxf(mm, o_sm->m[w][r]);
    }
    float ll = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mm != -INFINITY) {
      for (int s = 0; s < splits; ++s) {
        const CrossSplitSmem<D> *o_sm = cluster.map_shared_rank(&sm, s);
#pragma unroll
        for (int w = 0; w < kXsWarps; ++w) {
          const float mw = o_sm->m[w][r];
          const float a = mw == -INFINITY ? 0.f : ex2_approx((mw - mm) * c_s);
          const float4 x = *reinterpret_cast<const float4 *>(&o_sm->o[w][r][c]);
          ll = fmaf(a, o_sm->l[w][r], ll);
          acc.x = fmaf(a, x.x, acc.x);
          acc.y = fmaf(a, x.y, acc.y);
          acc.z = fmaf(a, x.z, acc.z);
          acc.w = fmaf(a, x.w, acc.w);
        }
      }
    }
    const float inv = ll > 0.f ? 1.f / ll : 0.f;
    const int row = tile * kXsRows + r;
    if (row < rows) {
      const int hr = row / p.Nq, h = hk * p.group + hr, i = row - hr * p.Nq;
      uint2 w = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      *reinterpret_cast<uint2 *>(p.out + b * p.out_sb + h * p.out_sh + int64_t(i) * p.out_sn + c) = w;
      if (c == 0 && p.lse != nullptr)
        p.lse[b * p.lse_sb + h * p.lse_sh + int64_t(i) * p.lse_sn] =
            ll > 0.f ? fmaf(mm, p.tau, logf(ll)) : -INFINITY;
    }
  }
  cluster.sync();  // no block leaves while another reads its shared memory
}

}  // namespace pba
