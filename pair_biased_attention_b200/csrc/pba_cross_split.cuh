// pba_cross_split.cuh -- cross attention for few query rows (a decoder's new
// tokens): the same sums as pba_cross_sm100.cuh, arranged for reading the keys
// and values once at full bandwidth.
//
// The query rows of the heads that share a key head (H / Hkv x Nq of them) are
// one matrix; a block takes 16 of its rows and a share of the keys, and each
// warp works on keys of its own, 16 at a time, which it copies ahead into its
// own ring in shared memory (about 190 KB on their way per SM; loads straight
// into registers, 8 KB a warp, left HBM at 0.42 of its rate).  16 rows are one
// warp-level matrix instruction high, which suits: the products are a small
// part of the time.  Two orders are chosen freely so that every operand is read
// from shared memory in 16-byte words:
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
//
// P is rounded to bf16 for the product with V, the sum is taken unrounded, as in
// pba_cross_sm100.cuh.
//
// Measured: one token of 16 sequences, 16 heads on 4, D = 64, up to 8192 keys
// (98.6 MB of keys and values): 23 us, 4.2 TB/s, with the launch, the joins and
// the uneven lengths in it.  At most eight blocks share 16 rows, so that few heads
// of one sequence leave SMs idle: 8 heads on 131072 keys 108 us, 2.5 TB/s from 64
// blocks.
#pragma once

#include "pba_cross_sm100.cuh"

namespace pba {

constexpr int kXsWarps = 4;
constexpr int kXsThreads = 32 * kXsWarps;
constexpr int kXsRows = 16;        // query rows of a block
constexpr int kXsKeys = 16;        // keys of a warp's step
// Blocks on an SM and steps under way per warp, by what registers and shared
// memory allow.
template <int D>
struct CrossSplitShape {
  static constexpr int kBlocksPerSm = D == 128 ? 2 : 4;
  static constexpr int kStages = D == 32 ? 6 : 3;
};

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

// A ring of steps per warp: [stage][K, V][16 keys][D] bf16, the 16-byte chunks
// of a row in an order that lets both kinds of reads touch all banks.
template <int D>
struct CrossRing {
  static constexpr int kRowChunks = D / 8;
  static constexpr int kTileBytes = kXsKeys * D * 2;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = CrossSplitShape<D>::kStages;
  static __device__ __forceinline__ int chunk_at(int row, int chunk) {
    return row * D * 2 + ((D == 32 ? chunk ^ ((row >> 1) & 3) : chunk ^ ((row >> 1) & 3) * 2 ^ (row & 1) * 4) << 4);
  }
};

// What the block's warps leave for the join; it takes the ring's place.
template <int D>
struct CrossSplitSmem {
  float o[kXsWarps][kXsRows][D + 4];
  float m[kXsWarps][kXsRows];
  float l[kXsWarps][kXsRows];
  float2 joined[kXsRows];  // maximum and sum of the block
};

template <int D>
constexpr int cross_split_smem() {
  constexpr int ring = kXsWarps * CrossRing<D>::kStages * CrossRing<D>::kStageBytes;
  constexpr int join = int(sizeof(CrossSplitSmem<D>));
  return ring > join ? ring : join;
}

template <int D>
__global__ void __launch_bounds__(kXsThreads, CrossSplitShape<D>::kBlocksPerSm)
    pba_cross_split_kernel(const __grid_constant__ CrossSplitParams p) {
  using Ring = CrossRing<D>;
  constexpr int kChunks = D / 32;            // 16-byte chunks of a key row per lane
  constexpr int kSteps = D / 16;             // matrix instructions along the features
  constexpr int kCols = D / 8;               // output accumulators: feature = kCols * column + accumulator, column 0..7
  constexpr int kWords = kCols / 2;          // 4-byte words of a value row per lane
  extern __shared__ __align__(16) uint8_t ring_smem[];
  CrossSplitSmem<D> &sm = *reinterpret_cast<CrossSplitSmem<D> *>(ring_smem);
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

  // this block's keys, and within them every kXsWarps-th step for the warp
  const int steps = (keys + kXsKeys - 1) / kXsKeys;
  const int per = (steps + splits - 1) / splits;
  const int s_begin = split * per + warp, s_end = min(steps, (split + 1) * per);
  const uint16_t *kb = p.k + b * p.k_sb + hk * p.k_sh, *vb = p.v + b * p.v_sb + hk * p.v_sh;
  const uint8_t *mrow = p.mask == nullptr ? nullptr : p.mask + b * p.mask_sb;
  uint8_t *ring = ring_smem + warp * Ring::kStages * Ring::kStageBytes;
  // Copies the 16 keys of the next step: a lane takes the same chunk of every
  // kLaneRows-th row.  Keys past the end are not read and become zeros.
  constexpr int kLaneRows = 32 / Ring::kRowChunks, kCopies = kXsKeys / kLaneRows;
  const int lane_row = lane / Ring::kRowChunks, lane_chunk = lane % Ring::kRowChunks;
  const uint16_t *k_at = kb + (int64_t(s_begin) * kXsKeys + lane_row) * p.k_sn + lane_chunk * 8;
  const uint16_t *v_at = vb + (int64_t(s_begin) * kXsKeys + lane_row) * p.v_sn + lane_chunk * 8;
  int s_next = s_begin;
  auto fetch = [&](int stage) {
    if (s_next < s_end) {
      uint8_t *kt = ring + stage * Ring::kStageBytes, *vt = kt + Ring::kTileBytes;
      if ((s_next + 1) * kXsKeys <= keys) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          const int to = Ring::chunk_at(i * kLaneRows + lane_row, lane_chunk);
          cp_async16(kt + to, k_at + i * kLaneRows * p.k_sn);
          cp_async16(vt + to, v_at + i * kLaneRows * p.v_sn);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          const int row = i * kLaneRows + lane_row, to = Ring::chunk_at(row, lane_chunk);
          const bool ok = s_next * kXsKeys + row < keys;
          cp_async16_part(kt + to, ok ? k_at + i * kLaneRows * p.k_sn : kb, ok ? 16 : 0);
          cp_async16_part(vt + to, ok ? v_at + i * kLaneRows * p.v_sn : vb, ok ? 16 : 0);
        }
      }
      s_next += kXsWarps;
      k_at += kXsWarps * kXsKeys * p.k_sn;
      v_at += kXsWarps * kXsKeys * p.v_sn;
    }
    cp_async_commit();
  };
  auto mask_byte = [&](int s) -> uint32_t {  // lane i: key i of the step
    const int key = s * kXsKeys + (lane & 15);
    if (mrow == nullptr || key >= keys) return key < keys ? 1u : 0u;
    return __ldg(mrow + key);
  };
#pragma unroll
  for (int i = 0; i < Ring::kStages; ++i) fetch(i);
  uint32_t next_mask = mask_byte(s_begin);

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

  const float c_s = p.tau * kXLog2e;
  float o[kCols][4] = {};
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  int stage = 0;
  for (int s = s_begin; s < s_end; s += kXsWarps) {
    // bit i: key i of the step takes part
    const uint32_t keep = __ballot_sync(0xffffffffu, next_mask != 0) & 0xFFFFu;
    next_mask = mask_byte(s + kXsWarps);
    cp_async_wait<Ring::kStages - 1>();
    __syncwarp();
    const uint8_t *kt = ring + stage * Ring::kStageBytes, *vt = kt + Ring::kTileBytes;
    // scores of 16 rows by 16 keys
    float sc[2][4] = {};
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const uint4 kr = *reinterpret_cast<const uint4 *>(kt + Ring::chunk_at(8 * n + g, t + 4 * i));
        mma_16816(sc[n], qa[2 * i], kr.x, kr.y);
        mma_16816(sc[n], qa[2 * i + 1], kr.z, kr.w);
      }
    }
    // value rows 2t, 2t + 1 (then + 8), features kCols g ... of each
    uint32_t vr[2][2][kWords];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * n + 2 * t + e;
        if (kWords == 2) {
          const uint2 x = *reinterpret_cast<const uint2 *>(vt + Ring::chunk_at(row, g >> 1) + (g & 1) * 8);
          vr[n][e][0] = x.x, vr[n][e][1] = x.y;
        } else {
#pragma unroll
          for (int i = 0; i < kWords; i += 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(vt + Ring::chunk_at(row, g * (kWords / 4) + i / 4));
            vr[n][e][i] = x.x, vr[n][e][(i + 1) % kWords] = x.y, vr[n][e][(i + 2) % kWords] = x.z,
            vr[n][e][(i + 3) % kWords] = x.w;
          }
        }
      }
    }
    if (keep != 0xFFFFu) {
      // whatever the others hold: their scores are -inf, their values 0
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!((keep >> (8 * n + 2 * t + (e & 1))) & 1u)) sc[n][e] = -INFINITY;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!((keep >> (8 * n + 2 * t + e)) & 1u)) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) vr[n][e][i] = 0;
          }
      }
    }
    __syncwarp();  // the stage has been read
    fetch(stage);
    stage = stage + 1 == Ring::kStages ? 0 : stage + 1;
    uint32_t pa[4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float mx = fmaxf(fmaxf(sc[0][2 * half], sc[0][2 * half + 1]), fmaxf(sc[1][2 * half], sc[1][2 * half + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float m_new = fmaxf(m[half], mx);
      const float neg = m_new == -INFINITY ? 0.f : -m_new * c_s;
      if (m_new != m[half]) {  // the maximum has risen
        const float alpha = m[half] == -INFINITY ? 0.f : ex2_approx(fmaf(m[half], c_s, neg));
        m[half] = m_new;
        l[half] *= alpha;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          o[c][2 * half] *= alpha;
          o[c][2 * half + 1] *= alpha;
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float a = ex2_approx(fmaf(sc[n][2 * half], c_s, neg));
        const float d = ex2_approx(fmaf(sc[n][2 * half + 1], c_s, neg));
        l[half] += a + d;
        pa[n * 2 + half] = pack_bf16x2(a, d);
      }
    }
    // output: rows 2t and 2t+1 of each eight interleaved
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      mma_16816(o[2 * i], pa, __byte_perm(vr[0][0][i], vr[0][1][i], 0x5410),
                __byte_perm(vr[1][0][i], vr[1][1][i], 0x5410));
      mma_16816(o[2 * i + 1], pa, __byte_perm(vr[0][0][i], vr[0][1][i], 0x7632),
                __byte_perm(vr[1][0][i], vr[1][1][i], 0x7632));
    }
  }
  cp_async_wait<0>();
  __syncthreads();  // the ring's memory now takes the partial sums
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
  // join over the block's warps, into warp 0's place
  const int live = min(kXsRows, rows - tile * kXsRows);  // rows of the tile that exist
  __syncthreads();
  for (int at = threadIdx.x; at < live * (D / 4); at += kXsThreads) {
    const int r = at / (D / 4), c = (at - r * (D / 4)) * 4;
    float mm = sm.m[0][r];
#pragma unroll
    for (int w = 1; w < kXsWarps; ++w) mm = fmaxf(mm, sm.m[w][r]);
    float ll = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kXsWarps; ++w) {
      const float mw = sm.m[w][r], a = mw == -INFINITY ? 0.f : ex2_approx((mw - mm) * c_s);
      const float4 x = *reinterpret_cast<const float4 *>(&sm.o[w][r][c]);
      ll = fmaf(a, sm.l[w][r], ll);
      acc.x = fmaf(a, x.x, acc.x);
      acc.y = fmaf(a, x.y, acc.y);
      acc.z = fmaf(a, x.z, acc.z);
      acc.w = fmaf(a, x.w, acc.w);
    }
    *reinterpret_cast<float4 *>(&sm.o[0][r][c]) = acc;
    if (c == 0) sm.joined[r] = make_float2(mm, ll);
  }
  cluster.sync();
  // join over the cluster's blocks, which share out the rows: every partial is
  // asked for before the first is used
  for (int at = split * kXsThreads + threadIdx.x; at < live * (D / 4); at += splits * kXsThreads) {
    const int r = at / (D / 4), c = (at - r * (D / 4)) * 4;
    float2 ml[kXMaxSplits];
    float4 x[kXMaxSplits];
#pragma unroll
    for (int s = 0; s < kXMaxSplits; ++s) {
      ml[s] = make_float2(-INFINITY, 0.f);
      x[s] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < splits) {
        const CrossSplitSmem<D> *o_sm = cluster.map_shared_rank(&sm, s);
        ml[s] = o_sm->joined[r];
        x[s] = *reinterpret_cast<const float4 *>(&o_sm->o[0][r][c]);
      }
    }
    float mm = ml[0].x;
#pragma unroll
    for (int s = 1; s < kXMaxSplits; ++s) mm = fmaxf(mm, ml[s].x);
    float ll = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < kXMaxSplits; ++s) {
      const float a = ml[s].x == -INFINITY ? 0.f : ex2_approx((ml[s].x - mm) * c_s);
      ll = fmaf(a, ml[s].y, ll);
      acc.x = fmaf(a, x[s].x, acc.x);
      acc.y = fmaf(a, x[s].y, acc.y);
      acc.z = fmaf(a, x[s].z, acc.z);
      acc.w = fmaf(a, x[s].w, acc.w);
    }
    const float inv = ll == 0.f ? 0.f : 1.f / ll;  // 0: no key
    const int row = tile * kXsRows + r;
    const int hr = row / p.Nq, h = hk * p.group + hr, i = row - hr * p.Nq;
    const uint2 w = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2 *>(p.out + b * p.out_sb + h * p.out_sh + int64_t(i) * p.out_sn + c) = w;
    if (c == 0 && p.lse != nullptr)
      p.lse[b * p.lse_sb + h * p.lse_sh + int64_t(i) * p.lse_sn] = ll == 0.f ? -INFINITY : fmaf(mm, p.tau, logf(ll));
  }
  cluster.sync();  // no block leaves while another reads its shared memory
}

}  // namespace pba
