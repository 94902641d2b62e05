// pba_relpos.cuh -- the learned relative position bias by buckets, and the
// gradient of its table.
//
//     out[b][h][i][j] = table[r(b,i,j)][h]  (+ base[b][h][i][j])
//     dtable[r][h]    = sum of dout[b][h][i][j] over the (b,i,j) with r(b,i,j) = r
//
// r is a function of the distance k_pos[j] - q_pos[i]: clipped, or logarithmic
// beyond the exact small distances, with one more row for pairs of different
// groups (chains).  The bias of pair-biased attention ("Fold-CP: A Context
// Parallelism Framework for Biomolecular Modeling", Table 1 "Attn Pair Bias")
// is this matrix or has it added; the pages name no rule for the positions.
//
// Both directions are bound by the N^2 H elements written (and read, with a
// base) or read, so the row of the table is found once per pair of positions
// and the arithmetic per element is a shared-memory read and a store.
#pragma once

#include "pba_vec8.cuh"

namespace pba {

constexpr int kRelposMaxRows = 1025;     // rows of the table
constexpr int kRelposMaxBorders = 512;   // borders of the logarithmic rows of one side
constexpr int kRelposThreads = 256;
constexpr int kRelposGradThreads = 128;

struct RelposRule {
  int32_t kind;       // 0 clipped, 1 logarithmic on both sides, 2 logarithmic, keys behind the query
  int32_t radius;     // clipped: rows are clamp(rel, -radius, radius) + radius
  int32_t exact;      // logarithmic: distances below it have rows of their own
  int32_t side;       // logarithmic: rows of one side
  int32_t n_borders;  // side - exact - 1
  int32_t cross;      // row of pairs of different groups (-1 without groups)
  // borders[t]: smallest distance of row exact + 1 + t
  int32_t borders[kRelposMaxBorders];
};

struct RelposParams {
  int32_t B, H, Nq, Nk;
  int32_t rows;              // rows of the table
  int32_t heads_per_block;   // forward: even for bf16, heads a block writes
  int32_t pos_vec;           // k_pos and k_group chunks readable as 16-byte words
  const int32_t *q_pos, *k_pos, *q_group, *k_group;
  int64_t q_sb, k_sb, qg_sb, kg_sb;  // batch strides (0: shared by the batch)
  const void *table;         // [rows][H]
  const void *base;          // forward, or null
  int64_t base_s[3];
  void *out;                 // forward: out; backward: dout (read)
  int64_t out_s[3];
  // backward
  float *part;               // [H][splits][rows]
  int32_t splits, row_splits, col_blocks, cols_log2;
  RelposRule rule;
};

// Row of the table for a distance rel = k_pos - q_pos (saturated, so that
// positions at the ends of the 32-bit range keep their order).
__device__ __forceinline__ int sub_sat(int a, int b) {
  int r;
  asm("sub.sat.s32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ int relpos_row(const RelposRule &r, const int *borders, int rel) {
  if (r.kind == 0) return min(max(rel, -r.radius), r.radius) + r.radius;
  rel = max(rel, -2147483647);
  const int d = r.kind == 1 ? abs(rel) : max(-rel, 0);
  int row = d;
  if (d >= r.exact) {
    // number of borders at or below d
    int lo = 0, hi = r.n_borders;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (borders[mid] <= d)
        lo = mid + 1;
      else
        hi = mid;
    }
    row = r.exact + lo;
  }
  return row + ((r.kind == 1 && rel > 0) ? r.side : 0);
}

// The positions (or groups) of keys c .. c+7, those past Nk as the last key.
__device__ __forceinline__ void load_keys8(const int32_t *p, int c, int Nk, bool vec, int (&k)[8]) {
  if (vec && c + 8 <= Nk) {
    const int4 a = __ldg(reinterpret_cast<const int4 *>(p + c)), b = __ldg(reinterpret_cast<const int4 *>(p + c + 4));
    k[0] = a.x, k[1] = a.y, k[2] = a.z, k[3] = a.w, k[4] = b.x, k[5] = b.y, k[6] = b.z, k[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) k[e] = __ldg(p + min(c + e, Nk - 1));
  }
}

// Forward.  A thread owns eight consecutive keys of one (batch, query): it
// finds their eight rows once and writes them for every head of the block.
// The block's columns of the table wait in shared memory, row-contiguous, so
// that neighbouring distances fall into neighbouring banks; bf16 keeps two
// heads per word, one read serving both.
template <typename T, bool kVec, bool kBase>
__global__ void __launch_bounds__(kRelposThreads) relpos_fwd_kernel(const __grid_constant__ RelposParams p) {
  constexpr bool kBf = sizeof(typename T::Word) == 2;
  constexpr int kHeadsPerWord = kBf ? 2 : 1;
  extern __shared__ uint32_t relpos_smem[];
  int *borders = reinterpret_cast<int *>(relpos_smem);
  uint32_t *tab = relpos_smem + p.rule.n_borders;
  const int h0 = blockIdx.y * p.heads_per_block;
  const int nh = min(p.heads_per_block, p.H - h0);
  const int words = (nh + kHeadsPerWord - 1) / kHeadsPerWord;
  for (int i = threadIdx.x; i < p.rule.n_borders; i += kRelposThreads) borders[i] = p.rule.borders[i];
  for (int i = threadIdx.x; i < words * p.rows; i += kRelposThreads) {
    const int w = i / p.rows, r = i - w * p.rows;
    if (kBf) {
      const uint16_t *t = static_cast<const uint16_t *>(p.table) + int64_t(r) * p.H + h0 + 2 * w;
      tab[i] = uint32_t(t[0]) | (2 * w + 1 < nh ? uint32_t(t[1]) << 16 : 0u);
    } else {
      tab[i] = static_cast<const uint32_t *>(p.table)[int64_t(r) * p.H + h0 + w];
    }
  }
  __syncthreads();

  const int chunks = (p.Nk + 7) >> 3;
  const int64_t total = int64_t(p.B) * p.Nq * chunks;
  const int64_t first = int64_t(blockIdx.x) * kRelposThreads + threadIdx.x;
  const int64_t step = int64_t(gridDim.x) * kRelposThreads;
  if (first >= total) return;
  // (batch, query) row and key chunk, advanced without a division
  int row = int(first / chunks), col = int(first - int64_t(row) * chunks);
  const int drow = int(step / chunks), dcol = int(step - int64_t(drow) * chunks);
  for (int64_t at = first; at < total; at += step) {
    const int b = row / p.Nq, i = row - b * p.Nq;
    const int c = col * 8, n = min(8, p.Nk - c);
    int r[8];
    {
      int k[8];
      load_keys8(p.k_pos + b * p.k_sb, c, p.Nk, p.pos_vec != 0, k);
      const int q = __ldg(p.q_pos + b * p.q_sb + i);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = relpos_row(p.rule, borders, sub_sat(k[e], q));
      if (p.rule.cross >= 0) {
        load_keys8(p.k_group + b * p.kg_sb, c, p.Nk, p.pos_vec != 0, k);
        const int qg = __ldg(p.q_group + b * p.qg_sb + i);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = k[e] == qg ? r[e] : p.rule.cross;
      }
    }
    using W = typename T::Word;
    W *out = static_cast<W *>(p.out) + b * p.out_s[0] + h0 * p.out_s[1] + int64_t(i) * p.out_s[2] + c;
    const W *base = kBase ? static_cast<const W *>(p.base) + b * p.base_s[0] + h0 * p.base_s[1] +
                                int64_t(i) * p.base_s[2] + c
                          : nullptr;
#pragma unroll 2
    for (int w = 0; w < words; ++w) {
      const uint32_t *t = tab + w * p.rows;
      uint32_t v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = t[r[e]];
#pragma unroll
      for (int s = 0; s < kHeadsPerWord; ++s) {
        const int h = w * kHeadsPerWord + s;
        if (h >= nh) break;
        float x[8];
        if (kBase) load8<T, kVec>(base + h * p.base_s[1], n, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float tv = !kBf ? __uint_as_float(v[e]) : (s == 0 ? bf16lo_to_f32(v[e]) : bf16hi_to_f32(v[e]));
          x[e] = kBase ? x[e] + tv : tv;
        }
        store8<T, kVec>(out + h * p.out_s[1], n, x);
      }
    }
    row += drow;
    col += dcol;
    if (col >= chunks) {
      col -= chunks;
      ++row;
    }
  }
}

// Backward.  A block takes one head, a block of keys and a share of the
// queries; a thread keeps eight keys and walks down the queries.  Most eights
// lie wholly in one of three rows: past the last border on either side, or in
// another group.  Their sums stay in three registers.  The others go element
// by element into the thread's own column of a table in shared memory, so no
// two threads ever add to the same word and the order of every sum is fixed.
// The columns are added at the end of the block, the blocks' tables by
// relpos_grad_sum_kernel.
template <typename T, bool kVec>
__global__ void relpos_grad_kernel(const __grid_constant__ RelposParams p) {
  extern __shared__ uint32_t relpos_smem[];
  int *borders = reinterpret_cast<int *>(relpos_smem);
  float *hist = reinterpret_cast<float *>(relpos_smem + p.rule.n_borders);
  const int threads = blockDim.x, tid = threadIdx.x;
  for (int i = tid; i < p.rule.n_borders; i += threads) borders[i] = p.rule.borders[i];
  for (int i = tid; i < p.rows * threads; i += threads) hist[i] = 0.f;
  __syncthreads();

  const int h = blockIdx.y, b = blockIdx.z;
  const int col_block = blockIdx.x % p.col_blocks, row_split = blockIdx.x / p.col_blocks;
  const int cols = 1 << p.cols_log2;  // threads along the keys; the others take further queries
  const int c = ((col_block << p.cols_log2) + (tid & (cols - 1))) * 8;
  const int lanes = threads >> p.cols_log2, lane_row = tid >> p.cols_log2;
  const int n = min(8, p.Nk - c);
  if (n > 0) {
    // a distance at or past these lies in the last row of its side
    const RelposRule &rule = p.rule;
    const int far = rule.kind == 0 ? rule.radius : (rule.n_borders > 0 ? rule.borders[rule.n_borders - 1] : rule.exact);
    // one-sided: keys ahead of the query all share row 0
    const int far_hi = rule.kind == 2 ? 0 : far;
    const int row_lo = rule.kind == 0 ? 0 : rule.side - 1;
    const int row_hi = rule.kind == 0 ? 2 * rule.radius : (rule.kind == 1 ? 2 * rule.side - 1 : 0);
    int k[8], kg[8];
    load_keys8(p.k_pos + b * p.k_sb, c, p.Nk, p.pos_vec != 0, k);
    const bool groups = rule.cross >= 0;
    if (groups) load_keys8(p.k_group + b * p.kg_sb, c, p.Nk, p.pos_vec != 0, kg);
    int k_min = k[0], k_max = k[0];
    bool one_group = true;
#pragma unroll
    for (int e = 1; e < 8; ++e) {
      k_min = min(k_min, k[e]);
      k_max = max(k_max, k[e]);
      if (groups) one_group = one_group && kg[e] == kg[0];
    }
    float lo = 0.f, hi = 0.f, cross = 0.f;
    const int per = (p.Nq + p.row_splits - 1) / p.row_splits;
    const int i_end = min(p.Nq, (row_split + 1) * per);
    using W = typename T::Word;
    const W *src = static_cast<const W *>(p.out) + b * p.out_s[0] + h * p.out_s[1] + c;
    const int32_t *qp = p.q_pos + b * p.q_sb, *qgp = groups ? p.q_group + b * p.qg_sb : nullptr;
    constexpr int kAhead = 4;
    for (int i0 = row_split * per + lane_row; i0 < i_end; i0 += kAhead * lanes) {
      float x[kAhead][8];
      int q[kAhead], qg[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int i = i0 + a * lanes;
        if (i < i_end) {
          load8<T, kVec>(src + int64_t(i) * p.out_s[2], n, x[a]);
          q[a] = __ldg(qp + i);
          qg[a] = groups ? __ldg(qgp + i) : 0;
        }
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (i0 + a * lanes >= i_end) break;
        const float sum = ((x[a][0] + x[a][1]) + (x[a][2] + x[a][3])) + ((x[a][4] + x[a][5]) + (x[a][6] + x[a][7]));
        if (groups && one_group && kg[0] != qg[a]) {
          cross += sum;
        } else if ((!groups || one_group) && sub_sat(k_min, q[a]) >= far_hi) {
          hi += sum;
        } else if ((!groups || one_group) && sub_sat(k_max, q[a]) <= -far) {
          lo += sum;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            int r = relpos_row(rule, borders, sub_sat(k[e], q[a]));
            if (groups && kg[e] != qg[a]) r = rule.cross;
            hist[r * threads + tid] += x[a][e];
          }
        }
      }
    }
    hist[row_lo * threads + tid] += lo;
    hist[row_hi * threads + tid] += hi;
    if (groups) hist[rule.cross * threads + tid] += cross;
  }
  __syncthreads();
  const int warp = tid >> 5, lane = tid & 31, warps = threads >> 5;
  const int split = b * (p.row_splits * p.col_blocks) + blockIdx.x;
  for (int r = warp; r < p.rows; r += warps) {
    float s = 0.f;
    for (int i = lane; i < threads; i += 32) s += hist[r * threads + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) p.part[(int64_t(h) * p.splits + split) * p.rows + r] = s;
  }
}

// dtable[r][h] = sum of the blocks' tables, in 64 bits: thread (x, y) of a
// block adds every blockDim.y-th table for row blockIdx.x * 32 + x.
__global__ void relpos_grad_sum_kernel(const float *part, float *dtable, int splits, int rows, int H) {
  __shared__ double acc[8][33];
  const int r = blockIdx.x * 32 + threadIdx.x, h = blockIdx.y;
  double s = 0.0;
  if (r < rows)
    for (int i = threadIdx.y; i < splits; i += 8) s += double(part[(int64_t(h) * splits + i) * rows + r]);
  acc[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && r < rows) {
#pragma unroll
    for (int y = 1; y < 8; ++y) s += acc[y][threadIdx.x];
    dtable[int64_t(r) * H + h] = float(s);
  }
}

}  // namespace pba
