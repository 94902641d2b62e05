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
// Both directions read or write N^2 H elements (and the base), so the row of
// the table is found once per pair of positions for all heads, and the
// arithmetic per element is a shared-memory read and a store, or an addition.
#pragma once

#include "pba_vec8.cuh"

namespace pba {

constexpr int kRelposMaxRows = 1025;     // rows of the table
constexpr int kRelposLutFar = 2048;      // farthest last border that is looked up by distance
constexpr int kRelposMaxBorders = 512;   // borders of the logarithmic rows of one side
constexpr int kRelposThreads = 256;
constexpr int kRelposBaseStages = 8;     // heads of the base on their way, per thread
constexpr int kRelposGradThreads = 128;

struct RelposRule {
  int32_t kind;       // 0 clipped, 1 logarithmic on both sides, 2 logarithmic, keys behind the query
  int32_t far;        // a distance at or past it lies in the last row of its side (clipped: the radius)
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
  int32_t ring_offset;       // forward with an aligned base: where its ring lies in shared memory
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

__device__ __forceinline__ int sub_sat(int a, int b) {
  int r;
  asm("sub.sat.s32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ int add_sat(int a, int b) {
  int r;
  asm("add.sat.s32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The table's row of a distance rel in [-far, far]; every distance beyond has
// the row of the nearer end.  Clipped: rel + far.  Logarithmic: looked up in
// shared memory, by distance where that table is small enough (lut, 2 far + 1
// entries), else by searching the borders.
struct RelposLookup {
  const uint16_t *lut;
  const int *borders;
};
// Words of shared memory that the lookup needs.
__host__ __device__ inline int relpos_lookup_words(const RelposRule &r) {
  return r.kind == 0 ? 0 : (r.far <= kRelposLutFar ? r.far + 1 : r.n_borders);
}
__device__ __forceinline__ int relpos_search(const RelposRule &r, const int *borders, int rel) {
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
// Filled by the whole block; the caller synchronises.
__device__ __forceinline__ RelposLookup relpos_lookup(const RelposRule &r, uint32_t *smem, int tid, int threads) {
  if (r.kind != 0) {
    if (r.far <= kRelposLutFar) {
      for (int i = tid; i <= 2 * r.far; i += threads)
        reinterpret_cast<uint16_t *>(smem)[i] = uint16_t(relpos_search(r, r.borders, i - r.far));
    } else {
      for (int i = tid; i < r.n_borders; i += threads) smem[i] = uint32_t(r.borders[i]);
    }
  }
  return RelposLookup{reinterpret_cast<const uint16_t *>(smem), reinterpret_cast<const int *>(smem)};
}
__device__ __forceinline__ int relpos_row(const RelposRule &r, const RelposLookup &look, int rel) {
  if (r.kind == 0) return rel + r.far;
  if (r.far <= kRelposLutFar) return look.lut[rel + r.far];
  return relpos_search(r, look.borders, rel);
}

// The positions (or groups) of a thread's eight keys, consecutive (kVec)
// or every 32nd; those past the row as its last key.
template <bool kVec>
__device__ __forceinline__ void load_keys8(const int32_t *p, int c, int Nk, bool vec, int (&k)[8]) {
  if (kVec && vec && c + 8 <= Nk) {
    const int4 a = __ldg(reinterpret_cast<const int4 *>(p + c)), b = __ldg(reinterpret_cast<const int4 *>(p + c + 4));
    k[0] = a.x, k[1] = a.y, k[2] = a.z, k[3] = a.w, k[4] = b.x, k[5] = b.y, k[6] = b.z, k[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) k[e] = __ldg(p + min(kVec ? c + e : c + 32 * e, Nk - 1));
  }
}

// Forward.  A thread owns eight keys of one (batch, query), consecutive ones of
// bf16 rows on 16 bytes (kVec), else every 32nd of the 256 that its warp owns: it
// finds their eight rows once and writes them for every head of the block.
// The block's columns of the table wait in shared memory, row-contiguous, so
// that neighbouring distances fall into neighbouring banks; bf16 keeps two
// heads per word, one read serving both.
// Measured at 4096 x 4096 x 16 heads, bf16, with a base: 177 us, 6.1 TB/s, 0.92
// of a copy's rate; fp32 at 2048 x 2048 x 16 90 us, 6.0 TB/s.  Without the base's
// ring, its loads one head ahead in registers, that was 279 us.  Rows of 2047
// keys, bf16: 30 us against 23 for 2048, their last eight element by element.
template <typename T, bool kVec, bool kBase>
__global__ void __launch_bounds__(kRelposThreads) relpos_fwd_kernel(const __grid_constant__ RelposParams p) {
  constexpr bool kBf = sizeof(typename T::Word) == 2;
  constexpr int kHeadsPerWord = kBf ? 2 : 1;
  extern __shared__ uint32_t relpos_smem[];
  uint32_t *tab = relpos_smem + relpos_lookup_words(p.rule);
  const RelposLookup look = relpos_lookup(p.rule, relpos_smem, threadIdx.x, kRelposThreads);
  const int h0 = blockIdx.y * p.heads_per_block;
  const int nh = min(p.heads_per_block, p.H - h0);
  const int words = (nh + kHeadsPerWord - 1) / kHeadsPerWord;
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

  // a unit is a thread's eight keys, or a warp's 256
  const int lane = threadIdx.x & 31;
  const int chunks = kVec ? (p.Nk + 7) >> 3 : (p.Nk + 255) >> 8;
  const int64_t total = int64_t(p.B) * p.Nq * chunks;
  const int units = kVec ? kRelposThreads : kRelposThreads / 32;  // of a block
  const int64_t first = int64_t(blockIdx.x) * units + (kVec ? threadIdx.x : threadIdx.x >> 5);
  const int64_t step = int64_t(gridDim.x) * units;
  if (first >= total) return;
  // (batch, query) row and key chunk, advanced without a division
  int row = int(first / chunks), col = int(first - int64_t(row) * chunks);
  const int drow = int(step / chunks), dcol = int(step - int64_t(drow) * chunks);
  // Aligned rows of the base run ahead of their use through the thread's own
  // ring in shared memory, one head after the other and on into the thread's
  // next eights.
  constexpr int slot_bytes = Ring8<T, true>::kSlotWords * kRelposThreads * 16;
  uint8_t *ring = reinterpret_cast<uint8_t *>(relpos_smem) + p.ring_offset + threadIdx.x * 16;
  int stage = 0, a_row = row, a_col = col, a_h = 0;
  int64_t a_at = first;
  auto fetch = [&]() {
    if (a_at < total) {
      const int b = a_row / p.Nq, i = a_row - b * p.Nq, c = a_col * 8;
      const typename T::Word *src = static_cast<const typename T::Word *>(p.base) + b * p.base_s[0] +
                                    (h0 + a_h) * p.base_s[1] + int64_t(i) * p.base_s[2] + c;
      Ring8<T, true>::fetch(ring + stage * slot_bytes, kRelposThreads * 16, src, min(8, p.Nk - c), true);
      if (++a_h == nh) {
        a_h = 0;
        a_at += step;
        a_row += drow;
        a_col += dcol;
        if (a_col >= chunks) {
          a_col -= chunks;
          ++a_row;
        }
      }
    }
    cp_async_commit();
    stage = stage + 1 == kRelposBaseStages ? 0 : stage + 1;
  };
  if (kBase && kVec)
    for (int i = 0; i < kRelposBaseStages; ++i) fetch();
  for (int64_t at = first; at < total; at += step) {
    const int b = row / p.Nq, i = row - b * p.Nq;
    const int c = kVec ? col * 8 : col * 256 + lane;
    const int n = kVec ? min(8, p.Nk - c) : max(0, min(8, (p.Nk - c + 31) >> 5));
    int r[8];
    {
      int k[8];
      load_keys8<kVec>(p.k_pos + b * p.k_sb, c, p.Nk, p.pos_vec != 0, k);
      const int q = __ldg(p.q_pos + b * p.q_sb + i);
      // distances are clamped before they are taken: no overflow wherever the positions lie
      const int q_lo = sub_sat(q, p.rule.far), q_hi = add_sat(q, p.rule.far);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = relpos_row(p.rule, look, min(max(k[e], q_lo), q_hi) - q);
      if (p.rule.cross >= 0) {
        load_keys8<kVec>(p.k_group + b * p.kg_sb, c, p.Nk, p.pos_vec != 0, k);
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
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[e] = !kBf ? __uint_as_float(v[e]) : (s == 0 ? bf16lo_to_f32(v[e]) : bf16hi_to_f32(v[e]));
        if (kBase) {
          float y[8];
          if (kVec) {
            cp_async_wait<kRelposBaseStages - 1>();
            const Raw8<T> raw = Ring8<T, true>::take(ring + stage * slot_bytes, kRelposThreads * 16, nullptr, true);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[2 * i] = raw.pair(i).x, y[2 * i + 1] = raw.pair(i).y;
            fetch();
          } else {
            load8<T>(base + h * p.base_s[1], n, 32, y);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] += y[e];
        }
        if constexpr (kVec)
          store8_word(out + h * p.out_s[1], n, x);
        else
          store8<T>(out + h * p.out_s[1], n, 32, x);
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
// queries; a thread keeps eight consecutive keys and walks down the queries,
// its next rows on their way into its own ring in shared memory.
// While the queries' group stays the same, so does the set of the eight that
// share it: the others' values go to the row of different groups, kept in a
// register.  The set itself mostly lies past the last border on one side, and
// those two sums stay in registers as well.  Only near the diagonal are the
// values added one by one, into the thread's own column of a table in shared
// memory; a block's queries lie row_splits apart, so that every block meets its
// share of the diagonal.  No two threads add to the same word, and the order of
// every sum is fixed.  The columns are added at the end of the block, in fp32 (in
// 64 bits that took 3 to 15 % of the call, for eight additions next to a thread's
// 4096), the blocks' tables by relpos_grad_sum_kernel in 64 bits.
// Measured at 4096 x 4096 x 16 heads, bf16, 66 rows with two chains: 150 us,
// 3.6 TB/s, a little over half of HBM's rate; where most pairs are near (32 x 12
// heads x 512^2, logarithmic up to 512) 1.3 TB/s.  Some 80 instructions per eight
// elements, a tenth of them near the diagonal, are what bounds it, with four
// blocks to an SM by their tables; a deeper ring changed nothing.
template <typename T, bool kVec>
struct RelposGradRing {
  using R = Ring8<T, kVec>;
  static constexpr int kStages = 4;
  static constexpr int kThreadBytes = kStages * R::kSlotWords * 16 + 64;  // and the eight keys' positions and groups
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kRelposGradThreads, 4) relpos_grad_kernel(const __grid_constant__ RelposParams p) {
  using Ring = RelposGradRing<T, kVec>;
  using R = typename Ring::R;
  extern __shared__ __align__(16) uint8_t relpos_grad_smem[];
  const int threads = blockDim.x, tid = threadIdx.x;
  // [stage][word][thread] 16-byte words, [four keys][thread] positions, then
  // groups, the lookup, [row][thread] sums
  uint8_t *ring = relpos_grad_smem + tid * 16;
  int4 *keys = reinterpret_cast<int4 *>(relpos_grad_smem + threads * Ring::kStages * R::kSlotWords * 16) + tid;
  uint32_t *look_smem = reinterpret_cast<uint32_t *>(relpos_grad_smem + threads * Ring::kThreadBytes);
  float *hist = reinterpret_cast<float *>(look_smem + relpos_lookup_words(p.rule));
  const RelposLookup look = relpos_lookup(p.rule, look_smem, tid, threads);
  for (int i = tid; i < p.rows * threads; i += threads) hist[i] = 0.f;
  __syncthreads();

  const int h = blockIdx.y, b = blockIdx.z;
  const int col_block = blockIdx.x % p.col_blocks, row_split = blockIdx.x / p.col_blocks;
  const int cols = 1 << p.cols_log2;  // threads along the keys; the others take further queries
  const int c = ((col_block << p.cols_log2) + (tid & (cols - 1))) * 8;
  const int lanes = threads >> p.cols_log2, lane_row = tid >> p.cols_log2;
  const int n = min(8, p.Nk - c);
  if (n > 0) {
    const RelposRule &rule = p.rule;
    // one-sided: keys ahead of the query all share row 0
    const int far = rule.far, far_hi = rule.kind == 2 ? 0 : far;
    const bool groups = rule.cross >= 0;
    // The keys' positions and groups wait in shared memory for where single
    // ones are needed; what stays in registers is which of the eight are
    // members of the queries' group, bit e for key e, and the members' range.
    uint32_t members = 0xFFu;
    int k_min = 2147483647, k_max = -2147483647 - 1;
    {
      int k[8], kg[8] = {};
      load_keys8<true>(p.k_pos + b * p.k_sb, c, p.Nk, p.pos_vec != 0, k);
      if (groups) load_keys8<true>(p.k_group + b * p.kg_sb, c, p.Nk, p.pos_vec != 0, kg);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        keys[i * threads] = make_int4(k[4 * i], k[4 * i + 1], k[4 * i + 2], k[4 * i + 3]);
        keys[(2 + i) * threads] = make_int4(kg[4 * i], kg[4 * i + 1], kg[4 * i + 2], kg[4 * i + 3]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        k_min = min(k_min, k[e]);
        k_max = max(k_max, k[e]);
      }
    }
    // queries below q_hi have all members past the border ahead, those above
    // q_lo behind (a bound that saturates is never passed, so this holds at the
    // ends of the range, where a few more values go one by one)
    int q_hi = sub_sat(k_min, far_hi - 1), q_lo = add_sat(k_max, far - 1);
    int group = 0;
    bool first = true;
    float2 lo = make_float2(0.f, 0.f), hi = lo, cross = lo;
    using W = typename T::Word;
    const W *src = static_cast<const W *>(p.out) + b * p.out_s[0] + h * p.out_s[1] + c;
    const int32_t *qp = p.q_pos + b * p.q_sb, *qgp = groups ? p.q_group + b * p.qg_sb : nullptr;
    const bool inner = c >= 8 && c + 16 <= p.Nk;
    const int step = lanes * p.row_splits, begin = row_split * lanes + lane_row;
    const int64_t row_step = int64_t(step) * p.out_s[2];
    const W *row = src + int64_t(begin) * p.out_s[2];   // this row's eight
    int ahead = begin;                                  // the row to be fetched next, and its eight
    const W *ahead_row = row;
    uint8_t *slot = ring;
    const int slot_bytes = R::kSlotWords * threads * 16;
    auto sum8 = [](const float2 (&v)[4]) { return fadd2(fadd2(v[0], v[1]), fadd2(v[2], v[3])); };
    auto fetch = [&](uint8_t *to) {
      if (ahead < p.Nq) R::fetch(to, threads * 16, ahead_row, n, inner);
      cp_async_commit();
      ahead += step;
      ahead_row += row_step;
    };
    for (int s = 0; s < Ring::kStages; ++s) fetch(ring + s * slot_bytes);
    int q = begin < p.Nq ? __ldg(qp + begin) : 0, qg = groups && begin < p.Nq ? __ldg(qgp + begin) : 0;
#pragma unroll 2
    for (int i = begin; i < p.Nq; i += step) {
      const int2 qq = make_int2(q, qg);
      const int next = min(i + step, p.Nq - 1);
      q = __ldg(qp + next);
      if (groups) qg = __ldg(qgp + next);
      cp_async_wait<Ring::kStages - 1>();
      const Raw8<T> x = R::take(slot, threads * 16, row, inner);
      if (groups && (first || qq.y != group)) {
        first = false;
        group = qq.y;
        k_min = 2147483647, k_max = -2147483647 - 1;
        members = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int4 kp = keys[i * threads], kg = keys[(2 + i) * threads];
          const int pos[4] = {kp.x, kp.y, kp.z, kp.w}, grp[4] = {kg.x, kg.y, kg.z, kg.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (grp[e] == group) {
              members |= 1u << (4 * i + e);
              k_min = min(k_min, pos[e]);
              k_max = max(k_max, pos[e]);
            }
          }
        }
        q_hi = sub_sat(k_min, far_hi - 1);
        q_lo = add_sat(k_max, far - 1);
      }
      float2 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = x.pair(e);
      if (members != 0xFFu && members != 0) {
        // selected, not multiplied by 0 or 1: an infinity or a NaN stays in its row
        float2 others[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool mx = (members >> (2 * e)) & 1u, my = (members >> (2 * e + 1)) & 1u;
          others[e] = make_float2(mx ? 0.f : v[e].x, my ? 0.f : v[e].y);
          v[e] = make_float2(mx ? v[e].x : 0.f, my ? v[e].y : 0.f);
        }
        cross = fadd2(cross, sum8(others));
      }
      if (members == 0) {
        cross = fadd2(cross, sum8(v));
      } else if (qq.x < q_hi) {
        hi = fadd2(hi, sum8(v));
      } else if (qq.x > q_lo) {
        lo = fadd2(lo, sum8(v));
      } else {
        const int k_lo = sub_sat(qq.x, far), k_hi = add_sat(qq.x, far);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int4 kp = keys[i * threads];
          const int pos[4] = {kp.x, kp.y, kp.z, kp.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // (0 of a key that is no member)
            const float2 pair = v[2 * i + (e >> 1)];
            const int r = relpos_row(rule, look, min(max(pos[e], k_lo), k_hi) - qq.x);
            hist[r * threads + tid] += e & 1 ? pair.y : pair.x;
          }
        }
      }
      fetch(slot);
      row += row_step;
      slot = slot + slot_bytes == ring + Ring::kStages * slot_bytes ? ring : slot + slot_bytes;
    }
    cp_async_wait<0>();
    auto add = [&](int r, float2 s) { hist[r * threads + tid] += s.x + s.y; };
    add(rule.kind == 0 ? 0 : rule.side - 1, lo);
    add(rule.kind == 0 ? 2 * rule.far : (rule.kind == 1 ? 2 * rule.side - 1 : 0), hi);
    if (groups) add(rule.cross, cross);
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
