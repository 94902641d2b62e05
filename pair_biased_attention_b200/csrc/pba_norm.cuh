// pba_norm.cuh -- the norms before and after a block, fused with its gate and
// residual scale, and their gradients.
//
//     u = post(f)                       (no norm after the block: u = f)
//     h = x + scale * sigmoid(gate) * u (no block: h = x)
//     y = pre(h)                        the next block's input
//
// post and pre bring a row to mean 0 (layer norm only) and mean square 1 and
// apply a weight and a bias per channel.  Triangle attention and pair-biased
// attention sit between two such steps: f is what the block's output
// projection returns, y what the next block's projections read.
//
// A row of C channels is held by blockDim.x threads of eight channels each,
// all of it in registers: one pass over the data, the mean first and then the
// squares around it.  Up to 256 channels (32 threads) several rows share a
// block and sums go by shuffles; beyond, a block takes one row at a time and
// sums go through shared memory.  Bound by the bytes read and written.
#pragma once

#include "pba_vec8.cuh"

namespace pba {

constexpr int kNormMaxC = 8192;
constexpr int kNormNarrowC = 256;  // widest row that shares its block with others
constexpr int kNormNarrowThreads = 256;
constexpr int kNormParams = 5;  // dscale, dpost_w, dpost_b, dpre_w, dpre_b

struct NormParams {
  int64_t rows;
  int32_t C;
  int32_t layer;     // 1 layer norm, 0 root mean square
  int32_t param_f32; // weights, biases and scale in fp32 (else bf16)
  float eps, inv_c;
  const void *x, *f, *gate;  // forward inputs (backward: f, gate)
  const void *scale, *post_w, *post_b, *pre_w, *pre_b;
  void *h, *y;               // forward outputs; backward: h is read
  const void *dh, *dy;       // backward inputs
  void *dx, *df, *dgate;     // backward outputs
  int64_t x_s, f_s, gate_s, h_s, y_s, dh_s, dy_s, dx_s, df_s, dgate_s;  // row strides
  float *part;               // backward: [blocks][kNormParams][C]
};

// A thread's channels of a per-channel parameter as fp32 (0 past the end), in
// the order of load8.  Parameters stay in L1: they are read for every row.
template <bool kVec>
__device__ __forceinline__ void param8(const void *p, bool f32, int c, int n, int step, float (&x)[8]) {
  if (f32) {
    const float *q = static_cast<const float *>(p) + c;
    if (kVec && n >= 8) {
      const float4 a = __ldg(reinterpret_cast<const float4 *>(q)), b = __ldg(reinterpret_cast<const float4 *>(q) + 1);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = e < n ? __ldg(q + (kVec ? e : e * step)) : 0.f;
    }
  } else {
    const uint16_t *q = static_cast<const uint16_t *>(p) + c;
    if (kVec && n >= 8) {
      unpack8(__ldg(reinterpret_cast<const uint4 *>(q)), x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = e < n ? Bf16::to_f32(__ldg(q + (kVec ? e : e * step))) : 0.f;
    }
  }
}

// A thread's first channel, and how many of its eight exist (none for a thread
// past the end, which still takes part in the sums): eight consecutive ones,
// or every blockDim.x-th.
template <bool kVec>
__device__ __forceinline__ int norm_first() {
  return kVec ? threadIdx.x * 8 : threadIdx.x;
}
template <bool kVec>
__device__ __forceinline__ int norm_count(int C) {
  const int left = C - norm_first<kVec>();
  return max(0, kVec ? min(8, left) : (left + int(blockDim.x) - 1) / int(blockDim.x));
}

// Sums of N values over the threads of a row.  kWide: the row is the block
// (a multiple of 32 threads), `buf` holds 2 x N x 32 floats used in turn;
// otherwise the row is `lanes` neighbouring lanes, a power of two.
template <bool kWide, int N>
struct RowSum {
  float *buf;
  int lanes;
  int turn;
  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (!kWide && o >= lanes) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
    if (kWide) {
      // the two halves of `buf` alternate, so a thread still reading one
      // round's sums is not overtaken by the next round's writes
      float *b = buf + turn * N * 32;
      turn ^= 1;
      const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) b[i * 32 + warp] = v[i];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = lane < warps ? b[i * 32 + lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
      }
    }
  }
};

// Subtracts the mean (layer norm) and returns the reciprocal root of the mean
// square of what is left; channels past the end stay 0.
template <bool kWide, int N>
__device__ __forceinline__ float centre(float (&x)[8], int n, const NormParams &p, RowSum<kWide, N> &sum) {
  float v[N] = {};
  if (p.layer) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[0] += x[e];
    sum(v);
    const float mean = v[0] * p.inv_c;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = e < n ? x[e] - mean : 0.f;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[0] = fmaf(x[e], x[e], v[0]);
  sum(v);
  return rsqrtf(fmaf(v[0], p.inv_c, p.eps));
}

__device__ __forceinline__ float sigmoid_f32(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

template <typename T, bool kVec, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 4 : 1) block_norm_fwd_kernel(const __grid_constant__ NormParams p) {
  using W = typename T::Word;
  constexpr bool kWide = kThreads > kNormNarrowThreads;
  __shared__ float buf[kWide ? 2 * 32 : 1];
  const int lanes = blockDim.x;                        // threads of a row
  const int c = norm_first<kVec>(), n = norm_count<kVec>(p.C);
  RowSum<kWide, 1> sum{buf, lanes, 0};
  const int64_t step = int64_t(gridDim.x) * blockDim.y;
  // every thread of a warp runs the same number of rounds: a row past the
  // end is carried along without loads and stores
  for (int64_t r0 = int64_t(blockIdx.x) * blockDim.y; r0 < p.rows; r0 += step) {
    const int64_t r = r0 + threadIdx.y;
    const int m = r < p.rows ? n : 0;
    float h[8], u[8], g[8];
    load8<T, kVec>(static_cast<const W *>(p.x) + r * p.x_s + c, m, lanes, h);
    if (p.f != nullptr) {
      load8<T, kVec>(static_cast<const W *>(p.f) + r * p.f_s + c, m, lanes, u);
      if (p.gate != nullptr) load8<T, kVec>(static_cast<const W *>(p.gate) + r * p.gate_s + c, m, lanes, g);
      if (p.post_w != nullptr) {
        const float rs = centre(u, m, p, sum);
        float w[8];
        param8<kVec>(p.post_w, p.param_f32, c, m, lanes, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] *= rs * w[e];
        if (p.post_b != nullptr) {
          param8<kVec>(p.post_b, p.param_f32, c, m, lanes, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] += w[e];
        }
      }
      if (p.gate != nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] *= sigmoid_f32(g[e]);
      }
      if (p.scale != nullptr) {
        param8<kVec>(p.scale, p.param_f32, c, m, lanes, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] += u[e];
      store8<T, kVec>(static_cast<W *>(p.h) + r * p.h_s + c, m, lanes, h);
    }
    if (p.pre_w != nullptr) {
      const float rs = centre(h, m, p, sum);
      float w[8];
      param8<kVec>(p.pre_w, p.param_f32, c, m, lanes, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] *= rs * w[e];
      if (p.pre_b != nullptr) {
        param8<kVec>(p.pre_b, p.param_f32, c, m, lanes, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] += w[e];
      }
      store8<T, kVec>(static_cast<W *>(p.y) + r * p.y_s + c, m, lanes, h);
    }
  }
}

// Gradients.  With t = dL/dh including what comes through pre,
//     dx = t, du = scale sigmoid(gate) t, dgate = scale u sigmoid' t,
//     dscale = sum over rows of sigmoid(gate) u t, and through each norm
//     dv = (w dv' - mean(w dv') - v mean(w dv' v)) / rms   (mean only for layer norm)
// The statistics are taken again from h and f, which the formulas need
// anyway.  Sums over rows stay in each thread's registers for its channels,
// then per block in shared memory, then in `part`, always in the same order.
template <typename T, bool kVec, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 2 : 1) block_norm_bwd_kernel(const __grid_constant__ NormParams p) {
  using W = typename T::Word;
  constexpr bool kWide = kThreads > kNormNarrowThreads;
  __shared__ float buf[kWide ? 2 * 2 * 32 : kNormNarrowThreads * 8];
  const int lanes = blockDim.x;
  const int c = norm_first<kVec>(), n = norm_count<kVec>(p.C);
  RowSum<kWide, 2> sum{buf, lanes, 0};
  const int64_t step = int64_t(gridDim.x) * blockDim.y;
  float acc[kNormParams][8] = {};
  for (int64_t r0 = int64_t(blockIdx.x) * blockDim.y; r0 < p.rows; r0 += step) {
    const int64_t r = r0 + threadIdx.y;
    const int m = r < p.rows ? n : 0;
    float t[8], h[8], dy[8], f[8], g[8], w[8];
    if (p.dh != nullptr) {
      load8<T, kVec>(static_cast<const W *>(p.dh) + r * p.dh_s + c, m, lanes, t);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = 0.f;
    }
    if (p.pre_w != nullptr) {
      load8<T, kVec>(static_cast<const W *>(p.h) + r * p.h_s + c, m, lanes, h);
      load8<T, kVec>(static_cast<const W *>(p.dy) + r * p.dy_s + c, m, lanes, dy);
    }
    if (p.f != nullptr) {
      load8<T, kVec>(static_cast<const W *>(p.f) + r * p.f_s + c, m, lanes, f);
      if (p.gate != nullptr) load8<T, kVec>(static_cast<const W *>(p.gate) + r * p.gate_s + c, m, lanes, g);
    }
    if (p.pre_w != nullptr) {
      const float rs = centre(h, m, p, sum);
      param8<kVec>(p.pre_w, p.param_f32, c, m, lanes, w);
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[e] *= rs;
        acc[3][e] = fmaf(dy[e], h[e], acc[3][e]);
        acc[4][e] += dy[e];
        dy[e] *= w[e];
        v[0] += dy[e];
        v[1] = fmaf(dy[e], h[e], v[1]);
      }
      sum(v);
      const float a = p.layer ? v[0] * p.inv_c : 0.f, b = v[1] * p.inv_c;
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = fmaf(rs, dy[e] - a - h[e] * b, t[e]);
    }
    store8<T, kVec>(static_cast<W *>(p.dx) + r * p.dx_s + c, m, lanes, t);
    if (p.f != nullptr) {
      float rs = 1.f;
      float u[8];
      if (p.post_w != nullptr) {
        rs = centre(f, m, p, sum);
        param8<kVec>(p.post_w, p.param_f32, c, m, lanes, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[e] *= rs;
          u[e] = f[e] * w[e];
        }
        if (p.post_b != nullptr) {
          float pb[8];
          param8<kVec>(p.post_b, p.param_f32, c, m, lanes, pb);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] += pb[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = f[e];
      }
      float sc[8];
      if (p.scale != nullptr) {
        param8<kVec>(p.scale, p.param_f32, c, m, lanes, sc);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) sc[e] = 1.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float s = p.gate != nullptr ? sigmoid_f32(g[e]) : 1.f;
        if (m <= 0) t[e] = 0.f;  // t holds no row here
        acc[0][e] = fmaf(t[e] * s, u[e], acc[0][e]);
        t[e] *= sc[e];
        g[e] = t[e] * u[e] * s * (1.f - s);
        t[e] *= s;
      }
      if (p.gate != nullptr) store8<T, kVec>(static_cast<W *>(p.dgate) + r * p.dgate_s + c, m, lanes, g);
      if (p.post_w != nullptr) {
        float v[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          acc[1][e] = fmaf(t[e], f[e], acc[1][e]);
          acc[2][e] += t[e];
          t[e] *= w[e];
          v[0] += t[e];
          v[1] = fmaf(t[e], f[e], v[1]);
        }
        sum(v);
        const float a = p.layer ? v[0] * p.inv_c : 0.f, b = v[1] * p.inv_c;
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = rs * (t[e] - a - f[e] * b);
      }
      store8<T, kVec>(static_cast<W *>(p.df) + r * p.df_s + c, m, lanes, t);
    }
  }
  // the block's sums: its rows' threads of a channel added in order
#pragma unroll
  for (int k = 0; k < kNormParams; ++k) {
    float *dst = p.part + (int64_t(blockIdx.x) * kNormParams + k) * p.C + c;
    if (!kWide) {
      __syncthreads();
      float *mine = buf + (threadIdx.y * blockDim.x + threadIdx.x) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) mine[e] = acc[k][e];
      __syncthreads();
      if (threadIdx.y == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[k][e] = 0.f;
        for (int y = 0; y < int(blockDim.y); ++y) {
          const float *o = buf + (y * blockDim.x + threadIdx.x) * 8;
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[k][e] += o[e];
        }
      }
    }
    if (kWide || threadIdx.y == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) dst[kVec ? e : e * lanes] = acc[k][e];
    }
  }
}

struct NormSumParams {
  const float *part;
  int32_t blocks, C;
  float *out[kNormParams];  // null: not wanted
};

// Gradients of the per-channel parameters: the blocks' sums added in 64 bits.
__global__ void block_norm_sum_kernel(const __grid_constant__ NormSumParams p) {
  __shared__ double acc[8][33];
  const int k = blockIdx.y, c = blockIdx.x * 32 + threadIdx.x;
  if (p.out[k] == nullptr) return;
  double s = 0.0;
  if (c < p.C)
    for (int i = threadIdx.y; i < p.blocks; i += 8)
      s += double(p.part[(int64_t(i) * kNormParams + k) * p.C + c]);
  acc[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < p.C) {
#pragma unroll
    for (int y = 1; y < 8; ++y) s += acc[y][threadIdx.x];
    p.out[k][c] = float(s);
  }
}

}  // namespace pba
