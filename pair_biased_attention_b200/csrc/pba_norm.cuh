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
// A row of C channels is held by blockDim.x threads, all of it in registers: one
// pass over the data, the mean first and then the squares around it, while the
// thread's next rows are on their way.  Rows of up to 32 threads share a block and
// their sums go by shuffles; beyond, a block takes one row at a time and sums
// go through shared memory.  Bound by the bytes read and written, and close
// behind by the instructions per element: channels are worked on in packed
// pairs, and a thread takes 32 bytes of every tensor where its registers allow.
// Measured: 1024^2 rows of 128 channels, bf16, with both layer norms, gate and
// scale (5 tensors, 1.34 GB) 230 us, 5.8 TB/s, 0.89 of a copy's rate.  With the
// parameters unpacked from L1 for every row and the rows' addresses multiplied
// out it was 283 us, bound by instructions; three blocks of 256 threads an SM
// were no faster, scalar arithmetic took 314 us.  The gradients at 512^2 rows
// (8 tensors, 0.54 GB) 105 us, 5.1 TB/s.  fp32 rows: 5.6 to 5.8 TB/s either way.
// Rows of a block, where a row's sums meet at barriers and a block has one row
// under way, are slower: 32768 rows of 768, bf16, residual and RMS norm 5.2 and
// 4.5 TB/s forward and backward, with all parts 2.4 and 3.3 (fp32 4.5 and 5.6).
// Over 4096 channels, fp32 forward and both types backward, a block has 1024
// threads of 64 registers, into which the parts do not fit: 660 to 992 bytes a
// thread spill in the backward, 100 in the forward.  4096 rows of 8192, bf16, 5.9
// and 1.4 TB/s, with all parts 2.1 and 1.1 (fp32 5.3 and 2.6, 3.2 and 2.0).
#pragma once

#include <cfloat>

#include "pba_vec8.cuh"

namespace pba {

constexpr int kNormMaxC = 8192;
constexpr int kNormNarrowThreads = 256;
constexpr int kNormParams = 5;  // dscale, dpost_w, dpost_b, dpre_w, dpre_b
constexpr int kNormMaxThreadRows = 512;  // backward: rows that a thread adds up in fp32

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

// Channels that a thread takes of each row: 32 bytes forward, eight backward,
// where the sums over rows need registers too.
template <typename T>
__host__ __device__ constexpr int norm_fwd_channels() {
  return 32 / int(sizeof(typename T::Word));
}
constexpr int kNormBwdChannels = 8;

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// E channels of a thread as packed pairs.
template <int E>
struct Channels {
  float2 v[E / 2];
  __device__ __forceinline__ float &at(int e) { return e & 1 ? v[e >> 1].y : v[e >> 1].x; }
  __device__ __forceinline__ float total() const {
    float2 s[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int i = 4; i < E / 2; ++i) s[i & 3] = fadd2(s[i & 3], v[i]);
    const float2 t = fadd2(fadd2(s[0], s[1]), fadd2(s[2], s[3]));
    return t.x + t.y;
  }
};
template <int E>
__device__ __forceinline__ float dot(const Channels<E> &x, const Channels<E> &y) {
  float2 s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = fmul2(x.v[i], y.v[i]);
#pragma unroll
  for (int i = 4; i < E / 2; ++i) s[i & 3] = ffma2(x.v[i], y.v[i], s[i & 3]);
  const float2 t = fadd2(fadd2(s[0], s[1]), fadd2(s[2], s[3]));
  return t.x + t.y;
}

// Where a thread's channels lie.  kVec (16-byte aligned rows): words of 16
// bytes, G channels, number threadIdx.x, + blockDim.x, ..., each there or not as
// a whole.  Otherwise every blockDim.x-th channel from threadIdx.x on.  Either
// way neighbouring threads touch neighbouring places (32 bytes a thread in one
// piece, half a sector to an access, held fp32 rows at 3.9 TB/s).
template <bool kVec, int E, int G>
struct Place {
  int lanes, t, C;
  __device__ __forceinline__ explicit Place(int channels) : lanes(blockDim.x), t(threadIdx.x), C(channels) {}
  __device__ __forceinline__ int channel(int e) const { return kVec ? G * (t + e / G * lanes) + e % G : t + e * lanes; }
  __device__ __forceinline__ bool has(int e) const { return channel(kVec ? e / G * G : e) < C; }
};
template <typename T>
__host__ __device__ constexpr int norm_word() {
  return 16 / int(sizeof(typename T::Word));
}

// A thread's channels of `kArrays` tensors, row after row.  Aligned rows run
// through a ring in shared memory, kStages rows deep, that the thread fills with
// asynchronous copies and reads alone: with all parts 196 KB on their way per SM
// forward and 164 KB backward (bf16, rows of up to 32 threads), a third and a
// fifth of it for each tensor (one row ahead in registers, 48 KB, reached 0.69 of
// HBM's rate).  Other rows are read element by element when they are needed.
// Every tensor has a pointer that walks down its rows.
template <typename T, bool kVec, int E, int kArrays, int kStages, int kThreads>
struct RowStream {
  using W = typename T::Word;
  static constexpr int G = norm_word<T>();
  static constexpr int kWords = E / G;  // 16-byte words of a row
  static constexpr int kThreadBytes = kVec ? kArrays * kStages * kWords * 16 : 0;
  const Place<kVec, E, G> &at;
  int word_bytes;  // from a word of the ring to the thread's next
  uint8_t *ring, *stage;
  const uint8_t *src[kArrays];  // kVec: the row to be fetched next, else the one to be read next
  int64_t by[kArrays];

  __device__ __forceinline__ RowStream(uint8_t *smem, const Place<kVec, E, G> &place) : at(place) {
    word_bytes = 16 * (kThreads == kNormNarrowThreads ? kNormNarrowThreads : int(blockDim.x));
    ring = stage = smem + (threadIdx.y * blockDim.x + threadIdx.x) * 16;
  }
  // rows first, first + step, ... of a tensor
  __device__ __forceinline__ void open(int array, const void *base, int64_t stride, int64_t first, int64_t step) {
    src[array] = static_cast<const uint8_t *>(base) + (first * stride + at.channel(0)) * int64_t(sizeof(W));
    by[array] = step * stride * int64_t(sizeof(W));
  }
  __device__ __forceinline__ uint8_t *word(int array, int i) const { return stage + (array * kWords + i) * word_bytes; }
  // starts copying the tensor's next row into the stage in turn; zeros for a
  // row past the end and for channels past the last
  __device__ __forceinline__ void fetch(int array, bool row) {
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if (row && at.has(G * i))
          cp_async16(word(array, i), src[array] + i * at.lanes * 16);
        else
          *reinterpret_cast<uint4 *>(word(array, i)) = make_uint4(0, 0, 0, 0);
      }
      src[array] += by[array];
    }
  }
  __device__ __forceinline__ void turn() {  // the stage's last fetch has been started
    if constexpr (kVec) {
      cp_async_commit();
      constexpr int kStageWords = kArrays * kWords;
      stage = stage == ring + (kStages - 1) * kStageWords * word_bytes ? ring : stage + kStageWords * word_bytes;
    }
  }
  __device__ __forceinline__ void wait() const {
    if (kVec) cp_async_wait<kStages - 1>();
  }
  __device__ __forceinline__ Channels<E> get(int array, bool row) {
    Channels<E> r;
    if (kVec) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint4 v = *reinterpret_cast<const uint4 *>(word(array, i));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if (sizeof(W) == 2) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            r.v[(4 * i + k) % (E / 2)] = make_float2(bf16lo_to_f32(w[k]), bf16hi_to_f32(w[k]));
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            r.v[(2 * i + k) % (E / 2)] = make_float2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
        }
      }
    } else {
      const W *p = reinterpret_cast<const W *>(src[array]);
#pragma unroll
      for (int e = 0; e < E; ++e) r.at(e) = row && at.has(e) ? T::to_f32(p[e * at.lanes]) : 0.f;
      src[array] += by[array];
    }
    return r;
  }
};

// The rows of an output that a thread writes, one after the other.
template <typename T, bool kVec, int E>
struct RowOut {
  using W = typename T::Word;
  static constexpr int G = norm_word<T>();
  W *dst;
  int64_t by;
  __device__ __forceinline__ RowOut(void *base, int64_t stride, int64_t first, int64_t step)
      : dst(static_cast<W *>(base) + first * stride), by(step * stride) {}
  __device__ __forceinline__ void put(bool row, const Place<kVec, E, G> &at, Channels<E> &c) {
    if (row) {
      if (kVec) {
#pragma unroll
        for (int i = 0; i < E / G; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 v = c.v[(G == 8 ? 4 * i + k : 2 * i + k / 2) % (E / 2)];
            w[k] = G == 8 ? pack_bf16x2(v.x, v.y) : __float_as_uint(k & 1 ? v.y : v.x);
          }
          if (at.has(G * i)) st_stream16(dst + at.channel(G * i), make_uint4(w[0], w[1], w[2], w[3]));
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (at.has(e)) dst[at.channel(e)] = T::from_f32(c.at(e));
      }
    }
    dst += by;
  }
};

// A thread's channels of a per-channel parameter as fp32 (0 past the end).
template <bool kVec, int E, int G>
__device__ __forceinline__ Channels<E> param(const void *p, bool f32, const Place<kVec, E, G> &at) {
  Channels<E> r;
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {  // four channels at a time
    float x[4] = {};
    if (kVec) {
      if (at.has(4 * i)) {
        if (f32) {
          const float4 a = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at.channel(4 * i)));
          x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        } else {
          const uint2 a = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + at.channel(4 * i)));
          x[0] = bf16lo_to_f32(a.x), x[1] = bf16hi_to_f32(a.x), x[2] = bf16lo_to_f32(a.y), x[3] = bf16hi_to_f32(a.y);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at.has(4 * i + e))
          x[e] = f32 ? __ldg(static_cast<const float *>(p) + at.channel(4 * i + e))
                     : Bf16::to_f32(__ldg(static_cast<const uint16_t *>(p) + at.channel(4 * i + e)));
    }
    r.v[2 * i] = make_float2(x[0], x[1]);
    r.v[2 * i + 1] = make_float2(x[2], x[3]);
  }
  return r;
}

// The parameters as the kernels multiply with them, for every row anew: N
// tensors of C channels.  Narrow rows find them in shared memory as fp32
// (unpacking bf16 from L1 took a tenth of the instructions); for wide ones,
// whose ring fills it, they come from L1.
template <bool kWide, bool kVec, int E, int G, int N>
struct Params {
  static constexpr int kChannels = 32 * E;  // of the widest narrow row
  static constexpr int kFloats = kWide ? 1 : N * kChannels;
  float *buf;
  const NormParams &p;
  const Place<kVec, E, G> &at;
  // eights: their halves in two planes, so that neighbouring threads read
  // neighbouring words
  __device__ __forceinline__ float *slot(int k, int c) const {
    return buf + k * kChannels + (kVec && G == 8 ? ((c >> 2) & 1) * (kChannels / 2) + (c >> 3) * 4 + (c & 3) : c);
  }
  // load(c): the parameter's channel c.  The caller synchronises.
  template <typename F>
  __device__ __forceinline__ void stage(int k, bool there, F load) {
    if constexpr (!kWide) {
      if (!there) return;
      for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < kChannels; c += kNormNarrowThreads)
        *slot(k, c) = c < p.C ? load(c) : 0.f;
    }
  }
  __device__ __forceinline__ float one(const void *t, int c) const {
    return p.param_f32 ? static_cast<const float *>(t)[c] : Bf16::to_f32(static_cast<const uint16_t *>(t)[c]);
  }
  // number k; wide: `t`, times `scale` where that is given
  __device__ __forceinline__ Channels<E> get(int k, const void *t, const void *scale = nullptr) const {
    Channels<E> r;
    if constexpr (kWide) {
      r = param(t, p.param_f32, at);
      if (scale != nullptr) {
        const Channels<E> s = param(scale, p.param_f32, at);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) r.v[i] = fmul2(r.v[i], s.v[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        if (kVec) {
          const float4 x = *reinterpret_cast<const float4 *>(slot(k, at.channel(4 * i)));
          r.v[2 * i] = make_float2(x.x, x.y);
          r.v[2 * i + 1] = make_float2(x.z, x.w);
        } else {
#pragma unroll
          for (int e = 4 * i; e < 4 * i + 4; ++e) r.at(e) = *slot(k, at.channel(e));
        }
      }
    }
    return r;
  }
};

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
    for (int o = 1; o < 32; o <<= 1) {
      if (!kWide && o >= lanes) break;
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

// x - mean; channels past the end stay 0.
template <bool kVec, int E, int G>
__device__ __forceinline__ void take_mean(Channels<E> &x, float mean, const Place<kVec, E, G> &at) {
  if (kVec) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x.v[i] = fadd2(x.v[i], both(at.has(2 * i) ? -mean : 0.f));
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) x.at(e) = at.has(e) ? x.at(e) - mean : 0.f;
  }
}

// Subtracts the mean (layer norm) and returns the reciprocal root of the mean
// square of what is left.
template <bool kWide, bool kVec, int E, int G>
__device__ __forceinline__ float centre(Channels<E> &x, const NormParams &p, const Place<kVec, E, G> &at,
                                        RowSum<kWide, 1> &sum) {
  float v[1];
  if (p.layer) {
    v[0] = x.total();
    sum(v);
    take_mean(x, v[0] * p.inv_c, at);
  }
  v[0] = dot(x, x);
  sum(v);
  return rsqrtf(fmaf(v[0], p.inv_c, p.eps));
}
// The same for two rows at once.
template <bool kWide, bool kVec, int E, int G>
__device__ __forceinline__ float2 centre2(Channels<E> &x, Channels<E> &y, const NormParams &p,
                                          const Place<kVec, E, G> &at, RowSum<kWide, 2> &sum) {
  float v[2];
  if (p.layer) {
    v[0] = x.total(), v[1] = y.total();
    sum(v);
    take_mean(x, v[0] * p.inv_c, at);
    take_mean(y, v[1] * p.inv_c, at);
  }
  v[0] = dot(x, x), v[1] = dot(y, y);
  sum(v);
  return make_float2(rsqrtf(fmaf(v[0], p.inv_c, p.eps)), rsqrtf(fmaf(v[1], p.inv_c, p.eps)));
}

// 1 / (1 + 2^(-x log2 e)) on the exp2 and reciprocal units, each good to about
// 2^-22: below the rounding of an fp32 product chain, and exact in the limits
// (the exponential overflows to infinity, whose reciprocal is 0).
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  const float2 a = fmul2(x, both(-1.4426950408889634f));
  const float2 d = fadd2(make_float2(ex2_approx(a.x), ex2_approx(a.y)), both(1.f));
  return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}
// The same and its complement 1 - sigmoid, as the exponential times the sigmoid: a
// difference would lose it next to 1 (at x = 8 a thousandth of it, from 17 on
// all).  Where the sigmoid is 0 the complement comes out as 0 too, not as 1: it is
// only used times the sigmoid.
__device__ __forceinline__ float2 sigmoid2(float2 x, float2 &complement) {
  const float2 a = fmul2(x, both(-1.4426950408889634f));
  const float2 e = make_float2(ex2_approx(a.x), ex2_approx(a.y)), d = fadd2(e, both(1.f));
  const float2 s = make_float2(rcp_approx(d.x), rcp_approx(d.y));
  complement = fmul2(s, make_float2(fminf(e.x, FLT_MAX), fminf(e.y, FLT_MAX)));
  return s;
}

template <int kThreads>
__host__ __device__ constexpr int norm_fwd_stages() {
  return kThreads == 1024 ? 2 : 4;
}
template <typename T, bool kVec, int kThreads>
using NormFwdStream = RowStream<T, kVec, norm_fwd_channels<T>(), 3, norm_fwd_stages<kThreads>(), kThreads>;

template <typename T, bool kVec, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 2 : 1)
    block_norm_fwd_kernel(const __grid_constant__ NormParams p) {
  constexpr bool kWide = kThreads > kNormNarrowThreads;
  constexpr int E = norm_fwd_channels<T>();
  using Par = Params<kWide, kVec, E, norm_word<T>(), 4>;
  __shared__ float buf[kWide ? 2 * 32 : 1];
  __shared__ __align__(16) float param_buf[Par::kFloats];
  extern __shared__ __align__(16) uint8_t norm_smem[];
  constexpr int G = norm_word<T>();
  const Place<kVec, E, G> at(p.C);
  RowSum<kWide, 1> sum{buf, int(blockDim.x), 0};
  const int64_t step = int64_t(gridDim.x) * blockDim.y;
  NormFwdStream<T, kVec, kThreads> in(norm_smem, at);
  int64_t r = int64_t(blockIdx.x) * blockDim.y + threadIdx.y, ahead = r;
  const bool post = p.post_w != nullptr, pre = p.pre_w != nullptr, has_f = p.f != nullptr, has_gate = p.gate != nullptr;
  in.open(0, p.x, p.x_s, r, step);
  if (has_f) in.open(1, p.f, p.f_s, r, step);
  if (has_gate) in.open(2, p.gate, p.gate_s, r, step);
  RowOut<T, kVec, E> h_out(p.h, p.h_s, r, step), y_out(p.y, p.y_s, r, step);
  auto fetch = [&]() {
    const bool row = ahead < p.rows;
    in.fetch(0, row);
    if (has_f) in.fetch(1, row);
    if (has_gate) in.fetch(2, row);
    in.turn();
    ahead += step;
  };
  for (int i = 0; i < norm_fwd_stages<kThreads>(); ++i) fetch();
  // h = x + sigmoid(gate) (a v + b), v the normalised f: the scale is part of
  // the weight a and the bias b.  y = pre_w v + pre_b.
  const void *a_of = post ? p.post_w : p.scale, *a_scale = post ? p.scale : nullptr;
  Par par{param_buf, p, at};
  par.stage(0, a_of != nullptr,
            [&](int c) { return par.one(a_of, c) * (a_scale != nullptr ? par.one(a_scale, c) : 1.f); });
  par.stage(1, p.post_b != nullptr,
            [&](int c) { return par.one(p.post_b, c) * (p.scale != nullptr ? par.one(p.scale, c) : 1.f); });
  par.stage(2, pre, [&](int c) { return par.one(p.pre_w, c); });
  par.stage(3, p.pre_b != nullptr, [&](int c) { return par.one(p.pre_b, c); });
  if (!kWide) __syncthreads();
  // every thread of a warp runs the same number of rounds: a row past the
  // end is carried along as zeros
  for (int64_t r0 = int64_t(blockIdx.x) * blockDim.y; r0 < p.rows; r0 += step, r += step) {
    const bool row = r < p.rows;
    in.wait();
    Channels<E> h = in.get(0, row), u, g;
    if (has_f) u = in.get(1, row);
    if (has_gate) g = in.get(2, row);
    fetch();
    if (has_f) {
      const float rs = post ? centre<kWide>(u, p, at, sum) : 1.f;
      if (a_of != nullptr) {
        const Channels<E> a = par.get(0, a_of, a_scale);
        if (p.post_b != nullptr) {
          const Channels<E> b = par.get(1, p.post_b, p.scale);
#pragma unroll
          for (int i = 0; i < E / 2; ++i) u.v[i] = ffma2(u.v[i], fmul2(a.v[i], both(rs)), b.v[i]);
        } else {
#pragma unroll
          for (int i = 0; i < E / 2; ++i) u.v[i] = fmul2(u.v[i], fmul2(a.v[i], both(rs)));
        }
      }
      if (has_gate) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) h.v[i] = ffma2(u.v[i], sigmoid2(g.v[i]), h.v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) h.v[i] = fadd2(h.v[i], u.v[i]);
      }
      h_out.put(row, at, h);
    }
    if (pre) {
      const float rs = centre<kWide>(h, p, at, sum);
      const Channels<E> w = par.get(2, p.pre_w);
      if (p.pre_b != nullptr) {
        const Channels<E> b = par.get(3, p.pre_b);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) h.v[i] = ffma2(h.v[i], fmul2(w.v[i], both(rs)), b.v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) h.v[i] = fmul2(h.v[i], fmul2(w.v[i], both(rs)));
      }
      y_out.put(row, at, h);
    }
  }
}

// Gradients.  With t = dL/dh including what comes through pre,
//     dx = t, du = scale sigmoid(gate) t, dgate = scale u sigmoid' t,
//     dscale = sum over rows of sigmoid(gate) u t, and through each norm
//     dv = (w dv' - mean(w dv') - v mean(w dv' v)) / rms   (mean only for layer norm)
// The statistics are taken again from h and f, which the formulas need
// anyway.  Sums over rows stay in each thread's registers for its channels, at
// most kNormMaxThreadRows rows long in fp32; a block's rows are joined in 64 bits
// in shared memory, and its share, rounded to fp32 once, goes to `part`, always in
// the same order.
template <typename T, int kThreads>
__host__ __device__ constexpr int norm_bwd_stages() {
  return (kThreads == 1024 ? 4 : 8) / int(sizeof(typename T::Word));
}
template <typename T, bool kVec, int kThreads>
using NormBwdStream = RowStream<T, kVec, kNormBwdChannels, 5, norm_bwd_stages<T, kThreads>(), kThreads>;

// kParts: which parts there are (norm_parts), known when the kernel is built for
// the usual sets of them, with dh; or -1, asked at run time.  The formulas are
// long enough for that to count: 512^2 rows of 128 channels, bf16, when each set
// was measured both ways, all parts 141 us asked and 109 known, residual and layer
// norm 108 and 77.  Sets without dh, and a last block without pre, are asked.  The
// forward gained nothing by it.
__host__ __device__ constexpr int norm_parts(bool f, bool gate, bool post, bool pre) {
  return f + 2 * gate + 4 * post + 8 * pre;
}
template <typename T, bool kVec, int kThreads, int kParts>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 2 : 1)
    block_norm_bwd_kernel(const __grid_constant__ NormParams p) {
  constexpr bool kWide = kThreads > kNormNarrowThreads;
  constexpr int E = kNormBwdChannels;
  using Ch = Channels<E>;
  using Par = Params<kWide, kVec, E, norm_word<T>(), 4>;
  __shared__ __align__(16) float param_buf[Par::kFloats];
  __shared__ float buf[kWide ? 2 * 2 * 32 : kNormNarrowThreads * E];
  constexpr int G = norm_word<T>();
  const Place<kVec, E, G> at(p.C);
  RowSum<kWide, 2> sum{buf, int(blockDim.x), 0};
  const int64_t step = int64_t(gridDim.x) * blockDim.y;
  Ch acc[kNormParams] = {};
  constexpr bool kKnown = kParts >= 0;
  const bool has_f = kKnown ? kParts & 1 : p.f != nullptr, has_gate = kKnown ? kParts & 2 : p.gate != nullptr;
  const bool post = kKnown ? kParts & 4 : p.post_w != nullptr, pre = kKnown ? kParts & 8 : p.pre_w != nullptr;
  const bool has_dh = kKnown || p.dh != nullptr;
  const bool has_scale = p.scale != nullptr, has_post_b = p.post_b != nullptr, layer = p.layer;
  extern __shared__ __align__(16) uint8_t norm_smem[];
  NormBwdStream<T, kVec, kThreads> in(norm_smem, at);
  int64_t r = int64_t(blockIdx.x) * blockDim.y + threadIdx.y, ahead = r;
  if (has_dh) in.open(0, p.dh, p.dh_s, r, step);
  if (pre) {
    in.open(1, p.h, p.h_s, r, step);
    in.open(2, p.dy, p.dy_s, r, step);
  }
  if (has_f) in.open(3, p.f, p.f_s, r, step);
  if (has_gate) in.open(4, p.gate, p.gate_s, r, step);
  using Out = RowOut<T, kVec, E>;
  Out dx_out(p.dx, p.dx_s, r, step), df_out(p.df, p.df_s, r, step), dg_out(p.dgate, p.dgate_s, r, step);
  auto fetch = [&]() {
    const bool row = ahead < p.rows;
    if (has_dh) in.fetch(0, row);
    if (pre) {
      in.fetch(1, row);
      in.fetch(2, row);
    }
    if (has_f) in.fetch(3, row);
    if (has_gate) in.fetch(4, row);
    in.turn();
    ahead += step;
  };
  for (int i = 0; i < norm_bwd_stages<T, kThreads>(); ++i) fetch();
  Par par{param_buf, p, at};
  par.stage(0, has_scale, [&](int c) { return par.one(p.scale, c); });
  par.stage(1, post, [&](int c) { return par.one(p.post_w, c); });
  par.stage(2, has_post_b, [&](int c) { return par.one(p.post_b, c); });
  par.stage(3, pre, [&](int c) { return par.one(p.pre_w, c); });
  if (!kWide) __syncthreads();
  for (int64_t r0 = int64_t(blockIdx.x) * blockDim.y; r0 < p.rows; r0 += step, r += step) {
    const bool row = r < p.rows;
    in.wait();
    Ch t = {}, h = {}, dy = {}, f = {}, g = {};
    if (has_dh) t = in.get(0, row);
    if (pre) {
      h = in.get(1, row);
      dy = in.get(2, row);
    }
    if (has_f) f = in.get(3, row);
    if (has_gate) g = in.get(4, row);
    fetch();
    float2 rs = both(1.f);  // of h and of f
    Ch u = f;               // the block's output after its norm
    if (post) {
      rs = centre2<kWide>(h, f, p, at, sum);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) f.v[i] = fmul2(f.v[i], both(rs.y));
    } else if (pre) {
      Ch none = {};
      rs = centre2<kWide>(h, none, p, at, sum);
    }
    if (pre) {
      const Ch w = par.get(3, p.pre_w);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        h.v[i] = fmul2(h.v[i], both(rs.x));
        acc[3].v[i] = ffma2(dy.v[i], h.v[i], acc[3].v[i]);
        acc[4].v[i] = fadd2(dy.v[i], acc[4].v[i]);
        dy.v[i] = fmul2(dy.v[i], w.v[i]);
      }
      float v[2] = {dy.total(), dot(dy, h)};
      sum(v);
      const float a = layer ? -v[0] * p.inv_c : 0.f, b = -v[1] * p.inv_c;
#pragma unroll
      for (int i = 0; i < E / 2; ++i)
        t.v[i] = ffma2(both(rs.x), ffma2(h.v[i], both(b), fadd2(dy.v[i], both(a))), t.v[i]);
    }
    dx_out.put(row, at, t);
    if (has_f) {
      Ch w;
      if (post) {
        w = par.get(1, p.post_w);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) u.v[i] = fmul2(f.v[i], w.v[i]);
        if (has_post_b) {
          const Ch b = par.get(2, p.post_b);
#pragma unroll
          for (int i = 0; i < E / 2; ++i) u.v[i] = fadd2(u.v[i], b.v[i]);
        }
      }
      Ch s;  // sigmoid(gate); g becomes 1 - sigmoid(gate)
      // A row past the end is all zeros here: its t, dy and h are.  Channels
      // past the end of a row may hold the mean's share in t; u is 0 there,
      // and so is the weight that t is multiplied with below.
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        s.v[i] = has_gate ? sigmoid2(g.v[i], g.v[i]) : both(1.f);
        t.v[i] = fmul2(t.v[i], s.v[i]);
        acc[0].v[i] = ffma2(t.v[i], u.v[i], acc[0].v[i]);
      }
      if (has_scale) {
        const Ch sc = par.get(0, p.scale);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) t.v[i] = fmul2(t.v[i], sc.v[i]);
      }
      if (has_gate) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
          g.v[i] = fmul2(fmul2(t.v[i], u.v[i]), g.v[i]);
        dg_out.put(row, at, g);
      }
      if (post) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          acc[1].v[i] = ffma2(t.v[i], f.v[i], acc[1].v[i]);
          acc[2].v[i] = fadd2(t.v[i], acc[2].v[i]);
          t.v[i] = fmul2(t.v[i], w.v[i]);
        }
        float v[2] = {t.total(), dot(t, f)};
        sum(v);
        const float a = layer ? -v[0] * p.inv_c : 0.f, b = -v[1] * p.inv_c;
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
          t.v[i] = fmul2(both(rs.y), ffma2(f.v[i], both(b), fadd2(t.v[i], both(a))));
      }
      df_out.put(row, at, t);
    }
  }
  // The block's sums.  Rows that share it: all its threads join, each eight rows of
  // one channel in 64 bits, then the neighbouring lanes of the channel.
#pragma unroll
  for (int k = 0; k < kNormParams; ++k) {
    float *dst = p.part + (int64_t(blockIdx.x) * kNormParams + k) * p.C;
    if (kWide) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (at.has(e)) dst[at.channel(e)] = acc[k].at(e);
    } else {
      __syncthreads();
      const int tid = threadIdx.y * blockDim.x + threadIdx.x;
#pragma unroll
      for (int e = 0; e < E; ++e) buf[tid * E + e] = acc[k].at(e);
      __syncthreads();
      const int lanes = blockDim.x, per = 32 / lanes;  // blockDim.y = 8 per
      const int i = tid / per, first = tid & (per - 1);  // the row's channel number i, by place
      double s = 0.0;
#pragma unroll
      for (int y = 0; y < kNormNarrowThreads / 32; ++y) s += double(buf[(first + y * per) * lanes * E + i]);
      for (int o = per / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      Place<kVec, E, G> there(p.C);
      there.t = i / E;
      const int c = there.channel(i % E);
      if (first == 0 && c < p.C) dst[c] = float(s);
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
