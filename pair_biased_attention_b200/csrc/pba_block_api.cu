// pba_block_api.cu -- the operators around the attention block declared in
// include/pba.h: the relative position bias with its gradient and the block
// norms with theirs.  Argument checks, launch shapes and launches; the
// computation runs in the kernels of pba_relpos.cuh and pba_norm.cuh.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <utility>

#include "pba.h"
#include "pba_host.cuh"
#include "pba_norm.cuh"
#include "pba_relpos.cuh"

using namespace pba_host;

namespace {

// The SMs that launch shapes are planned for (B200).  A constant, so that
// workspaces have the same size wherever they are asked for.
constexpr int64_t kPlanSms = 148;
// Dynamic shared memory that the relative position kernels may ask for.
constexpr int kRelposSmem = 200 * 1024;
// And the block norms' ring of rows.
constexpr int kNormSmem = 200 * 1024;
// Blocks of the table's gradient on an SM.
constexpr int64_t kRelposGradResident = 4;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t pow2_ceil(int64_t x) {
  int64_t r = 1;
  while (r < x) r *= 2;
  return r;
}
bool aligned_to(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & uintptr_t(bytes - 1)) == 0; }
int dtype_size(int dtype) { return dtype == PBA_BF16 ? 2 : 4; }
bool known_dtype(int dtype) { return dtype == PBA_BF16 || dtype == PBA_F32; }

// ------------------------------------------------------------ relative position bias
// A whole number of up to kRelposMaxBorders factors below 2^30, for comparing
// products exactly.
struct Whole {
  uint32_t word[pba::kRelposMaxBorders];
  int n = 1;
  Whole() { word[0] = 1; }
  void times(uint32_t f) {
    uint64_t carry = 0;
    for (int i = 0; i < n; ++i) {
      carry += uint64_t(word[i]) * f;
      word[i] = uint32_t(carry);
      carry >>= 32;
    }
    if (carry != 0) word[n++] = uint32_t(carry);
  }
  bool at_least(const Whole &o) const {
    if (n != o.n) return n > o.n;
    for (int i = n - 1; i >= 0; --i)
      if (word[i] != o.word[i]) return word[i] > o.word[i];
    return true;
  }
};

// Where row e + t of a logarithmic side begins: the smallest whole d with
// d >= e (far / e)^(t / m), that is d^m >= e^(m-t) far^t.  The root is good to
// 3e-15 of itself (far / e is below 2^31, so the exponent's rounding counts 21
// times, the other three once); where it lies too near a whole number to say on
// which side, the whole numbers are compared.
int32_t log_border(int e, int m, int t, int far) {
  const double x = e * std::pow(double(far) / e, double(t) / m);
  const double near = std::round(x);
  if (std::fabs(x - near) > 1e-13 * x) return int32_t(std::ceil(x));
  Whole have, need;
  for (int i = 0; i < m; ++i) {
    have.times(uint32_t(near));
    need.times(uint32_t(i < t ? far : e));
  }
  return int32_t(near) + (have.at_least(need) ? 0 : 1);
}

pba_status check_relpos(const pba_relpos_desc *d, bool groups) {
  if (d == nullptr) return PBA_ERR_INVALID_ARG;
  // B * Nq and Nk: the kernels step beyond them by less than 2^20, in 32 bits
  if (d->B < 1 || d->H < 1 || d->B > 65535 || d->H > 65535 || d->Nq < 0 || d->Nk < 0 || d->Nq > (1 << 30) ||
      d->Nk > kMaxI32 - (1 << 20) || d->B * d->Nq > kMaxI32 - (1 << 20))
    return PBA_ERR_INVALID_ARG;
  if (!known_dtype(d->dtype)) return PBA_ERR_UNSUPPORTED;
  const int buckets = d->rows - (groups ? 1 : 0);
  if (d->rows > pba::kRelposMaxRows) return PBA_ERR_UNSUPPORTED;
  if (d->rule == PBA_RELPOS_CLIP) return buckets >= 1 && buckets % 2 == 1 ? PBA_OK : PBA_ERR_INVALID_ARG;
  if (d->rule != PBA_RELPOS_LOG && d->rule != PBA_RELPOS_LOG_CAUSAL) return PBA_ERR_INVALID_ARG;
  const bool both = d->rule == PBA_RELPOS_LOG;
  if (buckets < (both ? 4 : 2) || (both && buckets % 2 != 0)) return PBA_ERR_INVALID_ARG;
  const int side = both ? buckets / 2 : buckets;
  if (d->max_distance <= side / 2 || d->max_distance > (1 << 30)) return PBA_ERR_INVALID_ARG;
  if (side - side / 2 - 1 > pba::kRelposMaxBorders) return PBA_ERR_UNSUPPORTED;
  return PBA_OK;
}

void fill_relpos(pba::RelposParams &p, const pba_relpos_desc *d, const int32_t *q_pos, const int32_t *k_pos,
                 const int32_t *q_group, const int32_t *k_group) {
  std::memset(&p, 0, sizeof(p));
  const bool groups = q_group != nullptr;
  p.B = int(d->B), p.H = int(d->H), p.Nq = int(d->Nq), p.Nk = int(d->Nk);
  p.rows = d->rows;
  p.q_pos = q_pos, p.k_pos = k_pos, p.q_group = q_group, p.k_group = k_group;
  p.q_sb = d->q_pos_stride_b, p.k_sb = d->k_pos_stride_b;
  p.qg_sb = d->q_group_stride_b, p.kg_sb = d->k_group_stride_b;
  p.pos_vec = aligned16(k_pos) && (d->B == 1 || d->k_pos_stride_b % 4 == 0) &&
              (!groups || (aligned16(k_group) && (d->B == 1 || d->k_group_stride_b % 4 == 0)));
  pba::RelposRule &r = p.rule;
  const int buckets = d->rows - (groups ? 1 : 0);
  r.cross = groups ? buckets : -1;
  r.kind = d->rule;
  if (d->rule == PBA_RELPOS_CLIP) {
    r.far = buckets / 2;
    return;
  }
  r.side = d->rule == PBA_RELPOS_LOG ? buckets / 2 : buckets;
  r.exact = r.side / 2;
  r.n_borders = r.side - r.exact - 1;
  for (int t = 1; t <= r.n_borders; ++t)
    r.borders[t - 1] = log_border(r.exact, r.side - r.exact, t, d->max_distance);
  r.far = r.n_borders > 0 ? r.borders[r.n_borders - 1] : r.exact;
}

// Rows of 8-element chunks that start on 16 bytes each.
bool rows_vec(const void *base, const int64_t s[3], int64_t B, int64_t H, int64_t N, int dtype) {
  const int64_t m = 16 / dtype_size(dtype);
  return aligned16(base) && (B <= 1 || s[0] % m == 0) && (H <= 1 || s[1] % m == 0) && (N <= 1 || s[2] % m == 0);
}

template <typename T, bool kVec, bool kBase>
cudaError_t launch_relpos(const pba::RelposParams &p, dim3 grid, int smem, cudaStream_t stream) {
  auto kern = pba::relpos_fwd_kernel<T, kVec, kBase>;
  static PerDeviceOnce once;
  const cudaError_t attr_err = once_per_device(
      once, [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRelposSmem); });
  if (attr_err != cudaSuccess) return attr_err;
  kern<<<grid, pba::kRelposThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, bool kVec>
cudaError_t dispatch_relpos(const pba::RelposParams &p, dim3 grid, int smem, cudaStream_t st) {
  return p.base != nullptr ? launch_relpos<T, kVec, true>(p, grid, smem, st)
                           : launch_relpos<T, kVec, false>(p, grid, smem, st);
}

// Launch shape of the table's gradient.
struct GradPlan {
  int threads, cols_log2, col_blocks, row_splits;
  int64_t splits;  // tables per head
};
GradPlan grad_plan(const pba_relpos_desc *d) {
  GradPlan g;
  // as many threads as columns of `rows` floats and the widest ring fit in a
  // block's shared memory
  const int lookup = (pba::kRelposLutFar + 1) * 4;  // the largest
  const int per_thread = d->rows * 4 + pba::RelposGradRing<pba::F32, false>::kThreadBytes;
  g.threads = pba::kRelposGradThreads;
  while (g.threads > 32 && per_thread * g.threads + lookup > kRelposSmem) g.threads /= 2;
  const int64_t chunks = ceil_div(d->Nk, 8);
  const int64_t cols = std::min<int64_t>(g.threads, pow2_ceil(chunks));
  g.cols_log2 = 0;
  while ((int64_t(1) << g.cols_log2) < cols) ++g.cols_log2;
  g.col_blocks = int(ceil_div(chunks, cols));
  const int64_t lanes = g.threads / cols;
  // Queries are split until the card is full once (or twice, three times, ...:
  // no thread takes over 512, which bounds the error of its fp32 sums), and not
  // further than eight to a thread.
  const int ring = d->dtype == PBA_BF16 ? pba::RelposGradRing<pba::Bf16, true>::kThreadBytes
                                        : pba::RelposGradRing<pba::F32, true>::kThreadBytes;
  const int64_t resident =
      std::min<int64_t>(kRelposGradResident, 227 * 1024 / (g.threads * (d->rows * 4 + ring) + 1024));
  const int64_t fill = std::max<int64_t>(1, kPlanSms * resident / (d->H * d->B * g.col_blocks));
  const int64_t most = ceil_div(d->Nq, lanes * 8), least = ceil_div(d->Nq, lanes * 512);
  g.row_splits = int(std::max(least, std::min(most, fill * ceil_div(least, fill))));
  g.splits = d->B * g.col_blocks * g.row_splits;
  return g;
}

template <typename T, bool kVec>
cudaError_t launch_relpos_grad(const pba::RelposParams &p, const GradPlan &g, cudaStream_t stream) {
  auto kern = pba::relpos_grad_kernel<T, kVec>;
  static PerDeviceOnce once;
  const cudaError_t attr_err = once_per_device(
      once, [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRelposSmem); });
  if (attr_err != cudaSuccess) return attr_err;
  const int smem = g.threads * (p.rows * 4 + pba::RelposGradRing<T, kVec>::kThreadBytes) +
                   pba::relpos_lookup_words(p.rule) * 4;
  kern<<<dim3(unsigned(g.col_blocks * g.row_splits), unsigned(p.H), unsigned(p.B)), g.threads, smem, stream>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------ block norms
pba_status check_norm(const pba_norm_desc *d, const void *f, const void *gate, const void *scale, const void *post_w,
                      const void *post_b, const void *pre_w, const void *pre_b) {
  if (d == nullptr) return PBA_ERR_INVALID_ARG;
  if (d->rows < 0 || d->C < 1) return PBA_ERR_INVALID_ARG;
  if (!known_dtype(d->dtype) || !known_dtype(d->param_dtype) || d->C > pba::kNormMaxC) return PBA_ERR_UNSUPPORTED;
  if (d->kind != PBA_NORM_LAYER && d->kind != PBA_NORM_RMS) return PBA_ERR_INVALID_ARG;
  if (!(d->eps >= 1e-30f) || std::isinf(d->eps)) return PBA_ERR_INVALID_ARG;
  if (f == nullptr && (gate != nullptr || scale != nullptr || post_w != nullptr || pre_w == nullptr))
    return PBA_ERR_INVALID_ARG;
  if ((post_w == nullptr && post_b != nullptr) || (pre_w == nullptr && pre_b != nullptr)) return PBA_ERR_INVALID_ARG;
  return PBA_OK;
}

// Threads of a row, `channels` each, and rows of a block: a power of two of
// lanes in blocks of 256, or a block of whole warps to a row.
dim3 norm_block(int64_t C, int channels) {
  const int64_t lanes = ceil_div(C, channels);
  if (lanes > 32) return dim3(unsigned(ceil_div(lanes, 32) * 32), 1);
  const int64_t l = pow2_ceil(lanes);
  return dim3(unsigned(l), unsigned(pba::kNormNarrowThreads / l));
}
int norm_channels(int dtype, bool backward) {
  if (backward) return pba::kNormBwdChannels;
  return dtype == PBA_BF16 ? pba::norm_fwd_channels<pba::Bf16>() : pba::norm_fwd_channels<pba::F32>();
}

// Blocks of a launch: 512 threads to an SM, which is what the kernels'
// registers leave room for, each walking over its share of the rows; for the
// gradients so many times over that no thread's sums pass kNormMaxThreadRows.
int64_t norm_blocks(int64_t rows, dim3 block, bool backward) {
  const int64_t per_sm = std::max<int64_t>(1, 512 / (int64_t(block.x) * block.y));
  int64_t full = kPlanSms * per_sm;
  if (backward) full *= std::max<int64_t>(1, ceil_div(rows, full * block.y * pba::kNormMaxThreadRows));
  return std::max<int64_t>(1, std::min(ceil_div(rows, block.y), full));
}

bool norm_vec(const pba_norm_desc *d, const void *const *rows, const int64_t *strides, int n_rows,
              const void *const *params, int n_params) {
  const int64_t m = 16 / dtype_size(d->dtype);
  if (d->C % m != 0) return false;
  for (int i = 0; i < n_rows; ++i)
    if (rows[i] != nullptr && (!aligned16(rows[i]) || (d->rows > 1 && strides[i] % m != 0))) return false;
  for (int i = 0; i < n_params; ++i)
    if (params[i] != nullptr && !aligned16(params[i])) return false;
  return true;
}

// Outputs (null ones aside) whose rows lie on one another.
bool norm_rows_overlap(const pba_norm_desc &d, std::initializer_list<std::pair<const void *, int64_t>> outputs) {
  for (const auto &o : outputs)
    if (o.first != nullptr && d.rows > 1 && o.second == 0) return true;
  return false;
}

template <typename K>
cudaError_t start_norm_kernel(K kern, PerDeviceOnce &once, int smem, const pba::NormParams &p, unsigned grid,
                              dim3 block, cudaStream_t st) {
  const cudaError_t e = once_per_device(
      once, [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem); });
  if (e != cudaSuccess) return e;
  kern<<<grid, block, smem, st>>>(p);
  return cudaGetLastError();
}
template <typename T, bool kVec, int kThreads>
cudaError_t start_norm(const pba::NormParams &p, bool backward, unsigned grid, dim3 block, cudaStream_t st) {
  static PerDeviceOnce once[2];
  const int threads = int(block.x * block.y);
  using Fwd = pba::NormFwdStream<T, kVec, kThreads>;
  using Bwd = pba::NormBwdStream<T, kVec, kThreads>;
  static_assert(kThreads * Fwd::kThreadBytes <= kNormSmem && kThreads * Bwd::kThreadBytes <= kNormSmem, "ring");
  if (!backward) {
    // bf16 rows forward, 16 channels to a thread, need 512 threads at most
    if constexpr (kThreads == 1024 && pba::kNormMaxC / pba::norm_fwd_channels<T>() <= 512)
      return cudaErrorInvalidConfiguration;
    else
      return start_norm_kernel(pba::block_norm_fwd_kernel<T, kVec, kThreads>, once[0], threads * Fwd::kThreadBytes, p,
                               grid, block, st);
  }
  const int smem = threads * Bwd::kThreadBytes;
  if constexpr (kVec && kThreads <= 512) {
    // the sets of parts that have a kernel of their own
    constexpr int kAll = pba::norm_parts(true, true, true, true), kNoGate = pba::norm_parts(true, false, true, true),
                  kNoPost = pba::norm_parts(true, true, false, true), kAdd = pba::norm_parts(true, false, false, true),
                  kNorm = pba::norm_parts(false, false, false, true);
    static PerDeviceOnce known[5];
    const int parts = p.dh == nullptr ? -1
                                      : pba::norm_parts(p.f != nullptr, p.gate != nullptr, p.post_w != nullptr,
                                                        p.pre_w != nullptr);
    auto start = [&](auto kern, int i) { return start_norm_kernel(kern, known[i], smem, p, grid, block, st); };
    switch (parts) {
      case kAll: return start(pba::block_norm_bwd_kernel<T, kVec, kThreads, kAll>, 0);
      case kNoGate: return start(pba::block_norm_bwd_kernel<T, kVec, kThreads, kNoGate>, 1);
      case kNoPost: return start(pba::block_norm_bwd_kernel<T, kVec, kThreads, kNoPost>, 2);
      case kAdd: return start(pba::block_norm_bwd_kernel<T, kVec, kThreads, kAdd>, 3);
      case kNorm: return start(pba::block_norm_bwd_kernel<T, kVec, kThreads, kNorm>, 4);
    }
  }
  return start_norm_kernel(pba::block_norm_bwd_kernel<T, kVec, kThreads, -1>, once[1], smem, p, grid, block, st);
}

template <typename T, bool kVec>
cudaError_t launch_norm(const pba::NormParams &p, bool backward, unsigned grid, dim3 block, cudaStream_t st) {
  // rows that share a block, rows of a block, and rows of a block so large
  // that each thread has half the registers
  if (block.x <= 32) return start_norm<T, kVec, pba::kNormNarrowThreads>(p, backward, grid, block, st);
  if (block.x <= 512) return start_norm<T, kVec, 512>(p, backward, grid, block, st);
  return start_norm<T, kVec, 1024>(p, backward, grid, block, st);
}

cudaError_t dispatch_norm(const pba::NormParams &p, int dtype, bool vec, bool backward, cudaStream_t st) {
  const dim3 block = norm_block(p.C, norm_channels(dtype, backward));
  const unsigned grid = unsigned(norm_blocks(p.rows, block, backward));
  if (dtype == PBA_BF16)
    return vec ? launch_norm<pba::Bf16, true>(p, backward, grid, block, st)
               : launch_norm<pba::Bf16, false>(p, backward, grid, block, st);
  return vec ? launch_norm<pba::F32, true>(p, backward, grid, block, st)
             : launch_norm<pba::F32, false>(p, backward, grid, block, st);
}

void fill_norm(pba::NormParams &p, const pba_norm_desc *d, const void *f, const void *gate, const void *scale,
               const void *post_w, const void *post_b, const void *pre_w, const void *pre_b) {
  std::memset(&p, 0, sizeof(p));
  p.rows = d->rows;
  p.C = int(d->C);
  p.layer = d->kind == PBA_NORM_LAYER;
  p.param_f32 = d->param_dtype == PBA_F32;
  p.eps = d->eps;
  p.inv_c = float(1.0 / double(d->C));
  p.f = f, p.gate = gate, p.scale = scale;
  p.post_w = post_w, p.post_b = post_b, p.pre_w = pre_w, p.pre_b = pre_b;
  p.x_s = d->x_stride, p.f_s = d->f_stride, p.gate_s = d->gate_stride, p.h_s = d->h_stride, p.y_s = d->y_stride;
  p.dh_s = d->dh_stride, p.dy_s = d->dy_stride, p.dx_s = d->dx_stride, p.df_s = d->df_stride;
  p.dgate_s = d->dgate_stride;
}

}  // namespace

extern "C" {

pba_status pba_relpos_bias_forward(const pba_relpos_desc *desc, const int32_t *q_pos, const int32_t *k_pos,
                               const int32_t *q_group, const int32_t *k_group, const void *table, const void *base,
                               void *out, void *stream_ptr) {
  pba_status s = check_relpos(desc, q_group != nullptr);
  if (s != PBA_OK) return s;
  if ((q_group == nullptr) != (k_group == nullptr)) return PBA_ERR_INVALID_ARG;
  const pba_relpos_desc &d = *desc;
  if (d.Nq == 0 || d.Nk == 0) return PBA_OK;  // nothing to write
  if (q_pos == nullptr || k_pos == nullptr || table == nullptr || out == nullptr) return PBA_ERR_INVALID_ARG;
  const int size = dtype_size(d.dtype);
  if (!aligned_to(q_pos, 4) || !aligned_to(k_pos, 4) || !aligned_to(q_group, 4) || !aligned_to(k_group, 4) ||
      !aligned_to(table, size) || !aligned_to(base, size) || !aligned_to(out, size) ||
      !rows_apart(d.out_stride, d.B, d.H, d.Nq))
    return PBA_ERR_INVALID_ARG;
  s = check_device();
  if (s != PBA_OK) return s;
  pba::RelposParams p;
  fill_relpos(p, desc, q_pos, k_pos, q_group, k_group);
  p.table = table, p.base = base, p.out = out;
  for (int i = 0; i < 3; ++i) p.base_s[i] = d.base_stride[i], p.out_s[i] = d.out_stride[i];
  // fp32 rows go element by element, 128 bytes of a warp at a time, wherever
  // they lie: eights of 32 bytes in two 16-byte accesses, half a sector each,
  // took 81 us for 16 x 2048^2 and 138 with a base, against 48 and 95.
  const bool vec = d.dtype == PBA_BF16 && rows_vec(out, d.out_stride, d.B, d.H, d.Nq, d.dtype) &&
                   (base == nullptr || rows_vec(base, d.base_stride, d.B, d.H, d.Nq, d.dtype));
  // Heads per block: all that fit (the rows of the table are found once for
  // them all), fewer when that would leave SMs without a block.
  const int per_word = d.dtype == PBA_BF16 ? 2 : 1;
  const int lookup = pba::relpos_lookup_words(p.rule);
  const int ring = base != nullptr && vec ? pba::kRelposBaseStages * pba::kRelposThreads * 8 * size : 0;
  const int64_t fit = ((kRelposSmem - ring) / 4 - lookup - 4) / d.rows * per_word;
  const int64_t blocks = vec ? ceil_div(d.B * d.Nq * ceil_div(d.Nk, 8), pba::kRelposThreads)
                             : ceil_div(d.B * d.Nq * ceil_div(d.Nk, 256), pba::kRelposThreads / 32);
  int64_t heads = std::min<int64_t>(d.H, fit);
  if (blocks * ceil_div(d.H, heads) < 2 * kPlanSms)
    heads = std::min(heads, std::max<int64_t>(per_word, d.H * blocks / (2 * kPlanSms) / per_word * per_word));
  if (heads < d.H) heads = std::max<int64_t>(per_word, heads / per_word * per_word);
  p.heads_per_block = int(heads);
  p.ring_offset = int(ceil_div((lookup + ceil_div(heads, per_word) * d.rows) * 4, 16) * 16);
  const int smem = p.ring_offset + ring;
  // a block stages its table once and then walks over its share of the rows
  const dim3 grid(unsigned(std::min<int64_t>(blocks, 8 * kPlanSms)), unsigned(ceil_div(d.H, heads)));
  cudaStream_t st = static_cast<cudaStream_t>(stream_ptr);
  const cudaError_t e = d.dtype == PBA_F32 ? dispatch_relpos<pba::F32, false>(p, grid, smem, st)
                        : vec              ? dispatch_relpos<pba::Bf16, true>(p, grid, smem, st)
                                           : dispatch_relpos<pba::Bf16, false>(p, grid, smem, st);
  return e == cudaSuccess ? PBA_OK : PBA_ERR_CUDA;
}

pba_status pba_relpos_bias_backward_workspace(const pba_relpos_desc *desc, int64_t *bytes) {
  // groups take a row of the table, not of the workspace: either reading of `rows` will do
  pba_status s = check_relpos(desc, false);
  if (s != PBA_OK) s = check_relpos(desc, true);
  if (s != PBA_OK) return s;
  if (bytes == nullptr) return PBA_ERR_INVALID_ARG;
  const int64_t splits = desc->Nq == 0 || desc->Nk == 0 ? 0 : grad_plan(desc).splits;
  if (splits > kMaxI32) return PBA_ERR_INVALID_ARG;  // as the backward itself
  *bytes = splits * desc->H * desc->rows * 4;
  return PBA_OK;
}

pba_status pba_relpos_bias_backward(const pba_relpos_desc *desc, const int32_t *q_pos, const int32_t *k_pos,
                                const int32_t *q_group, const int32_t *k_group, const void *dbias, float *dtable,
                                void *workspace, int64_t workspace_bytes, void *stream_ptr) {
  pba_status s = check_relpos(desc, q_group != nullptr);
  if (s != PBA_OK) return s;
  if ((q_group == nullptr) != (k_group == nullptr) || dtable == nullptr) return PBA_ERR_INVALID_ARG;
  const pba_relpos_desc &d = *desc;
  const bool empty = d.Nq == 0 || d.Nk == 0;
  const int size = dtype_size(d.dtype);
  if (!empty && (q_pos == nullptr || k_pos == nullptr || dbias == nullptr || workspace == nullptr))
    return PBA_ERR_INVALID_ARG;
  if (!aligned_to(q_pos, 4) || !aligned_to(k_pos, 4) || !aligned_to(q_group, 4) || !aligned_to(k_group, 4) ||
      !aligned_to(dbias, size) || !aligned_to(dtable, 4) || !aligned_to(workspace, 4))
    return PBA_ERR_INVALID_ARG;
  GradPlan g{};
  if (!empty) {
    g = grad_plan(desc);
    if (g.splits > kMaxI32 || workspace_bytes < g.splits * d.H * d.rows * 4) return PBA_ERR_INVALID_ARG;
  }
  s = check_device();
  if (s != PBA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream_ptr);
  float *part = static_cast<float *>(workspace);
  if (!empty) {
    pba::RelposParams p;
    fill_relpos(p, desc, q_pos, k_pos, q_group, k_group);
    p.out = const_cast<void *>(dbias);  // read
    for (int i = 0; i < 3; ++i) p.out_s[i] = d.out_stride[i];
    p.part = part;
    p.splits = int(g.splits), p.row_splits = g.row_splits, p.col_blocks = g.col_blocks, p.cols_log2 = g.cols_log2;
    const bool vec = rows_vec(dbias, d.out_stride, d.B, d.H, d.Nq, d.dtype);
    const cudaError_t e =
        d.dtype == PBA_BF16
            ? (vec ? launch_relpos_grad<pba::Bf16, true>(p, g, st) : launch_relpos_grad<pba::Bf16, false>(p, g, st))
            : (vec ? launch_relpos_grad<pba::F32, true>(p, g, st) : launch_relpos_grad<pba::F32, false>(p, g, st));
    if (e != cudaSuccess) return PBA_ERR_CUDA;
  }
  pba::relpos_grad_sum_kernel<<<dim3(unsigned(ceil_div(d.rows, 32)), unsigned(d.H)), dim3(32, 8), 0, st>>>(
      part, dtable, int(g.splits), d.rows, int(d.H));
  return cudaGetLastError() == cudaSuccess ? PBA_OK : PBA_ERR_CUDA;
}

pba_status pba_block_norm_forward(const pba_norm_desc *desc, const void *x, const void *f, const void *gate,
                              const void *scale, const void *post_w, const void *post_b, const void *pre_w,
                              const void *pre_b, void *h, void *y, void *stream_ptr) {
  pba_status s = check_norm(desc, f, gate, scale, post_w, post_b, pre_w, pre_b);
  if (s != PBA_OK) return s;
  const pba_norm_desc &d = *desc;
  if (d.rows == 0) return PBA_OK;  // nothing to write
  if (x == nullptr || (f != nullptr && h == nullptr) || (pre_w != nullptr && y == nullptr)) return PBA_ERR_INVALID_ARG;
  if (f == nullptr) h = nullptr;
  if (pre_w == nullptr) y = nullptr;
  const void *rows[] = {x, f, gate, h, y}, *params[] = {scale, post_w, post_b, pre_w, pre_b};
  const int64_t strides[] = {d.x_stride, d.f_stride, d.gate_stride, d.h_stride, d.y_stride};
  for (const void *r : rows)
    if (!aligned_to(r, dtype_size(d.dtype))) return PBA_ERR_INVALID_ARG;
  for (const void *r : params)
    if (!aligned_to(r, dtype_size(d.param_dtype))) return PBA_ERR_INVALID_ARG;
  if (norm_rows_overlap(d, {{h, d.h_stride}, {y, d.y_stride}})) return PBA_ERR_INVALID_ARG;
  s = check_device();
  if (s != PBA_OK) return s;
  pba::NormParams p;
  fill_norm(p, desc, f, gate, scale, post_w, post_b, pre_w, pre_b);
  p.x = x, p.h = h, p.y = y;
  const cudaError_t e = dispatch_norm(p, d.dtype, norm_vec(desc, rows, strides, 5, params, 5), false,
                                      static_cast<cudaStream_t>(stream_ptr));
  return e == cudaSuccess ? PBA_OK : PBA_ERR_CUDA;
}

pba_status pba_block_norm_backward_workspace(const pba_norm_desc *desc, int64_t *bytes) {
  if (desc == nullptr || bytes == nullptr || desc->rows < 0 || desc->C < 1) return PBA_ERR_INVALID_ARG;
  if (desc->C > pba::kNormMaxC) return PBA_ERR_UNSUPPORTED;
  const int64_t blocks =
      desc->rows == 0 ? 0 : norm_blocks(desc->rows, norm_block(desc->C, norm_channels(desc->dtype, true)), true);
  *bytes = blocks * pba::kNormParams * desc->C * 4;
  return PBA_OK;
}

pba_status pba_block_norm_backward(const pba_norm_desc *desc, const void *h, const void *f, const void *gate,
                               const void *scale, const void *post_w, const void *post_b, const void *pre_w,
                               const void *pre_b, const void *dh, const void *dy, void *dx, void *df, void *dgate,
                               float *dscale, float *dpost_w, float *dpost_b, float *dpre_w, float *dpre_b,
                               void *workspace, int64_t workspace_bytes, void *stream_ptr) {
  pba_status s = check_norm(desc, f, gate, scale, post_w, post_b, pre_w, pre_b);
  if (s != PBA_OK) return s;
  const pba_norm_desc &d = *desc;
  const bool pre = pre_w != nullptr;
  if (d.rows > 0) {
    if (dx == nullptr || (pre ? h == nullptr || dy == nullptr : dh == nullptr)) return PBA_ERR_INVALID_ARG;
    if ((f != nullptr && df == nullptr) || (gate != nullptr && dgate == nullptr) || workspace == nullptr)
      return PBA_ERR_INVALID_ARG;
  }
  // what is not read or written does not matter for the layout either
  if (!pre) h = nullptr, dy = nullptr;
  if (f == nullptr) df = nullptr;
  if (gate == nullptr) dgate = nullptr;
  const void *rows[] = {h, f, gate, dh, dy, dx, df, dgate}, *params[] = {scale, post_w, post_b, pre_w, pre_b};
  const int64_t strides[] = {d.h_stride,  d.f_stride,  d.gate_stride, d.dh_stride,
                             d.dy_stride, d.dx_stride, d.df_stride,   d.dgate_stride};
  for (const void *r : rows)
    if (!aligned_to(r, dtype_size(d.dtype))) return PBA_ERR_INVALID_ARG;
  for (const void *r : params)
    if (!aligned_to(r, dtype_size(d.param_dtype))) return PBA_ERR_INVALID_ARG;
  if (norm_rows_overlap(d, {{dx, d.dx_stride}, {df, d.df_stride}, {dgate, d.dgate_stride}})) return PBA_ERR_INVALID_ARG;
  pba::NormSumParams sp;
  std::memset(&sp, 0, sizeof(sp));
  sp.out[0] = scale != nullptr ? dscale : nullptr;
  sp.out[1] = post_w != nullptr ? dpost_w : nullptr;
  sp.out[2] = post_b != nullptr ? dpost_b : nullptr;
  sp.out[3] = pre ? dpre_w : nullptr;
  sp.out[4] = pre_b != nullptr ? dpre_b : nullptr;
  bool any = false;
  for (const float *o : sp.out) {
    if (!aligned_to(o, 4)) return PBA_ERR_INVALID_ARG;
    any = any || o != nullptr;
  }
  const int64_t blocks = d.rows == 0 ? 0 : norm_blocks(d.rows, norm_block(d.C, norm_channels(d.dtype, true)), true);
  if (!aligned_to(workspace, 4) || workspace_bytes < blocks * pba::kNormParams * d.C * 4) return PBA_ERR_INVALID_ARG;
  s = check_device();
  if (s != PBA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream_ptr);
  if (d.rows > 0) {
    pba::NormParams p;
    fill_norm(p, desc, f, gate, scale, post_w, post_b, pre_w, pre_b);
    p.h = const_cast<void *>(h);  // read
    p.dh = dh, p.dy = dy, p.dx = dx, p.df = df, p.dgate = dgate;
    p.part = static_cast<float *>(workspace);
    if (dispatch_norm(p, d.dtype, norm_vec(desc, rows, strides, 8, params, 5), true, st) !=
        cudaSuccess)
      return PBA_ERR_CUDA;
  }
  if (any) {
    sp.part = static_cast<const float *>(workspace);
    sp.blocks = int(blocks);
    sp.C = int(d.C);
    pba::block_norm_sum_kernel<<<dim3(unsigned(ceil_div(d.C, 32)), pba::kNormParams), dim3(32, 8), 0, st>>>(sp);
    if (cudaGetLastError() != cudaSuccess) return PBA_ERR_CUDA;
  }
  return PBA_OK;
}

}  // extern "C"
