// pba_cross_api.cu -- cross attention and its gradients as declared in
// include/pba.h: argument checks, tile descriptors, the choice of kernel and
// the launches.  The computation runs in the kernels of pba_cross_sm100.cuh,
// pba_cross_split.cuh and pba_cross_bwd_sm100.cuh.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "pba.h"
#include "pba_cross_bwd_sm100.cuh"
#include "pba_cross_sm100.cuh"
#include "pba_cross_split.cuh"
#include "pba_host.cuh"

using namespace pba_host;

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

pba_status check_cross(const pba_cross_desc *d) {
  if (d == nullptr) return PBA_ERR_INVALID_ARG;
  if (d->B < 1 || d->H < 1 || d->Hkv < 1 || d->Nq < 0 || d->Nk < 0) return PBA_ERR_INVALID_ARG;
  if (d->B > kMaxI32 || d->H > 65535 || d->Nq > kMaxI32 - 4096 || d->Nk > kMaxI32 - 4096)
    return PBA_ERR_INVALID_ARG;
  if (d->H % d->Hkv != 0) return PBA_ERR_INVALID_ARG;
  if (d->dtype != PBA_BF16) return PBA_ERR_UNSUPPORTED;
  if (d->D != 32 && d->D != 64 && d->D != 128) return PBA_ERR_UNSUPPORTED;
  if (!(d->softmax_scale >= 0.f) || std::isinf(d->softmax_scale)) return PBA_ERR_INVALID_ARG;
  return PBA_OK;
}

float cross_tau(const pba_cross_desc *d) {
  return d->softmax_scale > 0.f ? d->softmax_scale : float(1.0 / std::sqrt(double(d->D)));
}

bool strides_ok(const int64_t s[3], int64_t B, int64_t H, int64_t N) {
  return stride_ok_bf16(s[0], B) && stride_ok_bf16(s[1], H) && stride_ok_bf16(s[2], N);
}
// Rows that only plain 16-byte accesses touch: any sign, and 0 to share.
bool rows_ok(const int64_t s[3], int64_t B, int64_t H, int64_t N) {
  return (B <= 1 || s[0] % 8 == 0) && (H <= 1 || s[1] % 8 == 0) && (N <= 1 || s[2] % 8 == 0);
}

// [B][heads][n][D] as (D, n, heads, B): boxes of `rows` rows of at most 64 features.
bool cross_map(CUtensorMap *m, const void *base, int64_t D, int64_t n, int64_t heads, int64_t B, const int64_t s[3],
               int rows = pba::kXTile) {
  const uint64_t dims[4] = {uint64_t(D), uint64_t(n), uint64_t(heads), uint64_t(B)};
  const int64_t st[3] = {s[2] * 2, s[1] * 2, s[0] * 2};
  const uint32_t box[4] = {uint32_t(std::min<int64_t>(D, 64)), uint32_t(rows), 1, 1};
  return make_map(m, base, dims, st, box, D == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// What every call reads: q, k, v, and the mask.
pba_status check_cross_inputs(const pba_cross_desc &d, const void *q, const void *k, const void *v,
                              const int32_t *k_len) {
  if (d.Nq > 0 && q == nullptr) return PBA_ERR_INVALID_ARG;
  if (d.Nk > 0 && (k == nullptr || v == nullptr)) return PBA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(k_len) & 3u) != 0)
    return PBA_ERR_INVALID_ARG;
  if (!strides_ok(d.q_stride, d.B, d.H, d.Nq) || !strides_ok(d.k_stride, d.B, d.Hkv, d.Nk) ||
      !strides_ok(d.v_stride, d.B, d.Hkv, d.Nk))
    return PBA_ERR_INVALID_ARG;
  return PBA_OK;
}

bool mask_words(const pba_cross_desc &d, const uint8_t *mask) {
  return (reinterpret_cast<uintptr_t>(mask) & 3u) == 0 && (d.B == 1 || d.mask_stride_b % 4 == 0);
}

// Dynamic shared memory and the register split of a kernel whose warpgroups
// move registers with setmaxnreg: the split must fit in what the block is
// launched with, or the increase would wait forever.  Such a build is refused.
template <typename K>
cudaError_t set_up(K kern, int smem) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  cudaFuncAttributes fa;
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kern);
  if (e == cudaSuccess && fa.numRegs * pba::kXThreads < pba::kXRegSplitTotal) e = cudaErrorInvalidConfiguration;
  return e;
}

// A launch in clusters of `splits` blocks.
struct ClusterLaunch {
  cudaLaunchAttribute cluster;
  cudaLaunchConfig_t cfg;
  ClusterLaunch(int64_t grid, int threads, int splits, int smem, cudaStream_t stream) {
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = unsigned(splits), cluster.val.clusterDim.y = 1, cluster.val.clusterDim.z = 1;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
  }
  ClusterLaunch(const ClusterLaunch &) = delete;  // cfg points at cluster
};

// Clusters of 1 to kXMaxSplits blocks of a kernel that the current device holds
// at once: [blocks].  A cluster lies within one of the chip's groups of SMs, whose
// sizes differ, so this is less than the SMs' number divided (for one block an SM
// 15 clusters of eight on 148 SMs, 33 of four), and a cluster more waits for a
// whole round of the others.
struct ClusterRoom {
  PerDeviceOnce once;
  int room[kMaxDevices][pba::kXMaxSplits + 1] = {};
};
template <typename K, typename F>
cudaError_t cluster_room(ClusterRoom &r, K kern, int threads, int smem, F &&set_up_kernel, const int *&room) {
  const cudaError_t e = once_per_device(r.once, [&]() -> cudaError_t {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = set_up_kernel();
    for (int n = 1; n <= pba::kXMaxSplits && err == cudaSuccess; ++n) {
      ClusterLaunch c(n, threads, n, smem, nullptr);
      err = cudaOccupancyMaxActiveClusters(&r.room[dev][n], kern, &c.cfg);
    }
    return err;
  });
  if (e != cudaSuccess) return e;
  int dev = 0;
  const cudaError_t err = cudaGetDevice(&dev);
  room = r.room[dev];
  return err;
}

template <int D>
cudaError_t tile_room(const int *&room) {
  static ClusterRoom r;
  constexpr int smem = pba::CrossLayout<D>::kSmemAlloc;
  auto kern = pba::pba_cross_sm100_kernel<D, true>;
  return cluster_room(r, kern, pba::kXThreads, smem, [&] { return set_up(kern, smem); }, room);
}

template <int D>
cudaError_t split_room(const int *&room) {
  static ClusterRoom r;
  constexpr int smem = pba::cross_split_smem<D>();
  auto kern = pba::pba_cross_split_kernel<D>;
  return cluster_room(
      r, kern, pba::kXsThreads, smem,
      [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); }, room);
}

template <int D, bool kShared>
cudaError_t launch_cross(const pba::CrossParams &p, int64_t grid, cudaStream_t stream) {
  auto kern = pba::pba_cross_sm100_kernel<D, kShared>;
  constexpr int smem = pba::CrossLayout<D>::kSmemAlloc;
  if (kShared) {  // set up by tile_room
    ClusterLaunch c(grid, pba::kXThreads, p.splits, smem, stream);
    return cudaLaunchKernelEx(&c.cfg, kern, p);
  }
  static PerDeviceOnce once;
  const cudaError_t err = once_per_device(once, [&] { return set_up(kern, smem); });
  if (err != cudaSuccess) return err;
  kern<<<unsigned(grid), pba::kXThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

// CTAs that share a unit of the tile kernel: as many as the device holds clusters
// of for all units, a power of two (the join shares out 256 rows), each with two
// key tiles at least.
int tile_splits(const pba_cross_desc &d, int64_t units, const int *room) {
  const int64_t tiles = ceil_div(d.Nk, pba::kXTile);
  int s = 1;
  while (s < pba::kXMaxSplits && units <= room[2 * s] && tiles >= s * 4) s *= 2;
  return s;
}

template <int D>
pba_status run_tiles(const pba_cross_desc &d, const void *q, const void *k, const void *v, const int32_t *k_len,
                     const uint8_t *mask, void *out, float *lse, const int *room, cudaStream_t stream) {
  pba::CrossParams p;
  std::memset(&p, 0, sizeof(p));
  if (!cross_map(&p.tm_q, q, D, d.Nq, d.H, d.B, d.q_stride)) return PBA_ERR_INVALID_ARG;
  // without a key no unit loads any
  if (d.Nk > 0 && (!cross_map(&p.tm_k, k, D, d.Nk, d.Hkv, d.B, d.k_stride) ||
                   !cross_map(&p.tm_v, v, D, d.Nk, d.Hkv, d.B, d.v_stride)))
    return PBA_ERR_INVALID_ARG;
  p.B = int(d.B), p.H = int(d.H), p.group = int(d.H / d.Hkv), p.Nq = int(d.Nq), p.Nk = int(d.Nk);
  p.n_qblocks = int(ceil_div(d.Nq, pba::kXQTiles * pba::kXTile));
  const int64_t n_units = d.B * d.H * p.n_qblocks;
  if (n_units > kMaxI32 - 65536) return PBA_ERR_INVALID_ARG;
  p.n_units = int(n_units);
  p.tau = cross_tau(&d);
  p.k_len = k_len;
  p.mask = mask, p.mask_sb = d.mask_stride_b, p.mask_vec4 = mask_words(d, mask);
  p.out = static_cast<uint16_t *>(out);
  p.out_sb = d.out_stride[0], p.out_sh = d.out_stride[1], p.out_sn = d.out_stride[2];
  p.lse = lse;
  p.lse_sb = d.lse_stride[0], p.lse_sh = d.lse_stride[1], p.lse_sn = d.lse_stride[2];
  p.err = device_error_word();
  const int sms = sm_count();
  if (p.err == nullptr || sms < 1) return PBA_ERR_CUDA;
  p.timeout_ns = wait_timeout_ns();
  p.splits = tile_splits(d, n_units, room);
  // persistent, one CTA per SM, or a cluster for each unit
  const int64_t grid = p.splits > 1 ? n_units * p.splits : std::min<int64_t>(n_units, sms);
  const cudaError_t e = p.splits > 1 ? launch_cross<D, true>(p, grid, stream) : launch_cross<D, false>(p, grid, stream);
  return e == cudaSuccess ? PBA_OK : PBA_ERR_CUDA;
}

// Blocks that share 16 query rows: as many, up to a cluster, as the device holds
// clusters of for all units, each with at least one step per warp.
int split_count(const pba_cross_desc &d, int64_t units, const int *room) {
  const int64_t most = std::min<int64_t>(pba::kXMaxSplits, ceil_div(d.Nk, pba::kXsWarps * pba::kXsKeys));
  int n = 1;
  while (n < most && units <= room[n + 1]) ++n;
  return n;
}

template <int D>
pba_status run_split(const pba_cross_desc &d, const void *q, const void *k, const void *v, const int32_t *k_len,
                     const uint8_t *mask, void *out, float *lse, const int *room, cudaStream_t stream) {
  pba::CrossSplitParams p;
  std::memset(&p, 0, sizeof(p));
  p.B = int(d.B), p.H = int(d.H), p.Hkv = int(d.Hkv), p.group = int(d.H / d.Hkv), p.Nq = int(d.Nq), p.Nk = int(d.Nk);
  p.row_tiles = int(ceil_div(d.H / d.Hkv * d.Nq, pba::kXsRows));
  p.tau = cross_tau(&d);
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k), p.v = static_cast<const uint16_t *>(v);
  p.q_sb = d.q_stride[0], p.q_sh = d.q_stride[1], p.q_sn = d.q_stride[2];
  p.k_sb = d.k_stride[0], p.k_sh = d.k_stride[1], p.k_sn = d.k_stride[2];
  p.v_sb = d.v_stride[0], p.v_sh = d.v_stride[1], p.v_sn = d.v_stride[2];
  p.k_len = k_len, p.mask = mask, p.mask_sb = d.mask_stride_b;
  p.out = static_cast<uint16_t *>(out);
  p.out_sb = d.out_stride[0], p.out_sh = d.out_stride[1], p.out_sn = d.out_stride[2];
  p.lse = lse;
  p.lse_sb = d.lse_stride[0], p.lse_sh = d.lse_stride[1], p.lse_sn = d.lse_stride[2];
  const int64_t units = d.B * d.Hkv * p.row_tiles;
  const int splits = split_count(d, units, room);
  if (units * splits > kMaxI32) return PBA_ERR_INVALID_ARG;
  ClusterLaunch c(units * splits, pba::kXsThreads, splits, pba::cross_split_smem<D>(), stream);  // set up by split_room
  return cudaLaunchKernelEx(&c.cfg, pba::pba_cross_split_kernel<D>, p) == cudaSuccess ? PBA_OK : PBA_ERR_CUDA;
}

// What a call takes on either kernel, in us, from the measurements below: a
// start, a time per step of a block (or CTA) and, few rows, the rate at which
// the steps of all blocks read keys and values, from L2 after the first time.
template <int D>
struct CrossCost {
  static constexpr double kRowsStart = D == 32 ? 5.5 : D == 64 ? 6.0 : 7.0, kRowsRound = D == 128 ? 6.0 : 3.0;
  static constexpr double kRowsStep = D == 32 ? 0.34 : D == 64 ? 0.42 : 0.60;        // four warps, 16 keys each
  static constexpr double kRowsMbPerUs = D == 32 ? 7.0 : D == 64 ? 9.25 : 8.75;      // TB/s
  static constexpr double kTileStart = D == 128 ? 7.5 : 5.8, kTile = D == 128 ? 2.06 : 1.44;  // a CTA to a unit
  static constexpr double kSharedStart = 8.0, kSharedTile = D == 128 ? 2.65 : 1.5;            // clusters
  static constexpr double kSharedJoin = D == 32 ? 4.0 : D == 64 ? 11.0 : 20.0;                // over their CTAs
};

// Whether the kernel for few rows is the faster one.  It reads keys and values
// once for every 16 query rows of a key head; the tile kernel does the work of
// 256 rows of every head, however few of them there are.  The costs were fitted
// to both kernels' times at 1515 shapes (1 to 64 key heads in groups of 1 to 8, 1
// to 512 queries, 512 to 131072 keys, each D); at 1489 of them the faster kernel
// is chosen, at 1507 one within 5 % of it, at the worst one 9 % behind.  Few rows
// against tiles: D = 64, 8192 keys, 16 heads of 64 queries 21.7 and 35.6 us, 32
// heads of 64 34.7 and 36.1, of 128 59.8 and 36.0; D = 32, 2048 keys, 32 heads of
// 96 13.2 and 15.3; D = 128, 2048 keys, 32 heads of 64 23.0 and 30.0, of 128 37.7
// and 29.4.
template <int D>
bool few_rows(const pba_cross_desc &d, const int *tiles_room, const int *rows_room) {
  using C = CrossCost<D>;
  if (d.H / d.Hkv * d.Nq > kMaxI32 - pba::kXsRows) return false;  // rows of a key head count in 32 bits
  const int64_t r_units = d.B * d.Hkv * ceil_div(d.H / d.Hkv * d.Nq, pba::kXsRows);
  const int n = split_count(d, r_units, rows_room);
  const double steps = double(ceil_div(ceil_div(ceil_div(d.Nk, pba::kXsKeys), n), pba::kXsWarps));
  const double blocks = double(r_units) * n, rounds = std::ceil(blocks / std::max(1, rows_room[1]));
  const double mb = blocks * steps * (pba::kXsWarps * pba::kXsKeys * D * 4) * 1e-6;
  const double rows = C::kRowsStart + C::kRowsRound * (rounds - 1.0) +
                      std::max(rounds * steps * C::kRowsStep, mb / C::kRowsMbPerUs);
  const int64_t t_units = d.B * d.H * ceil_div(d.Nq, pba::kXQTiles * pba::kXTile);
  const int s = tile_splits(d, t_units, tiles_room);
  const double per = double(ceil_div(ceil_div(d.Nk, pba::kXTile), s));
  const double tiles = s > 1 ? C::kSharedStart + C::kSharedJoin / s + per * C::kSharedTile
                             : C::kTileStart + std::ceil(double(t_units) / std::max(1, tiles_room[1])) * per * C::kTile;
  return rows <= tiles;
}

template <int D>
pba_status run_forward(const pba_cross_desc &d, const void *q, const void *k, const void *v, const int32_t *k_len,
                       const uint8_t *mask, void *out, float *lse, cudaStream_t stream) {
  const int *tiles = nullptr, *rows = nullptr;
  if (tile_room<D>(tiles) != cudaSuccess || split_room<D>(rows) != cudaSuccess) return PBA_ERR_CUDA;
  return few_rows<D>(d, tiles, rows) ? run_split<D>(d, q, k, v, k_len, mask, out, lse, rows, stream)
                            : run_tiles<D>(d, q, k, v, k_len, mask, out, lse, tiles, stream);
}

template <int D>
cudaError_t launch_cross_bwd(const pba::CrossBwdParams &p, int64_t grid, cudaStream_t stream) {
  auto kern = pba::pba_cross_bwd_sm100_kernel<D>;
  constexpr int smem = pba::CrossBwdLayout<D>::kSmemAlloc;
  static PerDeviceOnce once;
  const cudaError_t err = once_per_device(once, [&] { return set_up(kern, smem); });
  if (err != cudaSuccess) return err;
  kern<<<unsigned(grid), pba::kXThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
pba_status run_cross_bwd(const pba_cross_desc &d, const void *q, const void *k, const void *v, const void *out,
                         const float *lse, const void *dout, const int32_t *k_len, const uint8_t *mask, void *dq,
                         void *dk, void *dv, float *delta, cudaStream_t stream) {
  pba::CrossBwdParams p;
  std::memset(&p, 0, sizeof(p));
  // a side without rows is loaded by no unit
  if (d.Nq > 0 && (!cross_map(&p.tm_q, q, D, d.Nq, d.H, d.B, d.q_stride, pba::kXBox) ||
                   !cross_map(&p.tm_do, dout, D, d.Nq, d.H, d.B, d.dout_stride, pba::kXBox)))
    return PBA_ERR_INVALID_ARG;
  if (d.Nk > 0 && (!cross_map(&p.tm_k, k, D, d.Nk, d.Hkv, d.B, d.k_stride, pba::kXBox) ||
                   !cross_map(&p.tm_v, v, D, d.Nk, d.Hkv, d.B, d.v_stride, pba::kXBox)))
    return PBA_ERR_INVALID_ARG;
  p.B = int(d.B), p.H = int(d.H), p.Hkv = int(d.Hkv), p.group = int(d.H / d.Hkv), p.Nq = int(d.Nq), p.Nk = int(d.Nk);
  p.tau = cross_tau(&d);
  p.k_len = k_len;
  p.mask = mask, p.mask_sb = d.mask_stride_b;
  p.lse = lse;
  p.lse_sb = d.lse_stride[0], p.lse_sh = d.lse_stride[1], p.lse_sn = d.lse_stride[2];
  p.delta = delta;
  p.dq = static_cast<uint16_t *>(dq), p.dk = static_cast<uint16_t *>(dk), p.dv = static_cast<uint16_t *>(dv);
  p.err = device_error_word();
  if (p.err == nullptr) return PBA_ERR_CUDA;
  p.timeout_ns = wait_timeout_ns();
  const int64_t q_tiles = ceil_div(d.Nq, pba::kXTile), k_tiles = ceil_div(d.Nk, pba::kXTile);
  const int64_t grid_a = d.B * d.H * q_tiles, grid_b = d.B * d.Hkv * k_tiles;
  if (grid_a + grid_b > kMaxI32 || d.H / d.Hkv * q_tiles * 2 > kMaxI32) return PBA_ERR_INVALID_ARG;
  if (d.Nq > 0) {
    pba::CrossDeltaParams dp;
    dp.dout = static_cast<const uint16_t *>(dout), dp.out = static_cast<const uint16_t *>(out);
    dp.do_sb = d.dout_stride[0], dp.do_sh = d.dout_stride[1], dp.do_sn = d.dout_stride[2];
    dp.o_sb = d.out_stride[0], dp.o_sh = d.out_stride[1], dp.o_sn = d.out_stride[2];
    dp.delta = delta;
    dp.rows = d.B * d.H * d.Nq;
    dp.H = int(d.H), dp.Nq = int(d.Nq);
    const int64_t blocks = ceil_div(dp.rows * (D / 8), 256);
    if (blocks > kMaxI32) return PBA_ERR_INVALID_ARG;
    pba::pba_cross_delta_kernel<D><<<unsigned(blocks), 256, 0, stream>>>(dp);
    if (cudaGetLastError() != cudaSuccess) return PBA_ERR_CUDA;
  }
  p.q_tiles = int(q_tiles), p.k_tiles = int(k_tiles);
  p.units_a = int(grid_a), p.units_b = int(grid_b);
  // a unit of kind B passes over the queries of a group with four products a
  // step, one of kind A over the keys with three
  p.b_first = 4 * p.group * q_tiles >= 3 * k_tiles;
  if (grid_a + grid_b == 0) return PBA_OK;
  return launch_cross_bwd<D>(p, grid_a + grid_b, stream) == cudaSuccess ? PBA_OK : PBA_ERR_CUDA;
}

}  // namespace

extern "C" {

pba_status pba_cross_attn_forward(const pba_cross_desc *desc, const void *q, const void *k, const void *v,
                                  const int32_t *k_len, const uint8_t *key_mask, void *out, float *lse,
                                  void *stream_ptr) {
  pba_status s = check_cross(desc);
  if (s != PBA_OK) return s;
  const pba_cross_desc &d = *desc;
  if (d.Nq == 0) return PBA_OK;  // nothing to write
  s = check_cross_inputs(d, q, k, v, k_len);
  if (s != PBA_OK) return s;
  if (out == nullptr || !aligned16(out) || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0 ||
      !rows_ok(d.out_stride, d.B, d.H, d.Nq) || !rows_apart(d.out_stride, d.B, d.H, d.Nq) ||
      (lse != nullptr && !rows_apart(d.lse_stride, d.B, d.H, d.Nq)))
    return PBA_ERR_INVALID_ARG;
  s = check_device();
  if (s != PBA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream_ptr);
  return d.D == 32   ? run_forward<32>(d, q, k, v, k_len, key_mask, out, lse, st)
         : d.D == 64 ? run_forward<64>(d, q, k, v, k_len, key_mask, out, lse, st)
                     : run_forward<128>(d, q, k, v, k_len, key_mask, out, lse, st);
}

pba_status pba_cross_attn_backward(const pba_cross_desc *desc, const void *q, const void *k, const void *v,
                                   const int32_t *k_len, const uint8_t *key_mask, const void *out, const float *lse,
                                   const void *dout, void *dq, void *dk, void *dv, float *delta, void *stream_ptr) {
  pba_status s = check_cross(desc);
  if (s != PBA_OK) return s;
  const pba_cross_desc &d = *desc;
  s = check_cross_inputs(d, q, k, v, k_len);
  if (s != PBA_OK) return s;
  if (d.Nq > 0 && (out == nullptr || lse == nullptr || dout == nullptr || dq == nullptr || delta == nullptr))
    return PBA_ERR_INVALID_ARG;
  if (d.Nk > 0 && (dk == nullptr || dv == nullptr)) return PBA_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) != 0 || (reinterpret_cast<uintptr_t>(delta) & 3u) != 0)
    return PBA_ERR_INVALID_ARG;
  if (!rows_ok(d.out_stride, d.B, d.H, d.Nq) || !strides_ok(d.dout_stride, d.B, d.H, d.Nq)) return PBA_ERR_INVALID_ARG;
  s = check_device();
  if (s != PBA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream_ptr);
  return d.D == 32   ? run_cross_bwd<32>(d, q, k, v, out, lse, dout, k_len, key_mask, dq, dk, dv, delta, st)
         : d.D == 64 ? run_cross_bwd<64>(d, q, k, v, out, lse, dout, k_len, key_mask, dq, dk, dv, delta, st)
                     : run_cross_bwd<128>(d, q, k, v, out, lse, dout, k_len, key_mask, dq, dk, dv, delta, st);
}

}  // extern "C"
