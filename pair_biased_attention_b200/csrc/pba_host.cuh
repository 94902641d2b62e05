// pba_host.cuh -- what the library's host code shares: device checks, Tensor
// Memory Accelerator descriptors, one-time kernel set-up per device, the
// device error word and the wait limit.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "pba.h"

namespace pba_host {

// The device error word of the current device, and the limit of the kernels'
// waits (both defined in pba_api.cu).
int *device_error_word();
uint64_t wait_timeout_ns();

using EncodeTiledFn = PFN_cuTensorMapEncodeTiled_v12000;

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// One-time per-device kernel set-up (the dynamic shared memory limit is a
// per-device attribute of a kernel): `setup` runs once for each device it is
// called on, with that device current, and its result is kept per device.
constexpr int kMaxDevices = 64;
struct PerDeviceOnce {
  std::once_flag flag[kMaxDevices];
  cudaError_t err[kMaxDevices] = {};
};
template <typename F>
cudaError_t once_per_device(PerDeviceOnce &o, F &&setup) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::call_once(o.flag[dev], [&] { o.err[dev] = setup(); });
  return o.err[dev];
}

constexpr int64_t kMaxI32 = 2147483647;

// 4-D tiled tensor map of bf16 (or, with f32, fp32) elements.  dims/strides
// innermost first; strides in bytes for dims 1..3.  A dim of extent 1 gets a
// harmless positive stride (its coordinate is always 0).
inline bool make_map(CUtensorMap *map, const void *base, const uint64_t dims[4], const int64_t strides_bytes[3],
              const uint32_t box[4], CUtensorMapSwizzle swizzle, bool f32 = false) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t gdim[4] = {dims[0], dims[1], dims[2], dims[3]};
  cuuint64_t gstride[3];
  int64_t prev_extent = int64_t(dims[0]) * (f32 ? 4 : 2);
  for (int i = 0; i < 3; ++i) {
    int64_t s = strides_bytes[i];
    if (dims[i + 1] == 1 || s <= 0) s = (prev_extent + 15) / 16 * 16;
    gstride[i] = cuuint64_t(s);
    prev_extent = s * int64_t(dims[i + 1]);
  }
  cuuint32_t bdim[4] = {box[0], box[1], box[2], box[3]};
  cuuint32_t estride[4] = {1, 1, 1, 1};
  CUresult r = enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                   const_cast<void *>(base), gdim, gstride, bdim, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

inline bool stride_ok_bf16(int64_t s, int64_t extent) { return extent <= 1 || (s > 0 && s % 8 == 0); }
inline bool stride_ok_f32(int64_t s, int64_t extent) { return extent <= 1 || (s > 0 && s % 4 == 0); }

// An output's (b, h, row) strides: 0 on an axis longer than 1 would write several
// rows to one place.
inline bool rows_apart(const int64_t s[3], int64_t B, int64_t H, int64_t N) {
  return (B <= 1 || s[0] != 0) && (H <= 1 || s[1] != 0) && (N <= 1 || s[2] != 0);
}

// Whether the current device is one that the kernels were built for (sm_100a).
inline pba_status check_device() {
  static PerDeviceOnce once;
  static bool fits[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PBA_ERR_CUDA;
  if (dev >= kMaxDevices) return PBA_ERR_UNSUPPORTED;
  const cudaError_t e = once_per_device(once, [&] {
    int major = 0, minor = 0;
    cudaError_t r = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (r == cudaSuccess) r = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    fits[dev] = major == 10 && minor == 0;
    return r;
  });
  if (e != cudaSuccess) return PBA_ERR_CUDA;
  return fits[dev] ? PBA_OK : PBA_ERR_UNSUPPORTED;
}

inline int sm_count() {  // of the current device; 0 when it cannot be had
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

}  // namespace pba_host
