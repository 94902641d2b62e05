// pba_vec8.cuh -- eight consecutive elements of a bf16 or fp32 row as fp32
// registers: the unit of work of the elementwise kernels (relative position
// bias, block norms).  16-byte accesses when the caller knows the row to be
// aligned, element by element otherwise and at a ragged row end.
#pragma once

#include <cstdint>

#include "pba_ptx.cuh"

namespace pba {

struct Bf16 {  // tag of a bf16 tensor, held as raw 16-bit words
  using Word = uint16_t;
  static __device__ __forceinline__ float to_f32(uint16_t w) { return __uint_as_float(uint32_t(w) << 16); }
  static __device__ __forceinline__ uint16_t from_f32(float x) { return uint16_t(pack_bf16x2(x, 0.f)); }
};
struct F32 {
  using Word = float;
  static __device__ __forceinline__ float to_f32(float w) { return w; }
  static __device__ __forceinline__ float from_f32(float x) { return x; }
};

// 16-byte global accesses marked for first eviction: rows that one launch
// touches once.
__device__ __forceinline__ uint4 ld_stream16(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void st_stream16(void *p, uint4 v) {
  asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

__device__ __forceinline__ void unpack8(const uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = bf16lo_to_f32(w[e]);
    x[2 * e + 1] = bf16hi_to_f32(w[e]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Elements at p[0 .. 8), of which the first n (0 to 8) exist; the others read
// as 0 and are not written.  kVec: p is 16-byte aligned, so whole chunks move
// as 16-byte words.  A chunk cut short never touches what lies behind it.
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const typename T::Word *p, int n, float (&x)[8]) {
  if (kVec && n >= 8) {
    if (sizeof(typename T::Word) == 2) {
      unpack8(ld_stream16(p), x);
    } else {
      const uint4 a = ld_stream16(p), b = ld_stream16(p + 4);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(w[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = e < n ? T::to_f32(p[e]) : 0.f;
  }
}

template <typename T, bool kVec>
__device__ __forceinline__ void store8(typename T::Word *p, int n, const float (&x)[8]) {
  if (kVec && n >= 8) {
    if (sizeof(typename T::Word) == 2) {
      st_stream16(p, pack8(x));
    } else {
      st_stream16(p, make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                                __float_as_uint(x[3])));
      st_stream16(p + 4, make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]),
                                    __float_as_uint(x[7])));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = T::from_f32(x[e]);
  }
}

}  // namespace pba
