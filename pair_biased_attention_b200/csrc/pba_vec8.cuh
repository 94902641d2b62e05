// pba_vec8.cuh -- eight elements of a bf16 or fp32 row as fp32 registers, the unit
// of work of the relative position kernels, with their stores and their rings
// of asynchronous copies; the element types and the 16-byte store are the block
// norms' too.
#pragma once

#include <cstdint>

#include "pba_ptx_more.cuh"

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

// A 16-byte store that leaves L1 alone: rows that one launch writes once.
__device__ __forceinline__ void st_stream16(void *p, uint4 v) {
  asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// Eight elements of a row, p[0], p[step], p[2 step], ..., of which the first n
// (0 to 8) exist; the others read as 0 and are not written.  Neighbouring
// threads take neighbouring elements, which keeps accesses coalesced on rows
// that start anywhere.
template <typename T>
__device__ __forceinline__ void load8(const typename T::Word *p, int n, int step, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = e < n ? T::to_f32(p[e * step]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store8(typename T::Word *p, int n, int step, const float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) p[e * step] = T::from_f32(x[e]);
}
// Eight consecutive bf16 on a 16-byte boundary as one word; a shorter eight
// element by element, so that it never touches what lies behind it.
__device__ __forceinline__ void store8_word(uint16_t *p, int n, const float (&x)[8]) {
  if (n >= 8)
    st_stream16(p, make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                              pack_bf16x2(x[6], x[7])));
  else
    store8<Bf16>(p, n, 1, x);
}

// Eight consecutive elements as they lie in memory: packed bf16 pairs, or fp32.
template <typename T>
struct Raw8 {
  static constexpr int kWords = int(sizeof(typename T::Word)) * 2;
  uint32_t w[kWords];
  __device__ __forceinline__ float2 pair(int i) const {
    return kWords == 4 ? make_float2(bf16lo_to_f32(w[i]), bf16hi_to_f32(w[i]))
                       : make_float2(__uint_as_float(w[(2 * i) % kWords]), __uint_as_float(w[(2 * i + 1) % kWords]));
  }
};

// Asynchronous copies of p[0 .. 8), the first n of them, into this thread's
// slot of a shared-memory ring: 16-byte words `stride` bytes apart.  kVec: p is
// 16-byte aligned and a short eight is filled up with zeros, reading nothing
// behind it.  Otherwise the slot has a word more: with `inner` (at least eight
// elements of the same row on either side) the aligned words around p are
// copied, for Raw8 to be shifted out of them; without, at a row's ends, the
// elements are put in place one by one.
template <typename T, bool kVec>
struct Ring8 {
  static constexpr int kData = Raw8<T>::kWords / 4;             // 16-byte words of eight elements
  static constexpr int kSlotWords = kVec ? kData : kData + 1;
  static __device__ __forceinline__ void fetch(uint8_t *slot, int stride, const typename T::Word *p, int n,
                                               bool inner) {
    constexpr int kSize = int(sizeof(typename T::Word));
    if (kVec) {
#pragma unroll
      for (int i = 0; i < kData; ++i) {
        const int bytes = min(16, max(0, n * kSize - 16 * i));
        // a word without any element: the address of one that has some
        cp_async16_part(slot + i * stride, reinterpret_cast<const uint8_t *>(p) + (bytes > 0 ? 16 * i : 0), bytes);
      }
    } else if (inner) {
      const uint8_t *base = reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15));
#pragma unroll
      for (int i = 0; i < kSlotWords; ++i) cp_async16(slot + i * stride, base + 16 * i);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        using W = typename T::Word;
        W *to = reinterpret_cast<W *>(slot + (e * kSize / 16) * stride) + e % (16 / kSize);
        *to = e < n ? p[e] : W(0);
      }
    }
  }
  // `p` as in the fetch: its place inside its aligned word
  static __device__ __forceinline__ Raw8<T> take(const uint8_t *slot, int stride, const typename T::Word *p,
                                                 bool inner) {
    constexpr int kW = Raw8<T>::kWords;
    uint32_t w[kSlotWords * 4];
#pragma unroll
    for (int i = 0; i < kSlotWords; ++i) {
      const uint4 v = *reinterpret_cast<const uint4 *>(slot + i * stride);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
    Raw8<T> x;
    if (kVec) {
#pragma unroll
      for (int i = 0; i < kW; ++i) x.w[i] = w[i];
    } else {
      const int off = inner ? int(reinterpret_cast<uintptr_t>(p) & 15) : 0;
      // by two words, by one, by half a word
#pragma unroll
      for (int i = 0; i < kW + 2; ++i) w[i] = (off & 8) ? w[(i + 2) % (kSlotWords * 4)] : w[i];
#pragma unroll
      for (int i = 0; i < kW + 1; ++i) w[i] = (off & 4) ? w[i + 1] : w[i];
#pragma unroll
      for (int i = 0; i < kW; ++i) x.w[i] = kW == 4 ? __funnelshift_r(w[i], w[i + 1], (off & 2) * 8) : w[i];
    }
    return x;
  }
};

}  // namespace pba
