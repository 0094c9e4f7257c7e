// mxfp4_rows8.h -- 8 consecutive elements of a row at any alignment, as fp32
// values and back, for the kernels that move rows.
#pragma once

#include "mxfp4_device.h"

namespace mxfp4 {

__device__ __forceinline__ uint16_t f32_to_bf16_rne(float f) {
  uint32_t u = __builtin_bit_cast(uint32_t, f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);  // quiet NaN
  u += 0x7FFFu + ((u >> 16) & 1u);
  return (uint16_t)(u >> 16);
}

// Two values rounded to bf16 (nearest even) by the hardware conversion, a in
// the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// Rows of any length start at any element: 16-byte accesses with the
// element's alignment (the hardware takes unaligned global accesses).
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

template <int DT>
struct Row8 {  // 8 consecutive elements of a row
  static constexpr int ES = DT == kBF16 ? 2 : 4, NW = 2 * ES;
};

template <int DT>
__device__ __forceinline__ void load8(uint32_t (&w)[Row8<DT>::NW], const uint8_t *p, int n) {
  if (n >= 8) {
#pragma unroll
    for (int q = 0; q < Row8<DT>::NW / 4; ++q) {
      const u32x4 v = *reinterpret_cast<const u32x4_a2 *>(p + 16 * q);
      w[4 * q] = v.x; w[4 * q + 1] = v.y; w[4 * q + 2] = v.z; w[4 * q + 3] = v.w;
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < Row8<DT>::NW; ++q) w[q] = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) {
      if (DT == kBF16) w[j >> 1] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[j] << (16 * (j & 1));
      else w[j % Row8<DT>::NW] = reinterpret_cast<const uint32_t *>(p)[j];
    }
}

template <int DT>
__device__ __forceinline__ void store8(uint8_t *p, const uint32_t (&w)[Row8<DT>::NW], int n) {
  if (n >= 8) {
#pragma unroll
    for (int q = 0; q < Row8<DT>::NW / 4; ++q) {
      const u32x4 v = {w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]};
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a2 *>(p + 16 * q));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) {
      if (DT == kBF16) reinterpret_cast<uint16_t *>(p)[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
      else reinterpret_cast<uint32_t *>(p)[j] = w[j % Row8<DT>::NW];
    }
}

template <int DT>
__device__ __forceinline__ float elem(const uint32_t (&w)[Row8<DT>::NW], int j) {
  if (DT == kBF16) return bits_f32(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
  return bits_f32(w[j % Row8<DT>::NW]);
}

template <int DT>
__device__ __forceinline__ void pack8(uint32_t (&w)[Row8<DT>::NW], const float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < Row8<DT>::NW; ++j)
    w[j] = DT == kBF16 ? pack_bf16(f[(2 * j) % 8], f[(2 * j + 1) % 8])
                       : __builtin_bit_cast(uint32_t, f[j % 8]);
}

}  // namespace mxfp4
