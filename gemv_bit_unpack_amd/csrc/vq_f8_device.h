// Device helpers of the 8-bit float layers: the block scale and the rounding to e4m3.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "vq_device.h"
#include "vq_q8_device.h"

namespace vqd {

constexpr float kF8Top = 448.0f;  // the largest e4m3 value

// The scale of a block whose largest |x| has the bits `big`: s = max|x| / 448, and what its quotients need (as Q8Scale
// does for rows in 8-bit integers: s = 0 for a zero block, NaN for one with an infinity or a NaN, whose values are zero).
__device__ __forceinline__ Q8Scale f8_scale(uint32_t big) {
  Q8Scale r;
  if (big >= 0x7F800000u) return Q8Scale{__builtin_nanf(""), 0.f, 1.f, 0.f};
  r.s = __builtin_bit_cast(float, big) / kF8Top;
  r.up = r.s < 0x1p-40f ? 0x1p80f : 1.0f;
  r.den = r.s * r.up;
  r.rcp = r.den > 0.f ? 1.0f / r.den : 0.f;
  if (!(r.den > 0.f)) r.den = 1.0f;
  return r;
}

// x / s rounded to fp32 (Markstein's division, as in q8_value), within +-448.
__device__ __forceinline__ float f8_quotient(float x, const Q8Scale& c) {
  const float a = x * c.up;
  const float t = a * c.rcp;
  const float e = __builtin_fmaf(-t, c.den, a);
  return __builtin_amdgcn_fmed3f(__builtin_fmaf(e, c.rcp, t), -kF8Top, kF8Top);
}

// 4 values as e4m3, rounded to nearest even by the hardware's conversion.
__device__ __forceinline__ uint32_t f8_pack4(const float* f, const Q8Scale& c) {
  if (c.up == 0.f) return 0;
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(f8_quotient(f[0], c), f8_quotient(f[1], c), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(f8_quotient(f[2], c), f8_quotient(f[3], c), w, true);
  return (uint32_t)w;
}

// Elements at .. at + CNT - 1 of a row that ends before element `end`, as fp32; zeros from there on.
template <vq_dtype XT, int CNT>
__device__ __forceinline__ void load_f32(const void* row, int32_t at, int32_t end, float (&f)[CNT]) {
  constexpr int es = XT == VQ_F32 ? 4 : 2;
  const char* p = (const char*)row + (int64_t)at * es;
  if (at + CNT <= end) {
    uint32_t v[CNT * es / 4];
    __builtin_memcpy(v, p, CNT * es);
#pragma unroll
    for (int k = 0; k < CNT; ++k) {
      if constexpr (XT == VQ_F32) {
        f[k] = __builtin_bit_cast(float, v[k]);
      } else {
        f[k] = x_to_f32<XT == VQ_F16 ? 0 : 1>(v[k / 2] >> (16 * (k & 1)));
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < CNT; ++k) {
      f[k] = 0.f;
      if (at + k < end) {
        if constexpr (XT == VQ_F32) {
          f[k] = ((const float*)p)[k];
        } else {
          f[k] = x_to_f32<XT == VQ_F16 ? 0 : 1>(((const uint16_t*)p)[k]);
        }
      }
    }
  }
}

}  // namespace vqd
