// Device helpers of the 8-bit float layers: the block scale and the rounding to e4m3.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "vq_device.h"
#include "vq_q8_device.h"

namespace vqd {

// The value of another lane of the 16-lane row, without LDS.  Where all lanes of a group of 2, 4 and 8 already hold the same,
// kXor1, kXor2, kHalf and kRow one after the other bring in the rest of 2, 4, 8 and 16 consecutive lanes.
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalf = 0x141, kRow = 0x140;
template <int CTRL>
__device__ __forceinline__ uint32_t other(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
// The largest of 8 (16) consecutive lanes.
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  static_assert(LANES == 8 || LANES == 16, "half a row or a row");
  v = max(v, other<kXor1>(v));
  v = max(v, other<kXor2>(v));
  v = max(v, other<kHalf>(v));
  if constexpr (LANES == 16) v = max(v, other<kRow>(v));
  return v;
}

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

// Elements at .. at + CNT - 1 of a row of `end` elements, as they are; zeros from its end on.  Nothing outside the row is
// read: where it ends inside, every word is loaded from no further than its last two elements (one for fp32), all of them
// together, and shifted or cleared afterwards.
template <vq_dtype XT, int CNT>
struct Run {
  uint32_t v[CNT * (XT == VQ_F32 ? 4 : 2) / 4];
};
template <vq_dtype XT, int CNT>
__device__ __forceinline__ Run<XT, CNT> load_run(const void* row, int32_t at, int32_t end) {
  constexpr int es = XT == VQ_F32 ? 4 : 2, per = 4 / es;  // elements of a word
  Run<XT, CNT> r;
  if (at + CNT <= end) {
    __builtin_memcpy(r.v, (const char*)row + (int64_t)at * es, CNT * es);
  } else if (end >= per) {
#pragma unroll
    for (int k = 0; k < CNT / per; ++k)
      __builtin_memcpy(&r.v[k], (const char*)row + (int64_t)min(at + k * per, end - per) * es, 4);
#pragma unroll
    for (int k = 0; k < CNT / per; ++k) {
      const int32_t e = at + k * per;
      if (per == 2 && e == end - 1) r.v[k] >>= 16;
      if (e >= end) r.v[k] = 0;
    }
  } else {  // a single 16-bit element
#pragma unroll
    for (int k = 0; k < CNT / per; ++k) r.v[k] = 0;
    if (at == 0 && end > 0) r.v[0] = *(const uint16_t*)row;
  }
  return r;
}
template <vq_dtype XT, int CNT>
__device__ __forceinline__ void widen(const Run<XT, CNT>& r, float (&f)[CNT]) {
#pragma unroll
  for (int k = 0; k < CNT; ++k) {
    if constexpr (XT == VQ_F32) {
      f[k] = __builtin_bit_cast(float, r.v[k]);
    } else {
      f[k] = x_to_f32<XT == VQ_F16 ? 0 : 1>(r.v[k / 2] >> (16 * (k & 1)));
    }
  }
}

}  // namespace vqd
