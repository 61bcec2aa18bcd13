// Device helpers of the 8-bit operators: the row scale and the rounding to 8 bits.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "vq_device.h"

namespace vqd {

// fp32 -> 16-bit type `t`, rounded to nearest even by the hardware conversions (bf16: two values per instruction).
template <int CNT>
__device__ __forceinline__ void narrow(const float (&f)[CNT], vq_dtype t, uint16_t (&v)[CNT]) {
  if (t == VQ_F16) {
#pragma unroll
    for (int k = 0; k < CNT; ++k) v[k] = f32_to_f16_rne(f[k]);
  } else {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int k = 0; k < CNT; k += 2) {
      const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{f[k], f[k + 1]}), b2));
      v[k] = (uint16_t)w;
      v[k + 1] = (uint16_t)(w >> 16);
    }
  }
}

__device__ __forceinline__ uint32_t abs_bits(float f) { return __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu; }

// The scale of a row whose largest |x| has the bits `big` (the bits of non-negative floats order like the floats, and
// NaN above infinity, so the row maximum is an integer maximum): s = max|x| / 127, and what its quotients need.
struct Q8Scale {
  float s;      // stored: 0 for a zero row, NaN for a row with an infinity or a NaN (its q are zero)
  float up;     // power of two that takes a tiny s, and with it x, clear of the subnormals
  float den;    // s * up
  float rcp;    // 1 / den, rounded to nearest; 0 where every q is zero
};
__device__ __forceinline__ Q8Scale q8_scale(uint32_t big) {
  Q8Scale r;
  if (big >= 0x7F800000u) return Q8Scale{__builtin_nanf(""), 0.f, 1.f, 0.f};
  r.s = __builtin_bit_cast(float, big) / 127.0f;
  r.up = r.s < 0x1p-40f ? 0x1p80f : 1.0f;
  r.den = r.s * r.up;
  r.rcp = r.den > 0.f ? 1.0f / r.den : 0.f;
  if (!(r.den > 0.f)) r.den = 1.0f;
  return r;
}

// x / s rounded to fp32 and then to the nearest integer, ties to even, within +-127.  The quotient is the correctly
// rounded one at three instructions (Markstein's division: with rcp = 1 / den correctly rounded and t = x rcp within an
// ulp, t + (x - t den) rcp in two fused steps rounds to x / den): what is a tie after the division stays one.
// rcp = 0 gives 0 for every finite x; a row with a non-finite value has up = 0 as well.
__device__ __forceinline__ int q8_value(float x, const Q8Scale& c) {
  if (c.up == 0.f) return 0;
  const float a = x * c.up;
  const float t = a * c.rcp;
  const float e = __builtin_fmaf(-t, c.den, a);
  const float v = __builtin_rintf(__builtin_fmaf(e, c.rcp, t));
  return (int)__builtin_fminf(__builtin_fmaxf(v, -127.0f), 127.0f);
}

}  // namespace vqd
