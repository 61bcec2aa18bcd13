// Device helpers that the tiled products share: loads to LDS, the bare barrier, the order of the tiles, runs of outputs and
// channel constants, the gate.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "vq_device.h"
#include "vq_q8_device.h"

namespace vqt {

// g / (1 + exp(-g)) to about 3 ulp.  exp(-g) = 2^h (1 + l ln 2), where h is -g log2(e) rounded and l what the rounding
// left (log2(e) itself in two parts): the hardware's 2^h alone would lose an ulp for every unit of |h|, and those
// decide which way a hidden value's 8-bit rounding falls.  Past +-200 the sigmoid is 0 or 1 in fp32, and infinities stay
// out of the remainder; a NaN comes back through the last product.
__device__ __forceinline__ float silu(float g) {
  constexpr float kL = 0x1.715476p+0f, kLow = 0x1.4ae0c0p-26f, kLn2 = 0x1.62e430p-1f;  // log2(e) = kL + kLow
  const float c = -__builtin_amdgcn_fmed3f(g, -200.0f, 200.0f);
  const float h = c * kL;
  const float l = __builtin_fmaf(c, kLow, __builtin_fmaf(c, kL, -h));
  const float e = __builtin_amdgcn_exp2f(h) * __builtin_fmaf(l, kLn2, 1.0f);
  return g * __builtin_amdgcn_rcpf(1.0f + e);
}

// Stores CNT consecutive outputs of one row from column n on (those below n_end), as one block where it is whole.
template <int CNT>
__device__ __forceinline__ void store_run(void* y, vq_dtype t, int64_t row_at, int32_t n, int32_t n_end,
                                          const float (&v)[CNT]) {
  if (n >= n_end) return;
  if (n + CNT <= n_end) {
    if (t == VQ_F32) {
      __builtin_memcpy((float*)y + row_at + n, v, 4 * CNT);
    } else {
      uint16_t h[CNT];
      vqd::narrow<CNT>(v, t, h);
      __builtin_memcpy((uint16_t*)y + row_at + n, h, 2 * CNT);
    }
  } else {
#pragma unroll
    for (int k = 0; k < CNT; ++k)
      if (n + k < n_end) vqd::store_out(y, (size_t)(row_at + n + k), v[k], t);
  }
}
// CNT consecutive channel scales (and biases) from channel n on; zeros past n_end.
template <int CNT>
__device__ __forceinline__ void load_run(const float* p, int32_t n, int32_t n_end, float (&v)[CNT]) {
  if (n + CNT <= n_end) {
    __builtin_memcpy(v, p + n, 4 * CNT);
  } else {
#pragma unroll
    for (int k = 0; k < CNT; ++k) v[k] = n + k < n_end ? p[n + k] : 0.f;
  }
}
template <int CNT>
__device__ __forceinline__ void load_bias(const uint16_t* p, int32_t n, int32_t n_end, float (&v)[CNT]) {
#pragma unroll
  for (int k = 0; k < CNT; ++k) v[k] = p && n + k < n_end ? vqd::f16_to_f32(p[n + k]) : 0.f;
}

// Copies 16 bytes per lane from `g` to LDS at the wavefront's `l` + 16 lane, past the registers.
__device__ __forceinline__ void to_lds(const uint8_t* g, uint8_t* l) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                   (__attribute__((address_space(3))) void*)l, 16, 0, 0);
}

// The workgroup's barrier alone.  __syncthreads() would also wait for every load to LDS that is still on its way; here
// each wavefront has waited for those that the others need, and for its own reads, and no memory operation moves across.
// 64 x 8192 x 8192 (64 x 32 tiles): 30 us with __syncthreads(), 21 us; 128 x 28672 x 8192 (128 x 128): 72 and 58 us.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// Order of the tiles: 8 row tiles by all columns, columns slowest.
__device__ __forceinline__ void tile_at(int32_t at, int32_t mt_count, int32_t nt, int32_t& mt, int32_t& nti) {
  const int32_t band = at / (8 * nt), in_band = at - band * 8 * nt;
  const int32_t band_rows = min(8, mt_count - band * 8);
  mt = band * 8 + in_band % band_rows;
  nti = in_band / band_rows;
}
// The tile of workgroup `id`: those of one XCD (id mod 8) are neighbours in that order.  false: no such tile.
__device__ __forceinline__ bool place(int32_t id, int32_t total, int32_t mt_count, int32_t nt, int32_t& mt, int32_t& nti) {
  const int32_t per = (total + 7) / 8;
  const int32_t at = (id & 7) * per + (id >> 3);
  if ((id >> 3) >= per || at >= total) return false;
  tile_at(at, mt_count, nt, mt, nti);
  return true;
}

}  // namespace vqt
