// vq_block_norm and vq_q8_quantize: one pass over the rows between two quantized layers.
//
//   u = N_post(z)                     z: what the block before wrote
//   r = res_scale * h + gate_scale * gate * u
//   x = N_pre(r)                      what the next block reads
//   q, s = 8-bit form of x (or x itself in x_dtype)
//
// with N(a) = (a - mean) / sqrt(mean((a - mean)^2) + eps) * (w_offset + w) + b; the RMS form has no mean, "none" is the
// identity.  The quantizer alone is the same kernel with z = x and both norms off.
//
// A row is held in registers from its one load to its one store: C chunks of 8 elements per thread (chunk c of thread t
// is elements 8 (c TPR + t) ..), fp32 from the first widening on, so the statistics of both norms, the residual add and
// the row's largest value cost no second read.  Everything is rounded once, at the store.  The variance is taken about
// the mean in a second sweep over the registers: no cancellation.  TPR threads share a row: 64 (four rows per workgroup,
// no barrier), 256 or 1024.
//
// Bound: the bytes of z, h, r and x once each.  Chunks go as 16-byte accesses also at odd row lengths (the hardware
// takes any alignment); only the row's last, partial chunk is taken element by element.
#include "vq_device.h"
#include "vq_q8_device.h"

namespace {

using vqi::NormArgs;

constexpr int kChunk = 8;


__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 r;
  __builtin_memcpy(&r, p, 16);
  return r;
}

// Chunk `at` (elements at .. at + 7) of a row of `d` elements, as raw bits: 16-bit types in lo, fp32 in lo and hi.
// Elements past the row's end read as zero.
__device__ __forceinline__ void load_chunk(const void* row, vq_dtype t, int at, int d, uint4& lo, uint4& hi) {
  lo = make_uint4(0, 0, 0, 0);
  hi = lo;
  if (at >= d) return;
  if (t == VQ_F32) {
    const float* p = (const float*)row + at;
    if (at + kChunk <= d) {
      lo = load16(p);
      hi = load16(p + 4);
    } else {
      uint32_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = at + k < d ? __builtin_bit_cast(uint32_t, p[k]) : 0u;
      lo = make_uint4(v[0], v[1], v[2], v[3]);
      hi = make_uint4(v[4], v[5], v[6], v[7]);
    }
  } else {
    const uint16_t* p = (const uint16_t*)row + at;
    if (at + kChunk <= d) {
      lo = load16(p);
    } else {
      uint32_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = at + k < d ? p[k] : 0u;
      lo = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
  }
}

__device__ __forceinline__ void widen(const uint4& lo, const uint4& hi, vq_dtype t, float (&f)[8]) {
  const uint32_t w[4] = {lo.x, lo.y, lo.z, lo.w};
  if (t == VQ_F32) {
    const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[k] = __builtin_bit_cast(float, w[k]);
      f[4 + k] = __builtin_bit_cast(float, h[k]);
    }
  } else if (t == VQ_F16) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = vqd::f16_to_f32(w[k] & 0xFFFFu);
      f[2 * k + 1] = vqd::f16_to_f32(w[k] >> 16);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __builtin_bit_cast(float, w[k] << 16);
      f[2 * k + 1] = __builtin_bit_cast(float, w[k] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ void store_chunk(void* row, vq_dtype t, int at, int d, const float (&f)[8]) {
  if (at >= d) return;
  if (t == VQ_F32) {
    float* p = (float*)row + at;
    if (at + kChunk <= d) {
      __builtin_memcpy(p, f, 32);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (at + k < d) p[k] = f[k];
    }
  } else {
    uint16_t v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = t == VQ_F16 ? vqd::f32_to_f16_rne(f[k]) : vqd::f32_to_bf16_rne(f[k]);
    uint16_t* p = (uint16_t*)row + at;
    if (at + kChunk <= d) {
      __builtin_memcpy(p, v, 16);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (at + k < d) p[k] = v[k];
    }
  }
}

// Sum (or maximum of bits) over the TPR threads of a row, the same value in all of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (TPR > 64) {
    __syncthreads();  // the part array's last readers are done
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int k = 0; k < TPR / 64; ++k) v += part[k];
  }
  return v;
}
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float* part) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  if constexpr (TPR > 64) {
    uint32_t* up = (uint32_t*)part;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) up[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int k = 0; k < TPR / 64; ++k) v = max(v, up[k]);
  }
  return v;
}

// f := N(f) for the row's chunks held by this thread.
template <int TPR, int C>
__device__ __forceinline__ void normalize(float (&f)[C][8], int kind, const NormArgs& a, const void* w, const void* b,
                                          int t, float* part) {
  if (kind == VQ_NORM_NONE) return;
  const int d = a.dim;
  const float inv_d = 1.0f / (float)d;
  if (kind == VQ_NORM_LAYER) {
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += f[c][k];  // zeros past the end
    const float mean = row_sum<TPR>(sum, part) * inv_d;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) f[c][k] = (c * TPR + t) * kChunk + k < d ? f[c][k] - mean : 0.f;
  }
  float sq = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) sq = __builtin_fmaf(f[c][k], f[c][k], sq);
  const float inv = 1.0f / __builtin_sqrtf(row_sum<TPR>(sq, part) * inv_d + a.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int at = (c * TPR + t) * kChunk;
    uint4 lo, hi;
    float g[8];
    if (w) {
      load_chunk(w, a.w_dtype, at, d, lo, hi);
      widen(lo, hi, a.w_dtype, g);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) f[c][k] = w ? f[c][k] * inv * (a.w_offset + g[k]) : f[c][k] * inv;
    if (b) {
      load_chunk(b, a.w_dtype, at, d, lo, hi);
      widen(lo, hi, a.w_dtype, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[c][k] += g[k];
    }
  }
}

template <int TPR, int C>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(NormArgs a) {
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;  // rows per workgroup
  __shared__ float part[16];
  const int t = TPR < 256 ? threadIdx.x % TPR : threadIdx.x;
  const int64_t m = (int64_t)blockIdx.x * kRows + (TPR < 256 ? threadIdx.x / TPR : 0);
  if (m >= a.rows) return;  // whole wavefronts, and only where no barrier follows (kRows > 1)
  const int d = a.dim;

  constexpr bool kAhead = TPR * C <= 4096;  // longer rows have no registers to hold h early
  uint4 lo[kAhead ? C : 1], hi[kAhead ? C : 1];
  float f[C][8];
  const size_t ez = a.z_dtype == VQ_F32 ? 4 : 2;
  const char* z = (const char*)a.z + (size_t)m * (size_t)a.ldz * ez;
  if constexpr (kAhead) {
#pragma unroll
    for (int c = 0; c < C; ++c) load_chunk(z, a.z_dtype, (c * TPR + t) * kChunk, d, lo[c], hi[c]);
#pragma unroll
    for (int c = 0; c < C; ++c) widen(lo[c], hi[c], a.z_dtype, f[c]);
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      load_chunk(z, a.z_dtype, (c * TPR + t) * kChunk, d, lo[0], hi[0]);
      widen(lo[0], hi[0], a.z_dtype, f[c]);
    }
  }

  const size_t eh = a.h_dtype == VQ_F32 ? 4 : 2;
  const char* h = (const char*)a.h + (size_t)m * (size_t)a.ldh * eh;
  if (kAhead && a.h) {  // in flight while the statistics of z are taken
#pragma unroll
    for (int c = 0; c < C; ++c) load_chunk(h, a.h_dtype, (c * TPR + t) * kChunk, d, lo[kAhead ? c : 0], hi[kAhead ? c : 0]);
  }

  normalize<TPR, C>(f, a.post, a, a.post_w, a.post_b, t, part);

  if (a.gate) {
    const size_t eg = a.gate_dtype == VQ_F32 ? 4 : 2;
    const char* g = (const char*)a.gate + (size_t)(m / a.gate_rows) * (size_t)d * eg;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      uint4 gl, gh;
      float gf[8];
      load_chunk(g, a.gate_dtype, (c * TPR + t) * kChunk, d, gl, gh);
      widen(gl, gh, a.gate_dtype, gf);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[c][k] *= gf[k];
    }
  }
  if (a.combine) {  // r differs from u: a residual or a scale
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float hf[8];
      if (!kAhead && a.h) load_chunk(h, a.h_dtype, (c * TPR + t) * kChunk, d, lo[0], hi[0]);
      if (a.h) widen(lo[kAhead ? c : 0], hi[kAhead ? c : 0], a.h_dtype, hf);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        f[c][k] *= a.gate_scale;
        if (a.h) f[c][k] += a.res_scale * hf[k];
      }
    }
  }
  if (a.r) {
    char* r = (char*)a.r + (size_t)m * (size_t)d * eh;
#pragma unroll
    for (int c = 0; c < C; ++c) store_chunk(r, a.h_dtype, (c * TPR + t) * kChunk, d, f[c]);
  }
  if (!a.x && !a.q) return;

  normalize<TPR, C>(f, a.pre, a, a.pre_w, a.pre_b, t, part);

  if (a.x) {
    char* x = (char*)a.x + (size_t)m * (size_t)d * (a.x_dtype == VQ_F32 ? 4 : 2);
#pragma unroll
    for (int c = 0; c < C; ++c) store_chunk(x, a.x_dtype, (c * TPR + t) * kChunk, d, f[c]);
  }
  if (a.q) {
    uint32_t big = 0;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if ((c * TPR + t) * kChunk + k < d) big = max(big, vqd::abs_bits(f[c][k]));
    const vqd::Q8Scale sc = vqd::q8_scale(row_max<TPR>(big, part));
    const int64_t ldq = vqi::q8_row_bytes(d);
    uint8_t* q = a.q + (size_t)m * (size_t)ldq;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * TPR + t) * kChunk;
      if (at < ldq) {  // pad bytes past the row's end are written as zero
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (at + k < d) w[k >> 2] |= (uint32_t)(uint8_t)vqd::q8_value(f[c][k], sc) << (8 * (k & 3));
        *(uint2*)(q + at) = make_uint2(w[0], w[1]);
      }
    }
    if (t == 0) a.s[m] = sc.s;
  }
}

template <int TPR, int C>
vq_status launch(const NormArgs& a, hipStream_t stream) {
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
  constexpr int kWg = TPR < 256 ? 256 : TPR;
  const int64_t blocks = ((int64_t)a.rows + kRows - 1) / kRows;
  if (!vqi::grid_ok(blocks, kWg)) return VQ_ERR_SHAPE;
  norm_kernel<TPR, C><<<dim3((uint32_t)blocks), dim3(kWg), 0, stream>>>(a);
  return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP;
}

}  // namespace

namespace vqi {

vq_status launch_norm(const NormArgs& a, void* stream_) {
  hipStream_t stream = (hipStream_t)stream_;
  const int d = a.dim;
  if (d <= 512) return launch<64, 1>(a, stream);
  if (d <= 1024) return launch<64, 2>(a, stream);
  // few rows: one chunk per thread, for the shortest chain; many: more chunks per thread, so that more loads are in flight
  const bool few = a.rows <= 512;
  if (few && d > 2048) {
    if (d <= 8192) return launch<1024, 1>(a, stream);
    if (d <= 16384) return launch<1024, 2>(a, stream);
  }
  if (d <= 2048) return launch<256, 1>(a, stream);
  if (d <= 4096) return launch<256, 2>(a, stream);
  if (d <= 8192) return launch<256, 4>(a, stream);
  if (d <= 16384) return launch<256, 8>(a, stream);
  if (d <= 32768) return launch<1024, 4>(a, stream);
  return launch<1024, 8>(a, stream);  // up to kNormMaxDim
}

}  // namespace vqi
