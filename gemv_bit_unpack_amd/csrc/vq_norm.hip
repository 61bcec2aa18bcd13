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
// A row is held by its threads from its one load to its one store, fp32 from the first widening on: C chunks of 8
// elements per thread (chunk c of thread t is elements 8 (c T + t) .. for T threads), so the statistics of both norms,
// the residual add and the row's largest value cost no second read, and everything is rounded once, at the store.  The
// variance is taken about the mean in a second sweep over the registers: no cancellation.
// Up to 32768 elements the registers hold it.  Longer rows, 8 chunks for each of 1024 threads, need more than the 128
// registers that these have: the compiler keeps 180 to 356 bytes a thread in scratch memory, and a row costs four times
// as much as one half as long (both norms, gate and residual in bf16: 16 x 65536 68 us, 16 x 32768 15; 1024 rows 391 and
// 86; the quantizer alone, fp32, 1024 rows 108 and 43).
//
// Bound: the bytes of z, h, r and x once each; 8192 x 8192 in bf16 with everything on, 537 MB, takes 140 us (3.8 TB/s;
// the vector instructions, about 20 per element, are half of that).  With few rows time is the chain load - sum - sum -
// store: the weights, biases and the gate are then loaded before the first sum, with z and h.
// Chunks go as 16-byte accesses also at odd row lengths (the hardware takes any alignment); only the row's last,
// partial chunk is taken element by element.
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

// A chunk as raw bits: a 16-bit type in lo, fp32 (WIDE) in lo and hi.  Which of the two z and h are is fixed when the
// kernel is built: the registers of hi are the difference between 5 and 8 wavefronts per SIMD.
template <bool WIDE>
struct Raw {
  uint4 lo;
  uint4 hi[WIDE ? 1 : 0];
};
template <>
struct Raw<false> {
  uint4 lo;
};

// Elements at .. at + 7 of a row of `d` elements; those past the row's end read as zero.
template <bool WIDE>
__device__ __forceinline__ Raw<WIDE> load_chunk(const void* row, int at, int d) {
  Raw<WIDE> r;
  r.lo = make_uint4(0, 0, 0, 0);
  if constexpr (WIDE) r.hi[0] = r.lo;
  if (at >= d) return r;
  if constexpr (WIDE) {
    const float* p = (const float*)row + at;
    if (at + kChunk <= d) {
      r.lo = load16(p);
      r.hi[0] = load16(p + 4);
    } else {
      uint32_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = at + k < d ? __builtin_bit_cast(uint32_t, p[k]) : 0u;
      r.lo = make_uint4(v[0], v[1], v[2], v[3]);
      r.hi[0] = make_uint4(v[4], v[5], v[6], v[7]);
    }
  } else {
    const uint16_t* p = (const uint16_t*)row + at;
    if (at + kChunk <= d) {
      r.lo = load16(p);
    } else {
      uint32_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = at + k < d ? p[k] : 0u;
      r.lo = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
  }
  return r;
}

template <bool WIDE>
__device__ __forceinline__ void widen(const Raw<WIDE>& r, vq_dtype t, float (&f)[8]) {
  const uint32_t w[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w};
  if constexpr (WIDE) {
    const uint32_t h[4] = {r.hi[0].x, r.hi[0].y, r.hi[0].z, r.hi[0].w};
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

// The same for a vector whose type is known at run time.
__device__ __forceinline__ void load_any(const void* row, vq_dtype t, int at, int d, float (&f)[8]) {
  if (t == VQ_F32) {
    widen(load_chunk<true>(row, at, d), t, f);
  } else {
    widen(load_chunk<false>(row, at, d), t, f);
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
    vqd::narrow<8>(f, t, v);
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

// Sums over the threads of a row, the same value in all of them; `flip` alternates between two LDS arrays, so that one
// barrier per sum is enough (a wavefront can be one sum ahead of another, never two).  ONE: the row is a wavefront's own.
constexpr int kMaxWaves = 16;
template <bool ONE>
struct RowReduce {
  float (*part)[kMaxWaves];
  int flip = 0;

  __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o, 64);
    if constexpr (!ONE) {
      if ((threadIdx.x & 63) == 0) part[flip][threadIdx.x >> 6] = v;
      __syncthreads();
      const int waves = blockDim.x >> 6;
      v = 0.f;
      for (int k = 0; k < waves; ++k) v += part[flip][k];
      flip ^= 1;
    }
    return v;
  }
  __device__ __forceinline__ uint32_t max_bits(uint32_t v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
    if constexpr (!ONE) {
      if ((threadIdx.x & 63) == 0) part[flip][threadIdx.x >> 6] = __builtin_bit_cast(float, v);
      __syncthreads();
      const int waves = blockDim.x >> 6;
      for (int k = 0; k < waves; ++k) v = max(v, __builtin_bit_cast(uint32_t, part[flip][k]));
      flip ^= 1;
    }
    return v;
  }
};

// A vector beside the row (norm weight, bias, gate row), this thread's chunks of it: loaded ahead of the first sum, or
// chunk by chunk when it is used, which leaves registers for more wavefronts.
template <int C, bool AHEAD>
struct Shared {
  const void* p;
  vq_dtype t;
  float ahead[AHEAD ? C : 1][8];
  __device__ __forceinline__ void fetch(const void* p_, vq_dtype t_, int at, int step, int d) {
    p = p_;
    t = t_;
    if constexpr (AHEAD) {
      if (p)
#pragma unroll
        for (int c = 0; c < C; ++c) load_any(p, t, at + c * step, d, ahead[c]);
    }
  }
  __device__ __forceinline__ void get(int c, int at, int d, float (&f)[8]) const {
    if constexpr (AHEAD) {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = ahead[c][k];
    } else {
      load_any(p, t, at, d, f);
    }
  }
};

// f := N(f) for the chunks held by this thread.
template <int C, bool ONE, class S>
__device__ __forceinline__ void normalize(float (&f)[C][8], int kind, const NormArgs& a, const S& w, const S& b, int t,
                                          int threads, RowReduce<ONE>& red) {
  if (kind == VQ_NORM_NONE) return;
  const int d = a.dim;
  const float inv_d = 1.0f / (float)d;
  if (kind == VQ_NORM_LAYER) {
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += f[c][k];  // zeros past the end
    const float mean = red.sum(sum) * inv_d;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) f[c][k] = (c * threads + t) * kChunk + k < d ? f[c][k] - mean : 0.f;
  }
  float sq = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) sq = __builtin_fmaf(f[c][k], f[c][k], sq);
  const float inv = 1.0f / __builtin_sqrtf(red.sum(sq) * inv_d + a.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int at = (c * threads + t) * kChunk;
    float g[8];
    if (w.p) {
      w.get(c, at, d, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[c][k] = f[c][k] * inv * (a.w_offset + g[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[c][k] *= inv;
    }
    if (b.p) {
      b.get(c, at, d, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[c][k] += g[k];
    }
  }
}

// ONE: a row per wavefront and four wavefronts per workgroup, without barriers; else a workgroup of any number of
// wavefronts up to 16 per row.
template <int C, bool ONE, int MAXT, bool AHEAD, bool ZW, bool HW>
__global__ __launch_bounds__(MAXT) void norm_kernel(NormArgs a) {
  __shared__ float part[2][kMaxWaves];
  RowReduce<ONE> red{part};
  const int t = ONE ? threadIdx.x & 63 : threadIdx.x;
  const int threads = ONE ? 64 : blockDim.x;
  const int64_t m = ONE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (m >= a.rows) return;  // ONE: whole wavefronts, no barrier follows
  const int d = a.dim;
  const int at0 = t * kChunk, apart = threads * kChunk;
  constexpr bool kAhead = C <= 4;  // longer rows have no registers to hold h early
  constexpr size_t ez = ZW ? 4 : 2, eh = HW ? 4 : 2;
  const size_t eg = a.gate_dtype == VQ_F32 ? 4 : 2;

  float f[C][8];
  Raw<HW> h[kAhead ? C : 1];
  const char* const hrow = (const char*)a.h + (size_t)m * (size_t)a.ldh * eh;
  {
    const char* z = (const char*)a.z + (size_t)m * (size_t)a.ldz * ez;
    Raw<ZW> zr[C];
#pragma unroll
    for (int c = 0; c < C; ++c) zr[c] = load_chunk<ZW>(z, at0 + c * apart, d);
    if (kAhead && a.h) {
#pragma unroll
      for (int c = 0; c < C; ++c) h[c] = load_chunk<HW>(hrow, at0 + c * apart, d);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) widen(zr[c], a.z_dtype, f[c]);
  }
  Shared<C, AHEAD> pw, pb, gt, nw, nb;
  pw.fetch(a.post_w, a.w_dtype, at0, apart, d);
  pb.fetch(a.post_b, a.w_dtype, at0, apart, d);
  gt.fetch(a.gate ? (const char*)a.gate + (size_t)(m / a.gate_rows) * (size_t)d * eg : nullptr, a.gate_dtype, at0, apart, d);
  nw.fetch(a.pre_w, a.w_dtype, at0, apart, d);
  nb.fetch(a.pre_b, a.w_dtype, at0, apart, d);

  normalize<C, ONE>(f, a.post, a, pw, pb, t, threads, red);

  if (a.gate) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float g[8];
      gt.get(c, at0 + c * apart, d, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[c][k] *= g[k];
    }
  }
  if (a.combine) {  // r differs from u: a residual or a scale
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float g[8];
      if (a.h) {
        if constexpr (kAhead) {
          widen(h[c], a.h_dtype, g);
        } else {
          widen(load_chunk<HW>(hrow, at0 + c * apart, d), a.h_dtype, g);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        f[c][k] *= a.gate_scale;
        if (a.h) f[c][k] = __builtin_fmaf(a.res_scale, g[k], f[c][k]);
      }
    }
  }
  if (a.r) {
    char* r = (char*)a.r + (size_t)m * (size_t)d * eh;
#pragma unroll
    for (int c = 0; c < C; ++c) store_chunk(r, a.h_dtype, at0 + c * apart, d, f[c]);
  }
  if (a.x || a.q) {
    normalize<C, ONE>(f, a.pre, a, nw, nb, t, threads, red);
    if (a.x) {
      char* x = (char*)a.x + (size_t)m * (size_t)d * (a.x_dtype == VQ_F32 ? 4 : 2);
#pragma unroll
      for (int c = 0; c < C; ++c) store_chunk(x, a.x_dtype, at0 + c * apart, d, f[c]);
    }
    if (a.q) {
      uint32_t big = 0;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (at0 + c * apart + k < d) big = max(big, vqd::abs_bits(f[c][k]));
      const vqd::Q8Scale sc = vqd::q8_scale(red.max_bits(big));
      const int64_t ldq = vqi::q8_row_bytes(d);
      uint8_t* q = a.q + (size_t)m * (size_t)ldq;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int at = at0 + c * apart;
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
}

template <int C, bool ONE, int MAXT, bool AHEAD>
vq_status launch(const NormArgs& a, hipStream_t stream, bool check_only) {
  // whole 128-byte steps of q have to be covered, pad included: 16 chunks
  const int chunks = (int)(vqi::q8_row_bytes(a.dim) / kChunk);
  const int wg = ONE ? 256 : ((chunks + C - 1) / C + 63) / 64 * 64;
  const int64_t blocks = ONE ? ((int64_t)a.rows + 3) / 4 : a.rows;
  if (!vqi::grid_ok(blocks, wg)) return VQ_ERR_SHAPE;
  if (check_only) return VQ_OK;
  const dim3 g((uint32_t)blocks), b(wg);
  if (a.z_dtype == VQ_F32) {
    if (a.h_dtype == VQ_F32) norm_kernel<C, ONE, MAXT, AHEAD, true, true><<<g, b, 0, stream>>>(a);
    else norm_kernel<C, ONE, MAXT, AHEAD, true, false><<<g, b, 0, stream>>>(a);
  } else {
    if (a.h_dtype == VQ_F32) norm_kernel<C, ONE, MAXT, AHEAD, false, true><<<g, b, 0, stream>>>(a);
    else norm_kernel<C, ONE, MAXT, AHEAD, false, false><<<g, b, 0, stream>>>(a);
  }
  return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP;
}

// Rows up to which a row gets as many threads as it has chunks (two rows per CU), and the vectors are loaded ahead.
constexpr int kFewRows = 512;

}  // namespace

namespace vqi {

vq_status launch_norm(const NormArgs& a, void* stream_, bool check_only) {
  hipStream_t stream = (hipStream_t)stream_;
  const int d = a.dim;
  if (d <= 512) return launch<1, true, 256, true>(a, stream, check_only);
  // measured, 8192-wide rows with both norms, gate and residual in bf16: 64 rows 6.7 us with one chunk per thread and
  // 7.4 us with two; 8192 rows 181 us and 140 us
  if (a.rows > kFewRows || d > 8192) {
    if (d <= 8192) return launch<2, false, 512, false>(a, stream, check_only);
    if (d <= 16384) return launch<2, false, 1024, false>(a, stream, check_only);
    if (d <= 32768) return launch<4, false, 1024, false>(a, stream, check_only);
    return launch<8, false, 1024, false>(a, stream, check_only);  // up to kNormMaxDim, partly in scratch
  }
  return launch<1, false, 1024, true>(a, stream, check_only);
}

}  // namespace vqi
