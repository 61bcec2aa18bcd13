// Routing for the products grouped by expert: vq_expert_plan sorts the chosen (token, slot) pairs by expert,
// vq_expert_combine joins a token's expert rows with its router weights.
#include "vq_device.h"
#include "vq_q8_device.h"

namespace {

// A stable counting sort with one workgroup per expert and no workspace.  Workgroup e counts the valid ids below e (its
// first sorted row) and those equal to e, each thread over a contiguous share of the pairs; a prefix sum over the
// threads gives every thread its first row, and the second sweep writes.  The pairs of an expert keep their order, so
// the plan does not depend on timing.  The id list is read E times from the caches (the first 8 of a thread's share stay in
// registers between the sweeps): 8192 pairs over 8 experts take 9 us, 1332 over 64 take 4.6, most of it latency.  Past
// 8192 pairs each thread reads the rest of its share one id after the other, twice: 32768 pairs over 128 experts take 39 us,
// 262144 over 64 take 258, about 1 us for each id of a share.
constexpr int kThreads = 1024;
constexpr int kHeld = 8;

__global__ __launch_bounds__(kThreads) void expert_plan_kernel(int32_t pairs, int32_t top, int32_t experts,
                                                              const int32_t* __restrict__ ids,
                                                              int32_t* __restrict__ offsets, int32_t* __restrict__ rows,
                                                              int32_t* __restrict__ pos) {
  __shared__ int32_t wave_eq[kThreads / 64], wave_lt[kThreads / 64];
  const int32_t e = (int32_t)blockIdx.x;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int32_t share = (pairs + kThreads - 1) / kThreads;
  const int64_t first = (int64_t)t * share;
  const int32_t lo = (int32_t)min(first, (int64_t)pairs), hi = (int32_t)min(first + share, (int64_t)pairs);
  int32_t eq = 0, lt = 0;
  int32_t held[kHeld];  // the share's first ids, loaded together and kept for the second sweep
#pragma unroll
  for (int k = 0; k < kHeld; ++k) held[k] = lo + k < hi ? ids[lo + k] : -1;
  auto count = [&](int32_t id) {
    eq += id == e;
    lt += id >= 0 && id < e;
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k) count(held[k]);
  for (int32_t i = lo + kHeld; i < hi; ++i) count(ids[i]);
  int32_t incl = eq;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int32_t up = __shfl_up(incl, o, 64);
    if (lane >= o) incl += up;
    lt += __shfl_xor(lt, o, 64);
  }
  if (lane == 63) {
    wave_eq[wave] = incl;
    wave_lt[wave] = lt;
  }
  __syncthreads();
  int32_t below = 0, all = 0, base = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    base += wave_lt[w];
    if (w < wave) below += wave_eq[w];
    all += wave_eq[w];
  }
  if (t == 0) {
    offsets[e] = base;
    if (e == experts - 1) offsets[experts] = base + all;
  }
  int32_t at = base + below + incl - eq;
  auto place = [&](int32_t i, int32_t id) {
    if (id == e) {
      rows[at] = i / top;
      pos[i] = at++;
    } else if (e == 0 && (id < 0 || id >= experts)) {
      pos[i] = -1;  // no expert here: the pair is dropped
    }
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (lo + k < hi) place(lo + k, held[k]);
  for (int32_t i = lo + kHeld; i < hi; ++i) place(i, ids[i]);
}

// y[t] = sum_j p[t][j] z[pos[t][j]] in fp32, j ascending; 4 columns per thread.  Bound by the bytes of z: 8192 rows of
// 4096 columns take 35 us (4.8 TB/s with the output).
__global__ __launch_bounds__(256) void expert_combine_kernel(int32_t tokens, int32_t top, int32_t n, int32_t zrows,
                                                             const float* __restrict__ z,
                                                             const int32_t* __restrict__ pos,
                                                             const float* __restrict__ p, void* y, vq_dtype y_dtype) {
  const int32_t groups = (n + 3) / 4;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (int64_t)tokens * groups) return;
  const int32_t t = (int32_t)(id / groups);
  const int32_t c = (int32_t)(id - (int64_t)t * groups) * 4;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int32_t j = 0; j < top; ++j) {
    const int32_t r = pos[(int64_t)t * top + j];
    if (r < 0 || r >= zrows) continue;
    const float w = p[(int64_t)t * top + j];
    const float* row = z + (int64_t)r * n + c;
    float v[4];
    if (c + 4 <= n) {
      __builtin_memcpy(v, row, 16);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = c + k < n ? row[k] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = __builtin_fmaf(w, v[k], acc[k]);
  }
  const int64_t at = (int64_t)t * n + c;
  if (c + 4 <= n) {
    if (y_dtype == VQ_F32) {
      __builtin_memcpy((float*)y + at, acc, 16);
    } else {
      uint16_t h[4];
      vqd::narrow<4>(acc, y_dtype, h);
      __builtin_memcpy((uint16_t*)y + at, h, 8);
    }
  } else {
    for (int k = 0; k < 4; ++k)
      if (c + k < n) vqd::store_out(y, (size_t)(at + k), acc[k], y_dtype);
  }
}

}  // namespace

namespace vqi {

vq_status launch_expert_plan(int32_t tokens, int32_t top, int32_t experts, const int32_t* ids, int32_t* offsets,
                             int32_t* rows, int32_t* pos, void* stream) {
  expert_plan_kernel<<<dim3((uint32_t)experts), dim3(kThreads), 0, (hipStream_t)stream>>>(tokens * top, top, experts, ids,
                                                                                         offsets, rows, pos);
  return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP;
}

vq_status launch_expert_combine(int32_t tokens, int32_t top, int32_t n, int32_t rows, const float* z,
                                const int32_t* pos, const float* p, void* y, vq_dtype y_dtype, void* stream,
                                bool check_only) {
  const int64_t items = (int64_t)tokens * ((n + 3) / 4);
  if (!vqi::grid_ok((items + 255) / 256, 256)) return VQ_ERR_SHAPE;
  if (check_only) return VQ_OK;
  expert_combine_kernel<<<dim3((uint32_t)((items + 255) / 256)), dim3(256), 0, (hipStream_t)stream>>>(
      tokens, top, n, rows, z, pos, p, y, y_dtype);
  return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP;
}

}  // namespace vqi
