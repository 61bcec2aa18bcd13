// The 8-bit products: y[m][n] = (sum_k q[m][k] w[n][k]) s[m] sw[n] (+ bias[n]), dense (vq_q8_gemm) and grouped by
// expert (vq_q8_gemm_grouped), on the int8 matrix instructions with exact int32 sums.
//
// Rows of q and w are whole 128-byte steps with zero pads, so no kernel has a K edge; rows past an edge of a tile read
// the last valid row again and are not stored.  Sums of integers have no order, so nothing here depends on how K is cut.
#include "vq_device.h"
#include "vq_q8_device.h"

namespace {

using vqi::Q8Args;

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kStep = 128;  // bytes of K per tile step

// ---------------------------------------------------------------- groups

// The rows of one tile: sorted rows [row0, end) of expert e, at most BM of them computed from row0 on.
struct Span {
  int32_t e, row0, end;
};

// Row tile `mt` of the grouped product: experts in order, each with ceil(rows / BM) tiles.  Every wavefront computes it
// by itself: 64 experts per pass, a prefix sum of their tile counts over the lanes.  false: there is no such tile.
template <int BM>
__device__ __forceinline__ bool find_span(const Q8Args& a, int32_t mt, Span& sp) {
  const int lane = threadIdx.x & 63;
  int32_t before = 0;
  for (int32_t e0 = 0; e0 < a.experts; e0 += 64) {
    const int32_t e = e0 + lane;
    int32_t lo = 0, hi = 0;
    if (e < a.experts) {  // bounded by m whatever the buffer holds
      lo = min(max(a.offsets[e], 0), a.m);
      hi = min(max(a.offsets[e + 1], lo), a.m);
    }
    const int32_t tiles = (hi - lo + BM - 1) / BM;
    int32_t incl = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int32_t up = __shfl_up(incl, o, 64);
      if (lane >= o) incl += up;
    }
    const uint64_t hit = __ballot(mt < before + incl);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      sp.e = e0 + at;
      sp.row0 = __shfl(lo + (mt - before - (incl - tiles)) * BM, at, 64);
      sp.end = __shfl(hi, at, 64);
      sp.e = __builtin_amdgcn_readfirstlane(sp.e);
      sp.row0 = __builtin_amdgcn_readfirstlane(sp.row0);
      sp.end = __builtin_amdgcn_readfirstlane(sp.end);
      return true;
    }
    before += __shfl(incl, 63, 64);
  }
  return false;
}
// Upper bound of the row tiles of a grouped product (sum of ceil(rows_e / bm)).
inline int64_t span_bound(const Q8Args& a, int bm) {
  const int64_t e = a.m < a.experts ? a.m : a.experts;
  return ((int64_t)a.m + e * (bm - 1)) / bm;
}

// Token of sorted row r.
__device__ __forceinline__ int32_t token_of(const Q8Args& a, int32_t r) {
  return a.rows ? min(max(a.rows[r], 0), a.tokens - 1) : min(r, a.tokens - 1);
}

__device__ __forceinline__ float silu(float g) { return g * (1.0f / (1.0f + expf(-g))); }

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

// ---------------------------------------------------------------- tiles

// Copies 16 bytes per lane from `g` to LDS at the wavefront's `l` + 16 lane, past the registers.
__device__ __forceinline__ void to_lds(const uint8_t* g, uint8_t* l) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                   (__attribute__((address_space(3))) void*)l, 16, 0, 0);
}

// A workgroup of WM x WN wavefronts computes BM tokens x BN weight rows (with the gate: BN / 2 outputs, 32-row blocks of
// gate and up rows in turn, so that a lane ends with both values of an output).  The weights are the matrix
// instruction's first operand: a lane then holds 16 outputs of one token, and since block row i holds weight row
// perm(i) they are 16 consecutive ones.
template <int BM, int BN, int WM, int WN, bool GATED, bool SPLIT>
__global__ __launch_bounds__(64 * WM * WN) void q8_tile_kernel(Q8Args a, int32_t nt, int32_t mt_count) {
  constexpr int kWaves = WM * WN;
  constexpr int MI = BM / WM / 32, NI = BN / WN / 32;
  constexpr int TL = BM / 8 / kWaves, WL = BN / 8 / kWaves;  // 8-row loads per wavefront and step
  static_assert(TL * 8 * kWaves == BM && WL * 8 * kWaves == BN, "whole loads");
  static_assert(!GATED || NI % 2 == 0, "gate and up blocks in one wavefront");
  constexpr int kOut = GATED ? BN / 2 : BN;  // outputs per tile
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][(BM + BN) * kStep];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // tiles of one XCD (workgroup mod 8) are neighbours: 8 row tiles by all columns, columns slowest
  const int32_t total = mt_count * nt;
  const int32_t per = (total + 7) / 8;
  const int32_t id = (int32_t)(blockIdx.x & 7) * per + (int32_t)(blockIdx.x >> 3);
  if ((int32_t)(blockIdx.x >> 3) >= per || id >= total) return;
  const int32_t band = id / (8 * nt), in_band = id - band * 8 * nt;
  const int32_t band_rows = min(8, mt_count - band * 8);
  const int32_t mt = band * 8 + in_band % band_rows;
  const int32_t n0 = in_band / band_rows * kOut;

  Span sp{0, 0, 0};
  if (a.experts) {
    if (!find_span<BM>(a, mt, sp)) return;
  } else {
    sp.row0 = mt * BM;
    sp.end = a.m;
  }
  const int64_t ld = vqi::q8_row_bytes(a.k);
  const int64_t wrows = GATED ? 2 * (int64_t)a.n : a.n;
  const uint8_t* const w = a.w + (int64_t)sp.e * wrows * ld;

  int32_t kt0 = 0, kt1 = (int32_t)(ld / kStep);
  if constexpr (SPLIT) {
    const int32_t all = kt1;
    kt0 = (int32_t)((int64_t)all * blockIdx.y / a.splits);
    kt1 = (int32_t)((int64_t)all * (blockIdx.y + 1) / a.splits);
  }

  // this lane's 16-byte piece of every load: row p of the tile, chunk lane % 8 of its LDS row, which holds chunk
  // (lane % 8) ^ (p / 2 % 8) of the matrix row (reads of 16 rows at one chunk then fall on all 64 banks)
  const uint8_t* gt[TL];
  const uint8_t* gw[WL];
#pragma unroll
  for (int j = 0; j < TL; ++j) {
    const int p = (j * kWaves + wave) * 8 + (lane >> 3);
    const int32_t r = min(sp.row0 + p, sp.end - 1);
    gt[j] = a.q + (int64_t)token_of(a, r) * ld + kt0 * kStep + (((lane & 7) ^ ((p >> 1) & 7)) * 16);
  }
#pragma unroll
  for (int j = 0; j < WL; ++j) {
    const int p = (j * kWaves + wave) * 8 + (lane >> 3);
    const int i = p & 31, b = p >> 5;
    const int pn = ((i >> 2) & 1) * 16 + (i >> 3) * 4 + (i & 3);
    int64_t r;
    if constexpr (GATED) {
      r = (int64_t)min(n0 + (b >> 1) * 32 + pn, a.n - 1) + (b & 1 ? a.n : 0);
    } else {
      r = min(n0 + b * 32 + pn, a.n - 1);
    }
    gw[j] = w + r * ld + kt0 * kStep + (((lane & 7) ^ ((p >> 1) & 7)) * 16);
  }
  auto fetch = [&](int buf) {
#pragma unroll
    for (int j = 0; j < TL; ++j) {
      to_lds(gt[j], &lds[buf][(j * kWaves + wave) * 1024]);
      gt[j] += kStep;
    }
#pragma unroll
    for (int j = 0; j < WL; ++j) {
      to_lds(gw[j], &lds[buf][BM * kStep + (j * kWaves + wave) * 1024]);
      gw[j] += kStep;
    }
  };

  const int wm = wave / WN, wn = wave % WN;
  const int col = lane & 31, half = lane >> 5;
  v16i acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  const int lt = (wm * MI * 32 + col) * kStep;
  const int lw = BM * kStep + (wn * NI * 32 + col) * kStep;
  auto multiply = [&](int buf) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const int c = ((2 * ks + half) ^ ((lane >> 1) & 7)) * 16;
      v4i t[MI], v[NI];
#pragma unroll
      for (int i = 0; i < MI; ++i) t[i] = *(const v4i*)&lds[buf][lt + i * 32 * kStep + c];
#pragma unroll
      for (int j = 0; j < NI; ++j) v[j] = *(const v4i*)&lds[buf][lw + j * 32 * kStep + c];
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(v[j], t[i], acc[i][j], 0, 0, 0);
    }
  };

  fetch(0);
  int buf = 0;
  for (int32_t kt = kt0; kt < kt1; ++kt) {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wavefront's part of step kt is in LDS
    __syncthreads();                     // everyone's is, and the other buffer's readers are done
    if (kt + 1 < kt1) fetch(buf ^ 1);
    multiply(buf);
    buf ^= 1;
  }

  // outputs: lane = token row0 + .., 16 consecutive channels per block
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int32_t m = sp.row0 + wm * MI * 32 + i * 32 + col;
    if (m >= sp.end) continue;
    if constexpr (SPLIT) {
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int32_t n = n0 + (wn * NI + j) * 32 + half * 16;
        int32_t* at = a.part + ((int64_t)blockIdx.y * a.m + m) * a.n;
        if (n + 16 <= a.n) {
          __builtin_memcpy(at + n, &acc[i][j], 64);
        } else {
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (n + r < a.n) at[n + r] = acc[i][j][r];
        }
      }
    } else {
      const float s = a.s[token_of(a, m)];
      const float* sw = a.sw + (int64_t)sp.e * wrows;
      const uint16_t* bias = a.bias ? a.bias + (int64_t)sp.e * wrows : nullptr;
      if constexpr (GATED) {
#pragma unroll
        for (int j = 0; j < NI; j += 2) {
          const int32_t n = n0 + (wn * NI + j) / 2 * 32 + half * 16;
          float g[16], u[16], bg[16], bu[16], v[16];
          load_run<16>(sw, n, a.n, g);
          load_run<16>(sw + a.n, n, a.n, u);
          load_bias<16>(bias, n, a.n, bg);
          load_bias<16>(bias ? bias + a.n : nullptr, n, a.n, bu);
#pragma unroll
          for (int r = 0; r < 16; ++r)
            v[r] = silu((float)acc[i][j][r] * s * g[r] + bg[r]) * ((float)acc[i][j + 1][r] * s * u[r] + bu[r]);
          store_run<16>(a.y, a.y_dtype, (int64_t)m * a.n, n, a.n, v);
        }
      } else {
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int32_t n = n0 + (wn * NI + j) * 32 + half * 16;
          float sc[16], b[16], v[16];
          load_run<16>(sw, n, a.n, sc);
          load_bias<16>(bias, n, a.n, b);
#pragma unroll
          for (int r = 0; r < 16; ++r) v[r] = (float)acc[i][j][r] * s * sc[r] + b[r];
          store_run<16>(a.y, a.y_dtype, (int64_t)m * a.n, n, a.n, v);
        }
      }
    }
  }
}

// y = (sum of the K splits) s sw + bias: 4 outputs per thread.
__global__ __launch_bounds__(256) void q8_join_kernel(Q8Args a) {
  const int32_t groups = (a.n + 3) / 4;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (int64_t)a.m * groups) return;
  const int32_t m = (int32_t)(id / groups);
  const int32_t n = (int32_t)(id - (int64_t)m * groups) * 4;
  int32_t sum[4] = {0, 0, 0, 0};
  for (int32_t k = 0; k < a.splits; ++k) {
    const int32_t* p = a.part + ((int64_t)k * a.m + m) * a.n + n;
    int32_t v[4] = {0, 0, 0, 0};
    if (n + 4 <= a.n) {
      __builtin_memcpy(v, p, 16);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = n + r < a.n ? p[r] : 0;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) sum[r] += v[r];
  }
  float sc[4], b[4], v[4];
  load_run<4>(a.sw, n, a.n, sc);
  load_bias<4>(a.bias, n, a.n, b);
  const float s = a.s[m];
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = (float)sum[r] * s * sc[r] + b[r];
  store_run<4>(a.y, a.y_dtype, (int64_t)m * a.n, n, a.n, v);
}

// ---------------------------------------------------------------- few rows

// Few tokens: the weights are read once, straight into the matrix instruction's registers.  A workgroup of 8 wavefronts
// takes RT blocks of 16 weight rows (with the gate: 8 RT outputs, one block of gate rows and one of up rows) and up to
// 16 MT tokens; its wavefronts cut K, their int32 sums meet in LDS.
template <int RT, int MT, bool GATED>
__global__ __launch_bounds__(512) void q8_few_kernel(Q8Args a) {
  constexpr int kWaves = 8;
  constexpr int kTiles = RT * MT;
  constexpr int U = 4;  // 64-byte steps in flight
  static_assert(!GATED || RT == 2, "one gate block and one up block");
  constexpr int kOut = GATED ? 16 : 16 * RT;
  __shared__ v4i red[kWaves][kTiles][64];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t n0 = (int32_t)blockIdx.x * kOut;
  Span sp{0, 0, 0};
  if (a.experts) {
    if (!find_span<16 * MT>(a, (int32_t)blockIdx.y, sp)) return;
  } else {
    sp.row0 = (int32_t)blockIdx.y * 16 * MT;
    sp.end = a.m;
  }
  const int64_t ld = vqi::q8_row_bytes(a.k);
  const int64_t wrows = GATED ? 2 * (int64_t)a.n : a.n;
  const int32_t steps = (int32_t)(ld / 64);
  const int32_t k0 = steps * wave / kWaves, k1 = steps * (wave + 1) / kWaves;
  const int row = lane & 15, grp = lane >> 4;

  const uint8_t* gw[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t r = GATED ? (int64_t)min(n0 + row, a.n - 1) + (i ? a.n : 0) : min(n0 + 16 * i + row, a.n - 1);
    gw[i] = a.w + ((int64_t)sp.e * wrows + r) * ld + (int64_t)k0 * 64 + grp * 16;
  }
  const uint8_t* gt[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j)
    gt[j] = a.q + (int64_t)token_of(a, min(sp.row0 + 16 * j + row, sp.end - 1)) * ld + (int64_t)k0 * 64 + grp * 16;

  v4i acc[RT][MT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = v4i{0, 0, 0, 0};

  int32_t k = k0;
  for (; k + U <= k1; k += U) {
    v4i w[U][RT], t[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < RT; ++i) w[u][i] = __builtin_nontemporal_load((const v4i*)(gw[i] + 64 * u));
#pragma unroll
      for (int j = 0; j < MT; ++j) t[u][j] = *(const v4i*)(gt[j] + 64 * u);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) gw[i] += 64 * U;
#pragma unroll
    for (int j = 0; j < MT; ++j) gt[j] += 64 * U;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][i], t[u][j], acc[i][j], 0, 0, 0);
  }
  for (; k < k1; ++k) {
    v4i t[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      t[j] = *(const v4i*)gt[j];
      gt[j] += 64;
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const v4i w = __builtin_nontemporal_load((const v4i*)gw[i]);
      gw[i] += 64;
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, t[j], acc[i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) red[wave][i * MT + j][lane] = acc[i][j];
  __syncthreads();

  // lane: token lane % 16, channels 4 (lane / 16) .. + 3 of a block
  const float* sw = a.sw + (int64_t)sp.e * wrows;
  const uint16_t* bias = a.bias ? a.bias + (int64_t)sp.e * wrows : nullptr;
  for (int o = wave; o < (GATED ? MT : kTiles); o += kWaves) {
    const int j = o % MT, i = o / MT;
    const int32_t m = sp.row0 + 16 * j + row;
    const int32_t n = n0 + 16 * i + 4 * grp;
    v4i sum = red[0][o][lane], up = v4i{0, 0, 0, 0};
#pragma unroll
    for (int k = 1; k < kWaves; ++k) sum += red[k][o][lane];
    if constexpr (GATED) {
#pragma unroll
      for (int k = 0; k < kWaves; ++k) up += red[k][MT + o][lane];
    }
    if (m >= sp.end) continue;
    const float s = a.s[token_of(a, m)];
    float sc[4], b[4], v[4];
    load_run<4>(sw, n, a.n, sc);
    load_bias<4>(bias, n, a.n, b);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = (float)sum[r] * s * sc[r] + b[r];
    if constexpr (GATED) {
      load_run<4>(sw + a.n, n, a.n, sc);
      load_bias<4>(bias ? bias + a.n : nullptr, n, a.n, b);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = silu(v[r]) * ((float)up[r] * s * sc[r] + b[r]);
    }
    store_run<4>(a.y, a.y_dtype, (int64_t)m * a.n, n, a.n, v);
  }
}

// ---------------------------------------------------------------- launches

template <int RT, int MT, bool GATED>
vq_status launch_few(const Q8Args& a, hipStream_t st) {
  const int out = GATED ? 16 : 16 * RT;
  const int64_t gy = a.experts ? span_bound(a, 16 * MT) : ((int64_t)a.m + 16 * MT - 1) / (16 * MT);
  if (gy > 65535 || !vqi::grid_ok((a.n + out - 1) / out, 512)) return VQ_ERR_SHAPE;
  q8_few_kernel<RT, MT, GATED><<<dim3((uint32_t)((a.n + out - 1) / out), (uint32_t)gy), dim3(512), 0, st>>>(a);
  return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP;
}

template <int BM, int BN, int WM, int WN, bool GATED, bool SPLIT>
vq_status launch_tile(const Q8Args& a, hipStream_t st) {
  const int out = GATED ? BN / 2 : BN;
  const int64_t mt = a.experts ? span_bound(a, BM) : ((int64_t)a.m + BM - 1) / BM;
  const int64_t nt = ((int64_t)a.n + out - 1) / out;
  if (mt * nt > 0x3FFFFFFF || !vqi::grid_ok(mt * nt + 8, 64 * WM * WN)) return VQ_ERR_SHAPE;
  const uint32_t blocks = (uint32_t)((mt * nt + 7) / 8 * 8);
  q8_tile_kernel<BM, BN, WM, WN, GATED, SPLIT>
      <<<dim3(blocks, SPLIT ? a.splits : 1), dim3(64 * WM * WN), 0, st>>>(a, (int32_t)nt, (int32_t)mt);
  return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP;
}

constexpr int kFewRows = 64;  // rows (of a group, on average) up to which the weights are streamed through registers

}  // namespace

namespace vqi {

int32_t q8_splits(int32_t m, int32_t n, int32_t k) {
  if (m <= kFewRows) return 1;
  const int64_t tiles = (((int64_t)m + 127) / 128) * (((int64_t)n + 127) / 128);
  if (tiles >= 256) return 1;
  const int64_t steps = q8_row_bytes(k) / kStep;
  int64_t s = 512 / tiles;
  if (s > steps / 8) s = steps / 8;
  return s < 1 ? 1 : (int32_t)s;
}

vq_status launch_q8(const Q8Args& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const int64_t groups = a.experts ? (a.m < a.experts ? a.m : a.experts) : 1;
  const int64_t avg = (a.m + groups - 1) / groups;
  if (avg <= kFewRows) {
    if (a.gated) {
      if (avg <= 16) return launch_few<2, 1, true>(a, st);
      if (avg <= 32) return launch_few<2, 2, true>(a, st);
      return launch_few<2, 4, true>(a, st);
    }
    if (avg <= 16) return launch_few<1, 1, false>(a, st);
    if (avg <= 32) return launch_few<1, 2, false>(a, st);
    return launch_few<1, 4, false>(a, st);
  }
  if (a.gated) return launch_tile<128, 128, 2, 2, true, false>(a, st);
  if (a.splits > 1) {
    const vq_status e = launch_tile<128, 128, 2, 2, false, true>(a, st);
    if (e != VQ_OK) return e;
    const int64_t items = (int64_t)a.m * ((a.n + 3) / 4);  // under 256 tiles of 128 x 128: a small grid
    q8_join_kernel<<<dim3((uint32_t)((items + 255) / 256)), dim3(256), 0, st>>>(a);
    return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP;
  }
  return launch_tile<128, 128, 2, 2, false, false>(a, st);
}

}  // namespace vqi
