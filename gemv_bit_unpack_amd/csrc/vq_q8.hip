// The 8-bit products: y[m][n] = (sum_k q[m][k] w[n][k]) s[m] sw[n] (+ bias[n]), dense (vq_q8_gemm) and grouped by
// expert (vq_q8_gemm_grouped), on the int8 matrix instructions with exact int32 sums.
//
// Up to some hundred rows the weights' bytes bound it (one row of 28672 x 8192: 48 us, 4.9 TB/s), above that the matrix
// pipes at the clock that the card holds under dense 8-bit products (8192^3: 2.2 - 2.4 POP/s on random values, 3.4 on
// zeros).
//
// Rows of q and w are whole 128-byte steps with zero pads, so no kernel has a K edge; rows past an edge of a tile read
// the last valid row again and are not stored.  Sums of integers have no order, so nothing here depends on how K is cut.
#include <algorithm>

#include "vq_device.h"
#include "vq_q8_device.h"

namespace {

using vqi::OneArgs;
using vqi::Q8Args;

constexpr int kOneSlots = vqi::kQ8OneSlots;

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
      sp.e = __builtin_amdgcn_readfirstlane(e0 + at);
      sp.row0 = __builtin_amdgcn_readfirstlane(__shfl(lo + (mt - before - (incl - tiles)) * BM, at, 64));
      sp.end = __builtin_amdgcn_readfirstlane(__shfl(hi, at, 64));
      // offsets that no plan wrote may overlap and their tiles overflow: still only rows of this group
      return sp.row0 >= __builtin_amdgcn_readfirstlane(__shfl(lo, at, 64)) && sp.row0 < sp.end;
    }
    before += __shfl(incl, 63, 64);
  }
  return false;
}
// Row tiles of the grouped product, as find_span counts them.
template <int BM>
__device__ __forceinline__ int32_t count_spans(const Q8Args& a) {
  int32_t tiles = 0;
  for (int32_t e = threadIdx.x & 63; e < a.experts; e += 64) {
    const int32_t lo = min(max(a.offsets[e], 0), a.m), hi = min(max(a.offsets[e + 1], lo), a.m);
    tiles += (hi - lo + BM - 1) / BM;
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) tiles += __shfl_xor(tiles, o, 64);
  return __builtin_amdgcn_readfirstlane(tiles);
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

// ---------------------------------------------------------------- tiles

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

// One tile: KG groups of WM x WN wavefronts, each with its share of K and its own steps in LDS, compute BM rows (from
// row0, those below end) by BN weight rows (with the gate: BN / 2 outputs, 32-row blocks of gate and up rows in turn, so
// that a lane ends with both values of an output).  The weights are the matrix instruction's first operand: a lane then
// holds 16 outputs of one token, and since block row i holds weight row perm(i) they are 16 consecutive ones.  The reads
// of the next 32-byte slice go between the products of this one (8192^3: 490 -> 470 us).
template <int BM, int BN, int WM, int WN, int NB, int KG, bool GATED, bool SPLIT>
__device__ __forceinline__ void tile(const Q8Args& a, const Span& sp, int32_t n0, uint8_t* lds) {
  constexpr int kWaves = WM * WN;
  constexpr int MI = BM / WM / 32, NI = BN / WN / 32;
  constexpr int TL = BM / 8 / kWaves, WL = BN / 8 / kWaves;  // 8-row loads per wavefront and step
  constexpr int kBuf = (BM + BN) * kStep;
  // steps in LDS: one is read while NB - 1 are on their way; vmcnt of a wavefront whose loads of one step more than the
  // next may be outstanding
  constexpr int kLater = (NB - 2) * (TL + WL);
  static_assert(NB >= 2 && kLater < 64, "the wait counter holds 6 bits");
  constexpr int kWaitNext = 0x0070 | (kLater & 15) | (kLater >> 4) << 14;  // and lgkmcnt(0)
  static_assert(TL * 8 * kWaves == BM && WL * 8 * kWaves == BN, "whole loads");
  static_assert(!GATED || NI % 2 == 0, "gate and up blocks in one wavefront");
  static_assert(KG == 1 || (KG == 2 && MI == 1 && NI == 1), "two groups of wavefronts halve K for single blocks");

  const int lane = threadIdx.x & 63;
  const int all_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = all_wave % kWaves, group = all_wave / kWaves;
  lds += group * NB * kBuf;
  const int64_t ld = vqi::q8_row_bytes(a.k);
  const int64_t wrows = GATED ? 2 * (int64_t)a.n : a.n;
  const uint8_t* const w = a.w + (int64_t)sp.e * wrows * ld;

  int32_t kt0 = 0, kt1 = (int32_t)(ld / kStep);
  if constexpr (SPLIT) {
    const int32_t all = kt1;
    kt0 = (int32_t)((int64_t)all * blockIdx.y / a.splits);
    kt1 = (int32_t)((int64_t)all * (blockIdx.y + 1) / a.splits);
  }

  // steps of each group of wavefronts; the second may have one less, and multiplies zeros in its place
  const int32_t n = (kt1 - kt0 + KG - 1) / KG;
  kt0 += group * n;
  const int32_t mine = KG == 1 ? n : min(n, kt1 - kt0);

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
  auto fetch = [&](int buf, int32_t step) {
    if (KG > 1 && step >= mine) {
#pragma unroll
      for (int j = 0; j < TL; ++j)
        *(v4i*)(lds + buf * kBuf + (j * kWaves + wave) * 1024 + lane * 16) = v4i{0, 0, 0, 0};
      return;
    }
#pragma unroll
    for (int j = 0; j < TL; ++j) {
      to_lds(gt[j], lds + buf * kBuf + (j * kWaves + wave) * 1024);
      gt[j] += kStep;
    }
#pragma unroll
    for (int j = 0; j < WL; ++j) {
      to_lds(gw[j], lds + buf * kBuf + BM * kStep + (j * kWaves + wave) * 1024);
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

  // fragments of one 32-byte slice of the step, two sets: the next slice is read while this one is multiplied
  const int lt = (wm * MI * 32 + col) * kStep;
  const int lw = BM * kStep + (wn * NI * 32 + col) * kStep;
  v4i ft[2][MI], fw[2][NI];
  auto read = [&](int set, int buf, int ks) {
    const int c = ((2 * ks + half) ^ ((lane >> 1) & 7)) * 16;
#pragma unroll
    for (int i = 0; i < MI; ++i) ft[set][i] = *(const v4i*)(lds + buf * kBuf + lt + i * 32 * kStep + c);
#pragma unroll
    for (int j = 0; j < NI; ++j) fw[set][j] = *(const v4i*)(lds + buf * kBuf + lw + j * 32 * kStep + c);
  };
  auto multiply = [&](int set) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[set][j], ft[set][i], acc[i][j], 0, 0, 0);
  };

#pragma unroll
  for (int b = 0; b < NB; ++b)
    if (b < NB - 1 && b < n) fetch(b, b);
  if (NB - 1 <= mine) {
    __builtin_amdgcn_s_waitcnt(kWaitNext);  // this wavefront's part of the first step is in LDS
  } else {
    __builtin_amdgcn_s_waitcnt(0x0070);
  }
  meet();  // and everyone's
  if (NB - 1 < n) fetch(NB - 1, NB - 1);
  read(0, 0, 0);
  int buf = 0;
  auto mix = [&] {  // the reads of the next slice between the products of this one
#pragma unroll
    for (int i = 0; i < MI + NI; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, MI * NI, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto first3 = [&] {
    multiply(0);
    read(1, buf, 1);
    mix();
    multiply(1);
    read(0, buf, 2);
    mix();
    multiply(0);
    read(1, buf, 3);
    mix();
  };
  for (int32_t kt = 0; kt + 1 < n; ++kt) {
    first3();
    // its part of the next step is in LDS (steps after that may still be on their way), its last reads are done
    if (kt + NB - 1 < mine) {
      __builtin_amdgcn_s_waitcnt(kWaitNext);
    } else {
      __builtin_amdgcn_s_waitcnt(0x0070);
    }
    meet();  // and everyone's: the next step may be read, this one overwritten
    if (kt + NB < n) fetch(buf, kt + NB);
    const int next = buf + 1 == NB ? 0 : buf + 1;
    __builtin_amdgcn_sched_barrier(0);
    multiply(1);
    read(0, next, 0);
    mix();
    buf = next;
  }
  first3();
  multiply(1);
  if constexpr (KG == 2) {  // the second group's sums join the first's
    v4i* const sums = (v4i*)(lds + (1 - group) * NB * kBuf) + wave * 4 * 64 + lane;
    meet();  // no one reads a step any more
    if (group == 1) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        sums[r * 64] = v4i{acc[0][0][4 * r], acc[0][0][4 * r + 1], acc[0][0][4 * r + 2], acc[0][0][4 * r + 3]};
    }
    __syncthreads();
    if (group == 1) return;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const v4i v = sums[r * 64];
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[0][0][4 * r + k] += v[k];
    }
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
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            g[r] *= (float)acc[i][j][r] * s;
            u[r] *= (float)acc[i][j + 1][r] * s;
          }
          if (bias) {
            load_bias<16>(bias, n, a.n, bg);
            load_bias<16>(bias + a.n, n, a.n, bu);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              g[r] += bg[r];
              u[r] += bu[r];
            }
          }
#pragma unroll
          for (int r = 0; r < 16; ++r) v[r] = silu(g[r]) * u[r];
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

// Tiles with several workgroups per CU.
template <int BM, int BN, int WM, int WN, int NB, int KG, bool GATED, bool SPLIT>
__global__ __launch_bounds__(64 * WM * WN * KG) void q8_tile_kernel(Q8Args a, int32_t nt, int32_t mt_count) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[KG * NB * (BM + BN) * kStep];
  int32_t mt, nti;
  if (!place((int32_t)blockIdx.x, mt_count * nt, mt_count, nt, mt, nti)) return;
  Span sp{0, mt * BM, a.m};
  if (a.experts && !find_span<BM>(a, mt, sp)) return;
  tile<BM, BN, WM, WN, NB, KG, GATED, SPLIT>(a, sp, nti * (GATED ? BN / 2 : BN), lds);
}

// 256 x 256 tiles on 8 wavefronts, one workgroup per CU: half the LDS reads and half the matrix bytes per operation of
// 128 x 128.  128 rows only where a group's (or the matrix's) last tile has no more left, and in the last round over the
// 256 CUs if at most half of them have a tile in it: two half tiles for each then take half a round.
// 4096 x 14336 x 4096 (3.5 rounds): 241 us with whole tiles only, 224 us.
template <bool GATED>
__global__ __launch_bounds__(512) void q8_big_kernel(Q8Args a, int32_t nt, int32_t mt_count) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * 512 * kStep];
  if (a.experts) mt_count = max(0, min(count_spans<256>(a), mt_count));  // the launch has room for the bound
  const int32_t total = mt_count * nt;
  const int32_t rest = total % 256;
  const int32_t full = rest <= 128 ? total - rest : total;  // ids from the next multiple of 8 on are halves
  const int32_t whole = (full + 7) / 8 * 8;
  const int32_t id = (int32_t)blockIdx.x;
  int32_t mt, nti, part = 0;
  const bool half = id >= whole;
  if (half) {
    const int32_t at = full + (id - whole) / 2;
    if (at >= total) return;
    part = (id - whole) & 1;
    tile_at(at, mt_count, nt, mt, nti);
  } else if (!place(id, full, mt_count, nt, mt, nti)) {
    return;
  }
  Span sp{0, mt * 256, a.m};
  if (a.experts && !find_span<256>(a, mt, sp)) return;
  sp.row0 += part * 128;
  if (sp.row0 >= sp.end) return;
  if (half) sp.end = min(sp.end, sp.row0 + 128);
  if (half || sp.end - sp.row0 <= 128) {
    tile<128, 256, 2, 4, 2, 1, GATED, false>(a, sp, nti * (GATED ? 128 : 256), lds);
  } else {
    tile<256, 256, 2, 4, 2, 1, GATED, false>(a, sp, nti * (GATED ? 128 : 256), lds);
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
  const int64_t apart = (int64_t)a.m * a.n;
  const int32_t* p = a.part + (int64_t)m * a.n + n;
  if (n + 4 <= a.n) {
#pragma unroll 8
    for (int32_t k = 0; k < a.splits; ++k) {
      int32_t v[4];
      __builtin_memcpy(v, p + k * apart, 16);
#pragma unroll
      for (int r = 0; r < 4; ++r) sum[r] += v[r];
    }
  } else {
    for (int32_t k = 0; k < a.splits; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r) sum[r] += n + r < a.n ? p[k * apart + r] : 0;
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
// takes RT blocks of 16 weight rows and up to 16 MT tokens; its wavefronts cut K, their int32 sums meet in LDS.  Bound by
// the weights' bytes (8 x 8192 x 8192: 17.9 us, 3.8 TB/s) and, with small matrices, by the latency of one pass over K
// (16 x 4096 x 4096: 7.1 us).
template <int RT, int MT>
__global__ __launch_bounds__(512) void q8_few_kernel(Q8Args a) {
  constexpr int kTiles = RT * MT;
  constexpr int U = RT * MT == 1 ? 8 : 4;  // 64-byte steps in flight
  __shared__ v4i red[8][kTiles][64];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t n0 = (int32_t)blockIdx.x * 16 * RT;
  const int64_t ld = vqi::q8_row_bytes(a.k);
  const int32_t steps = (int32_t)(ld / 64);
  const int32_t k0 = steps * wave / 8, k1 = steps * (wave + 1) / 8;
  const int row = lane & 15, grp = lane >> 4;

  const uint8_t* gw[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
    gw[i] = a.w + (int64_t)min(n0 + 16 * i + row, a.n - 1) * ld + (int64_t)k0 * 64 + grp * 16;
  const uint8_t* gt[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j)
    gt[j] = a.q + (int64_t)min(16 * j + row, a.m - 1) * ld + (int64_t)k0 * 64 + grp * 16;

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
    __builtin_amdgcn_sched_barrier(0);  // all U steps' loads are in flight before the first is used
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

  // lane: token lane % 16, channels 4 (lane / 16) .. + 3 of a block; the wavefronts share the blocks out
  for (int o = wave; o < kTiles; o += 8) {
    const int j = o % MT, i = o / MT;
    const int32_t m = 16 * j + row;
    const int32_t n = n0 + 16 * i + 4 * grp;
    v4i sum = red[0][o][lane];
#pragma unroll
    for (int v = 1; v < 8; ++v) sum += red[v][o][lane];
    if (m >= a.m) continue;
    const float s = a.s[m];
    float sc[4], b[4], v[4];
    load_run<4>(a.sw, n, a.n, sc);
    load_bias<4>(a.bias, n, a.n, b);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = (float)sum[r] * s * sc[r] + b[r];
    store_run<4>(a.y, a.y_dtype, (int64_t)m * a.n, n, a.n, v);
  }
}

// ---------------------------------------------------------------- one token

// Products of a single token, cut to 8 bits inside the kernel: each workgroup finds the row's scale (of the 1 + rows it
// needs: `slots`) and keeps the 8-bit row in LDS while its first weight loads are on their way, so a token costs one
// launch.  Weights go to the matrix instruction as in q8_few_kernel, with the token in all 16 columns.
//   dense   y = the product                                        w [n]
//   GATED   slot blockIdx.y: y[slot] = silu(g) u, fp32             w [experts][2 n], expert ids[slot], the same x for all
//   JOIN    y = sum over slots of p[slot] * product(x row slot)    w [experts][n], experts ids[slot]; the rows of all
//           slots are in LDS, so there is a bound on slots and columns together (kQ8OneSlots)
// Slots whose id is outside [0, experts) are left out.
// Bound by the weights' bytes (28672 x 8192: 48 us, 4.9 TB/s); a small matrix by the chain row -> scale -> 8 bits ->
// products (4096 x 4096: 6.6 us; cutting the row in a launch of its own made it 3.0 + 5.3 us and a gap).
template <int RT, int WN, bool GATED, bool JOIN, vq_dtype XT>
__global__ __launch_bounds__(512) void q8_one_kernel(OneArgs a) {
  constexpr int WK = 8 / WN;
  // 64-byte steps of a block (JOIN: 14336 columns are 28 steps per wavefront, whole blocks of 4: 30.6 us for 2 experts
  // of 4096 rows, 31.8 with blocks of 8 and 4 steps left over).  Steps left over are loaded one by one: with 10 steps per
  // wavefront 5120 x 5120 takes 13.8 us, with 8 4096 x 4096 takes 7.5, each with its weights from memory
  constexpr int U = RT == 1 && !JOIN ? 8 : 4;
  constexpr int kOut = GATED ? 16 : 16 * RT;
  static_assert(!GATED || RT == 2, "one gate block and one up block");
  static_assert(!JOIN || RT == 1, "one block per wavefront");
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ uint32_t big[8][kOneSlots];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wave % WK, wn = wave / WK;
  const int32_t n0 = ((int32_t)blockIdx.x * WN + wn) * kOut;
  const int64_t ld = vqi::q8_row_bytes(a.k);
  const int64_t wrows = GATED ? 2 * (int64_t)a.n : a.n;
  const int slots = JOIN ? a.slots : 1;
  const int32_t first = JOIN ? 0 : (int32_t)blockIdx.y;  // the slot (GATED) or the first slot
  auto expert = [&](int slot) { return a.experts ? a.ids[slot] : 0; };
  auto there = [&](int32_t e) { return a.experts == 0 || (e >= 0 && e < a.experts); };
  if (!JOIN && !there(expert(first))) return;

  const int32_t steps = (int32_t)(ld / 64);
  const int32_t k0 = steps * wk / WK, k1 = steps * (wk + 1) / WK;
  const int row = lane & 15, grp = lane >> 4;
  const uint8_t* gw[RT];
  auto aim = [&](int32_t e) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int64_t r = GATED ? (int64_t)min(n0 + row, a.n - 1) + (i ? a.n : 0) : min(n0 + 16 * i + row, a.n - 1);
      gw[i] = a.w + ((int64_t)e * wrows + r) * ld + (int64_t)k0 * 64 + grp * 16;
    }
  };
  v4i w[2][U][RT];  // two blocks of U steps: one on its way while the other is used
  auto load = [&](int set) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < RT; ++i) w[set][u][i] = __builtin_nontemporal_load((const v4i*)(gw[i] + 64 * u));
#pragma unroll
    for (int i = 0; i < RT; ++i) gw[i] += 64 * U;
  };
  const int32_t blocks = (k1 - k0) / U;  // whole blocks of U steps; the steps left over are loaded one by one
  // the first slot that has an expert; its first loads
  int slot = 0;
  while (JOIN && slot < slots && !there(expert(slot))) ++slot;
  if (slot < slots) {
    aim(expert(first + slot));
    if (blocks > 0) load(0);
    if (blocks > 1) load(1);
  }
  __builtin_amdgcn_sched_barrier(0);

  // the rows' largest values, then the rows in 8 bits
  const int64_t xrow = JOIN ? a.k : 0;  // GATED slots share the token's row
  auto chunk = [&](int j, int32_t c, float (&f)[8]) {
    constexpr int es = XT == VQ_F32 ? 4 : 2;
    const char* p = (const char*)a.x + (j * xrow + (int64_t)c * 8) * es;
    if (c * 8 + 8 <= a.k) {
      uint32_t v[2 * es];
      __builtin_memcpy(v, p, 8 * es);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (XT == VQ_F32) {
          f[k] = __builtin_bit_cast(float, v[k]);
        } else {
          f[k] = vqd::x_to_f32<XT == VQ_F16 ? 0 : 1>(v[k / 2] >> (16 * (k & 1)));
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        f[k] = 0.f;
        if (c * 8 + k < a.k) {
          if constexpr (XT == VQ_F32) {
            f[k] = ((const float*)p)[k];
          } else {
            f[k] = vqd::x_to_f32<XT == VQ_F16 ? 0 : 1>(((const uint16_t*)p)[k]);
          }
        }
      }
    }
  };
  const int32_t chunks = (a.k + 7) / 8;
  constexpr int kHold = JOIN ? 1 : 2;  // chunks per thread that stay in registers between the two sweeps
  float hold[kHold][8];
  for (int j = 0; j < slots; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
      const int32_t c = threadIdx.x + 512 * h;
#pragma unroll
      for (int k = 0; k < 8; ++k) hold[h][k] = 0.f;
      if (c < chunks) chunk(j, c, hold[h]);
    }
#pragma unroll
    for (int h = 0; h < kHold; ++h)
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, vqd::abs_bits(hold[h][k]));
    for (int32_t c = threadIdx.x + 512 * kHold; c < chunks; c += 512) {
      float f[8];
      chunk(j, c, f);
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, vqd::abs_bits(f[k]));
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
    if (lane == 0) big[wave][j] = m;
  }
  __syncthreads();
  auto scale = [&](int j) {
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < 8; ++v) m = max(m, big[v][j]);
    return vqd::q8_scale(m);
  };
  for (int j = 0; j < slots; ++j) {
    const vqd::Q8Scale sc = scale(j);
    auto put = [&](int32_t c, const float (&f)[8]) {
      uint32_t v[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k >> 2] |= (uint32_t)(uint8_t)vqd::q8_value(f[k], sc) << (8 * (k & 3));
      *(uint2*)(lds + j * ld + c * 8) = make_uint2(v[0], v[1]);
    };
    int32_t c = threadIdx.x;
    if (!JOIN) {
#pragma unroll
      for (int h = 0; h < kHold; ++h, c += 512)
        if (c * 8 < (int32_t)ld) put(c, hold[h]);  // zeros past the row's end
    }
    for (; c * 8 < (int32_t)ld; c += 512) {
      float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (c < chunks) chunk(j, c, f);
      put(c, f);
    }
  }
  __syncthreads();

  v4i* const red = (v4i*)(lds + slots * ld);  // [slots][8][RT][64]
  for (; slot < slots;) {
    v4i acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = v4i{0, 0, 0, 0};
    const uint8_t* xq = lds + slot * ld + (int64_t)k0 * 64 + grp * 16;
    int next = slot + 1;
    while (JOIN && next < slots && !there(expert(next))) ++next;
    auto use = [&](int set) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const v4i t = *(const v4i*)(xq + 64 * u);
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[set][u][i], t, acc[i], 0, 0, 0);
      }
      xq += 64 * U;
    };
    for (int32_t k = 0; k < blocks; k += 2) {
      use(0);
      if (k + 2 < blocks) load(0);
      if (k + 1 < blocks) {
        use(1);
        if (k + 3 < blocks) load(1);
      }
    }
    for (int32_t k = k0 + blocks * U; k < k1; ++k, xq += 64) {
      const v4i t = *(const v4i*)xq;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const v4i v = __builtin_nontemporal_load((const v4i*)gw[i]);
        gw[i] += 64;
        acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(v, t, acc[i], 0, 0, 0);
      }
    }
    if (JOIN && next < slots) {  // the next slot's weights are on their way while this one's sums are put down
      aim(expert(next));
      if (blocks > 0) load(0);
      if (blocks > 1) load(1);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) red[((slot * 8 + wave) * RT + i) * 64 + lane] = acc[i];
    slot = next;
  }
  __syncthreads();

  // lane: column lane % 16 (all alike), channels 4 (lane / 16) .. + 3 of a block: column 0 writes
  if (row != 0) return;
  auto total = [&](int j, int i) {
    v4i sum = v4i{0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < WK; ++v) sum += red[((j * 8 + wn * WK + v) * RT + i) * 64 + lane];
    return sum;
  };
  if constexpr (JOIN) {
    if (wk != 0) return;
    const int32_t n = n0 + 4 * grp;
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < slots; ++j) {
      const int32_t e = expert(j);
      if (!there(e)) continue;
      const v4i sum = total(j, 0);
      const float s = scale(j).s, p = a.p[j];
      float sc[4];
      load_run<4>(a.sw + (int64_t)e * wrows, n, a.n, sc);
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = __builtin_fmaf(p, (float)sum[r] * s * sc[r], y[r]);
    }
    store_run<4>(a.y, a.y_dtype, 0, n, a.n, y);
  } else {
    const float s = scale(0).s;
    const float* sw = a.sw + (int64_t)expert(first) * wrows;
    for (int i = wk; i < (GATED ? 1 : RT); i += WK) {
      const int32_t n = n0 + 16 * i + 4 * grp;
      const v4i sum = total(0, i);
      float sc[4], b[4], v[4];
      load_run<4>(sw, n, a.n, sc);
      load_bias<4>(a.bias, n, a.n, b);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = (float)sum[r] * s * sc[r] + b[r];
      if constexpr (GATED) {
        const v4i up = total(0, 1);
        load_run<4>(sw + a.n, n, a.n, sc);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = silu(v[r]) * ((float)up[r] * s * sc[r]);
      }
      store_run<4>(a.y, a.y_dtype, (int64_t)first * a.n, n, a.n, v);
    }
  }
}

// ---------------------------------------------------------------- launches

// Weight rows per workgroup of the kernels that stream the weights: 64, 32 or 16, as many as leave most CUs a workgroup.
// One token, 14336 x 4096: 15.9 us with 64 rows, 16.9 with 32 and 18.1 with 16; 4096 x 4096: 13.9, 9.2 and 8.4 us.
inline int rows_per_group(int32_t n) { return n / 64 >= 192 ? 64 : n / 32 > 144 ? 32 : 16; }

template <int RT, int MT>
vq_status launch_few(const Q8Args& a, hipStream_t st) {
  const int64_t blocks = ((int64_t)a.n + RT * 16 - 1) / (RT * 16);
  if (!vqi::grid_ok(blocks, 512)) return VQ_ERR_SHAPE;
  q8_few_kernel<RT, MT><<<dim3((uint32_t)blocks), dim3(512), 0, st>>>(a);
  return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP;
}

template <int BM, int BN, int WM, int WN, int NB, int KG, bool GATED, bool SPLIT>
vq_status launch_tile(const Q8Args& a, hipStream_t st, bool check_only = false) {
  const int out = GATED ? BN / 2 : BN;
  const int64_t mt = a.experts ? span_bound(a, BM) : ((int64_t)a.m + BM - 1) / BM;
  const int64_t nt = ((int64_t)a.n + out - 1) / out;
  constexpr int kThreads = 64 * WM * WN * KG;
  if (!vqi::grid_ok(mt * nt + 8, kThreads)) return VQ_ERR_SHAPE;
  if (check_only) return VQ_OK;
  const uint32_t blocks = (uint32_t)((mt * nt + 7) / 8 * 8);
  q8_tile_kernel<BM, BN, WM, WN, NB, KG, GATED, SPLIT>
      <<<dim3(blocks, SPLIT ? a.splits : 1), dim3(kThreads), 0, st>>>(a, (int32_t)nt, (int32_t)mt);
  return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP;
}
vq_status launch_join(const Q8Args& a, hipStream_t st) {
  const int64_t items = (int64_t)a.m * ((a.n + 3) / 4);  // at most 128 tiles of 128 x 128: a small grid
  q8_join_kernel<<<dim3((uint32_t)((items + 255) / 256)), dim3(256), 0, st>>>(a);
  return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP;
}
template <bool GATED>
vq_status launch_big(const Q8Args& a, hipStream_t st, bool check_only = false) {
  const int out = GATED ? 128 : 256;
  const int64_t mt = a.experts ? span_bound(a, 256) : ((int64_t)a.m + 255) / 256;
  const int64_t nt = ((int64_t)a.n + out - 1) / out;
  const int64_t blocks = mt * nt + 128 + 8;  // at most 128 tiles are cut in two
  if (!vqi::grid_ok(blocks, 512)) return VQ_ERR_SHAPE;
  if (check_only) return VQ_OK;
  q8_big_kernel<GATED><<<dim3((uint32_t)blocks), dim3(512), 0, st>>>(a, (int32_t)nt, (int32_t)mt);
  return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP;
}

}  // namespace

namespace vqi {

namespace {
template <int RT, int WN, bool GATED, bool JOIN>
vq_status launch_one_t(const OneArgs& a, hipStream_t st) {
  const int out = WN * (GATED ? 16 : 16 * RT);
  const dim3 g((uint32_t)((a.n + out - 1) / out), GATED ? a.slots : 1);
  const size_t lds = (a.join ? a.slots : 1) * ((size_t)q8_row_bytes(a.k) + (size_t)8 * 64 * 16 * RT);
  if (!grid_ok(g.x, 512)) return VQ_ERR_SHAPE;
  if constexpr (JOIN) {  // the hidden rows are fp32
    q8_one_kernel<RT, WN, GATED, JOIN, VQ_F32><<<g, dim3(512), lds, st>>>(a);
  } else if (a.x_dtype == VQ_F32) {
    q8_one_kernel<RT, WN, GATED, JOIN, VQ_F32><<<g, dim3(512), lds, st>>>(a);
  } else if (a.x_dtype == VQ_F16) {
    q8_one_kernel<RT, WN, GATED, JOIN, VQ_F16><<<g, dim3(512), lds, st>>>(a);
  } else {
    q8_one_kernel<RT, WN, GATED, JOIN, VQ_BF16><<<g, dim3(512), lds, st>>>(a);
  }
  return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP;
}
}  // namespace

vq_status launch_q8_one(const OneArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  if (a.gated) return launch_one_t<2, 1, true, false>(a, st);
  if (a.join) return launch_one_t<1, 1, false, true>(a, st);
  switch (rows_per_group(a.n)) {
    case 64: return launch_one_t<2, 2, false, false>(a, st);
    case 32: return launch_one_t<2, 1, false, false>(a, st);
    default: return launch_one_t<1, 1, false, false>(a, st);
  }
}

// How a dense product is computed.  kStreamed: q8_few_kernel.  The tiles differ in rows x columns and in the steps kept
// in LDS: one step of a tile takes about a microsecond to arrive, so a CU with one workgroup moves what the workgroup
// has on its way in that time.
namespace {
enum Way { kStreamed, k64x32, k64x64, k128x64, k128x128, k128x128Pair, k256x256 };
struct Plan {
  Way way;
  int32_t splits;  // cuts of K over the CUs
};
// Few rows are streamed as long as that costs less than the tiles' fixed part, several steps of a microsecond.  It grows
// with what the busiest CU does: its blocks of 16 weight rows, times the steps of K, times the weights and each block of
// 16 tokens.  us, streamed and in tiles, weights from memory:
//   one block, tokens x steps: 1030 x 777, 64 rows 4.9 and 5.2; 2500 x 2048, 32 rows 5.6 and 6.2, 48 rows 6.7 and 6.3;
//     4096 x 4096, 32 rows 8.4 and 9.4, 48 rows 10.4 and 10.0; 1030 x 5120, 16 rows 8.6 and 10.2, 32 rows 11.0 and 10.0
//   two: 4500 x 777, 32 rows 5.6 and 5.5, 48 rows 6.7 and 5.4; 7000 x 2048, 16 rows 6.2 and 7.6; 6144 x 4096, 16 rows
//     9.5 and 9.4; 7000 x 5120, 16 rows 14.5 and 11.7; where all CUs are at work 8192 x 8192, 2 rows 17.1 and 19.5, 8 rows
//     17.9 and 19.5, 16 rows 19.2 and 19.5 (7300 x 5120, 2 rows 14.3 and 12.5: steps left over from blocks of four)
//   four: 9000 x 2048, 2 rows 8.2 and 8.8, 16 rows 9.2 and 8.6; 11008 x 4096, 2 rows 15.2 and 14.7, 16 rows 16.9 and
//     13.5; wider ones: 14336 x 2048, 2 rows 9.6 and 9.2; 28672 x 8192, 16 rows 62 and 48
//   few columns with a long K, which the tiles cut over the CUs: 256 x 8192, 2 rows 8.0 and 7.0
bool streamed(int32_t m, int32_t n, int64_t steps) {
  if (m > 64 || (n < 1024 && steps >= 56)) return false;
  const int32_t tokens = (m + 15) / 16;
  const int32_t wide = rows_per_group(n);
  const int64_t groups = ((int64_t)n + wide - 1) / wide;
  const int64_t blocks = (groups + 255) / 256 * (wide / 16);
  if (blocks == 1) return tokens * steps <= 64 && (tokens <= 2 || steps <= 8);
  if (blocks == 2)
    return (tokens == 1 && steps <= 32) || (tokens == 2 && steps <= 8) || (m <= 8 && steps <= 64 && groups > 224);
  return wide == 32 && m <= 8 && steps <= 16;
}

Plan dense_plan(int32_t m, int32_t n, int32_t k) {
  const int64_t steps = q8_row_bytes(k) / kStep;
  if (streamed(m, n, steps)) return {kStreamed, 1};
  auto tiles = [&](int bm, int bn) { return (((int64_t)m + bm - 1) / bm) * (((int64_t)n + bn - 1) / bn); };
  // K is cut where the tiles leave CUs without work, if it is long enough to pay for the second launch (the int32 partial
  // sums), and then over as many CUs as find 8 steps each
  auto cut = [&](int64_t t) {
    return steps < 56 ? 1 : (int32_t)std::max<int64_t>(1, std::min<int64_t>(256 / t, steps / 8));
  };
  const int64_t narrow = tiles(64, 32), small = tiles(64, 64), tall = tiles(128, 64), wide = tiles(128, 128);
  // All us below: one run, weights from memory, / 4 for a K cut in 4 (with the join).
  // 512 x 28672 x 8192 (224 tiles): 122 against 154 in 128 x 128; 2048 x 8192 x 2048 (256): 38 and 47; 1024 x 8192 x 8192
  // (128): 87 and 78; 1500 x 4096 x 4096 (96): 40 and 36
  if (tiles(256, 256) >= 200) return {k256x256, 1};
  // at most one for each CU, with two groups of wavefronts that halve K, against 64 x 64: 37 x 5003 x 4099 10.7 and 12.4 / 3,
  // 128 x 4096 x 4096 10.7 and 12.8, 200 x 2000 x 3000 8.4 and 9.9, 64 x 8192 x 8192 23.0 and 23.2 / 2; 300 x 2500 x 2500
  // (395 of them) 13.1 and 9.5; longer K: 64 x 4096 x 14336 29 and 20 / 4, 64 x 8192 x 28672 64 and 53 / 2
  if (narrow <= 256 && steps < (narrow > 128 ? 100 : 56)) return {k64x32, 1};
  // 256 x 4096 x 4096: 13.1 against 17.5 in 128 x 64 and 21 / 4 in 128 x 128; 64 x 4096 x 14336: 20.0 / 4, 37 uncut;
  // longer K: 128 x 8192 x 28672 78 against 61 / 4 in 128 x 128
  if (m <= 64 || (small <= 256 && steps < (small > 128 ? 100 : 128))) return {k64x64, cut(small)};
  // against 64 x 64 and 128 x 128: 128 x 14336 x 4096 20.6, 23.7 and 25 / 2; 256 x 8192 x 8192 33.5, 38.5 and 35 / 2;
  // 512 x 4096 x 4096 17.6, 19.3 and 22.5; more than one round: 300 x 6500 x 2048 (306 tiles) 13.8, 10.9 and 14.9
  if (tall >= 160 && tall <= 256 && steps < 128) return {k128x64, 1};
  // against 128 x 128: 320 x 6500 x 3000 17.9 and 19.1; 300 x 6500 x 4900 (39 steps) 25.3 and 25.6; 400 x 5000 x 5120 (40)
  // 33.2 and 27.0.  With few rows 128 x 64 would be nearer: 128 x 9300 x 3000 19.1, 17.0 there
  if (small <= 512 && steps < 40) return {k64x64, 1};
  // one workgroup per CU and three steps in LDS, or two workgroups and two steps: 128 x 28672 x 8192 (224 tiles) 60.5
  // and 66.2; 700 x 7000 x 3000 (330) 36.6 and 29.0; 512 x 14336 x 4096 (448) 48.5 and 42.8
  if (wide <= 256) return {k128x128, cut(wide)};
  return {k128x128Pair, 1};
}
}  // namespace

int32_t q8_splits(int32_t m, int32_t n, int32_t k) { return dense_plan(m, n, k).splits; }

vq_status launch_q8(const Q8Args& a, void* stream, bool check_only) {  // check_only: the grouped product
  hipStream_t st = (hipStream_t)stream;
  if (a.experts) {
    // Rows of a group on average (in the larger of max_rows' bound): short groups take small tiles, in between the plain
    // product takes 128-row tiles while the CUs hold them all at once.  us, gated and plain product in 32-, 64-, 128- and
    // 256-row tiles, rows of a group on average in front:
    //   64 experts of 2048 x 1024     21: 51 + 29, 50 + 33, 58 + 37, 61 + 41      75: 90 + 46, 77 + 48, 88 + 59, 79 + 65
    //                                125: 124 + 62, 101 + 60, 104 + 70, 105 + 83  188: 167 + 84, 128 + 78, 132 + 86, 117 + 92
    //    8 experts of 4096 x 14336     4: 159 + 110, 167 + 113, 179 + 118, 181 + 139
    //      (plain: 256 tiles of 128)  50: 265 + 159, 227 + 129, 235 + 132, 223 + 159
    //                                125: 445 + 238, 332 + 159, 321 + 143, 280 + 183   250: 625 + 345, 520 + 296, 444 + 250, 384 + 195
    //   32 experts of 1536 x 5000    100: 212 + 99, 177 + 88, 188 + 99, 176 + 76
    const int64_t groups = a.m < a.experts ? a.m : a.experts;
    const int64_t avg = (a.m + groups - 1) / groups;
    if (a.gated) {
      if (avg <= 4) return launch_tile<32, 128, 1, 2, 2, 1, true, false>(a, st, check_only);
      return avg <= 96 ? launch_tile<64, 128, 2, 2, 2, 1, true, false>(a, st, check_only)
                       : launch_big<true>(a, st, check_only);
    }
    if (avg <= 48) return launch_tile<32, 128, 1, 4, 2, 1, false, false>(a, st, check_only);
    if (avg > 192) return launch_big<false>(a, st, check_only);
    return (avg + 127) / 128 * groups * (((int64_t)a.n + 127) / 128) <= 256
               ? launch_tile<128, 128, 2, 2, 2, 1, false, false>(a, st, check_only)
               : launch_tile<64, 128, 2, 2, 2, 1, false, false>(a, st, check_only);
  }
  switch (dense_plan(a.m, a.n, a.k).way) {
    case kStreamed:  // groups of 32 weight rows take 32 tokens at most, 64 none (streamed)
      if (rows_per_group(a.n) > 16) return a.m <= 16 ? launch_few<2, 1>(a, st) : launch_few<2, 2>(a, st);
      if (a.m <= 16) return launch_few<1, 1>(a, st);
      if (a.m <= 32) return launch_few<1, 2>(a, st);
      return a.m <= 48 ? launch_few<1, 3>(a, st) : launch_few<1, 4>(a, st);
    case k64x32: return launch_tile<64, 32, 2, 1, 4, 2, false, false>(a, st);
    case k64x64: {
      if (a.splits == 1) return launch_tile<64, 64, 2, 2, 4, 1, false, false>(a, st);
      const vq_status e = launch_tile<64, 64, 2, 2, 4, 1, false, true>(a, st);
      return e != VQ_OK ? e : launch_join(a, st);
    }
    case k128x64: return launch_tile<128, 64, 2, 2, 3, 1, false, false>(a, st);
    case k128x128: {
      if (a.splits == 1) return launch_tile<128, 128, 2, 2, 3, 1, false, false>(a, st);
      const vq_status e = launch_tile<128, 128, 2, 2, 3, 1, false, true>(a, st);
      return e != VQ_OK ? e : launch_join(a, st);
    }
    case k128x128Pair: return launch_tile<128, 128, 2, 2, 2, 1, false, false>(a, st);
    case k256x256: return launch_big<false>(a, st);
  }
  return VQ_ERR_UNSUPPORTED;
}

}  // namespace vqi
