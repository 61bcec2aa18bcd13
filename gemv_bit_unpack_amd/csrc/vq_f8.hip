// The 8-bit float products: y[m][n] = sum_b s[b][m] sw[n / 128][b] sum_{k in block b} q[m][k] w[n][k] (+ bias[n]), with
// e4m3 values and one fp32 scale for each 128 columns of a token and each 128 x 128 block of the weights; the gated form
// y = silu(g) u of two such products; and the cutting of tokens and weights to e4m3.
//
// A block of K is one matrix instruction deep (16 x 16 x 128), so its sum leaves the matrix pipe once, in fp32, and is
// added to the output's fp32 sum with the product of its two scales: one fused multiply-add per output and block, beside
// 128 multiply-adds of the matrix pipe.  That is half of the vector pipe's time under the matrix pipe's whole.
//
// Rows of q and w are whole 128-byte steps with zero pads, so no kernel has a K edge; rows past an edge of a tile read the
// last valid row again and are not stored.  A sum's order is fixed by the shape (waves, then K splits, in order): equal
// calls give equal bits, calls of different shapes may differ in the last ones.
#include <algorithm>

#include "vq_device.h"
#include "vq_f8_device.h"
#include "vq_q8_device.h"
#include "vq_tile_device.h"

namespace {

using vqi::F8Args;
using vqi::F8QuantArgs;
using vqt::load_bias;
using vqt::load_run;
using vqt::meet;
using vqt::place;
using vqt::silu;
using vqt::store_run;
using vqt::tile_at;
using vqt::to_lds;

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 128;  // bytes of K per step: one block
static_assert(kStep == vqi::kF8Block, "a step is a block");

// 16 rows of w times 16 rows of q over one block, both e4m3: lane l gives bytes 16 (l / 16) .. + 15 and 64 further on of
// row l % 16 (any order of K will do that is the same for both), and holds the sums of token l % 16 with weight rows
// 4 (l / 16) .. + 3.
//
// Two forms.  The 8-bit instruction adds 8 products at a time after cutting them at 2^-13 of the largest one's power of
// two: measured on unit-normal tokens and weights, a block's sum is off by 1.4e-5 of its spread (5.7e-5 where the
// magnitudes of the tokens spread over 2^16), nothing beside the half step of a 16-bit output (2^-9, 2^-12), but 200 times
// what fp32 sums are off by.  WIDE: the operands go to fp16, which holds every e4m3 value, and the 16-bit instruction adds
// their products in fp32 (1e-8), at half the rate.
template <bool WIDE>
struct Frag {
  v8i v;
};
template <>
struct Frag<true> {
  h8 v[4];
};
__device__ __forceinline__ h8 widen(int lo, int hi) {
  const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  const h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
template <bool WIDE>
__device__ __forceinline__ Frag<WIDE> join(v4i lo, v4i hi) {
  Frag<WIDE> f;
  if constexpr (WIDE) {
    f.v[0] = widen(lo[0], lo[1]);
    f.v[1] = widen(lo[2], lo[3]);
    f.v[2] = widen(hi[0], hi[1]);
    f.v[3] = widen(hi[2], hi[3]);
  } else {
    f.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  return f;
}
template <bool WIDE>
__device__ __forceinline__ v4f multiply(const Frag<WIDE>& w, const Frag<WIDE>& t) {
  v4f p = v4f{0.f, 0.f, 0.f, 0.f};
  if constexpr (WIDE) {
#pragma unroll
    for (int h = 0; h < 4; ++h) p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.v[h], t.v[h], p, 0, 0, 0);
  } else {
    p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, t.v, p, 0, 0, 0, 0, 0, 0);
  }
  return p;
}

// ---------------------------------------------------------------- to 8 bits

// Tokens: 16 lanes take a block of 128 columns, 8 each; a workgroup 16 rows by 4 blocks, all of its loads on their way
// before the first is used.
constexpr int kQuantCols = 4;
template <vq_dtype XT>
__global__ __launch_bounds__(256) void f8_tokens_kernel(F8QuantArgs a) {
  const int lane16 = threadIdx.x & 15;
  const int32_t row = (int32_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (row >= a.rows) return;  // 16 lanes at once: the others' shuffles stay inside their own 16
  constexpr int es = XT == VQ_F32 ? 4 : 2;
  const void* x = (const char*)a.x + (int64_t)row * a.ldx * es;
  const int64_t ld = vqi::q8_row_bytes(a.k);
  const int32_t blocks = (int32_t)(ld / kStep);
  const int32_t b0 = (int32_t)blockIdx.y * kQuantCols;
  float f[kQuantCols][8];
#pragma unroll
  for (int c = 0; c < kQuantCols; ++c) vqd::load_f32<XT, 8>(x, (b0 + c) * kStep + lane16 * 8, a.k, f[c]);
#pragma unroll
  for (int c = 0; c < kQuantCols; ++c) {
    if (b0 + c >= blocks) break;
    uint32_t big = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) big = max(big, vqd::abs_bits(f[c][k]));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) big = max(big, (uint32_t)__shfl_xor((int)big, o, 64));
    const vqd::Q8Scale sc = vqd::f8_scale(big);
    const uint2 v = make_uint2(vqd::f8_pack4(f[c], sc), vqd::f8_pack4(f[c] + 4, sc));
    *(uint2*)(a.q + (int64_t)row * ld + (b0 + c) * kStep + lane16 * 8) = v;
    if (lane16 == 0) a.s[(int64_t)(b0 + c) * a.rows + row] = sc.s;
  }
}

// Weights: a workgroup takes a block of 128 rows and columns, once for its largest value and once for its bytes.
template <vq_dtype XT>
__global__ __launch_bounds__(256) void f8_weights_kernel(F8QuantArgs a) {
  __shared__ uint32_t part[4];
  const int32_t kb = (int32_t)blockIdx.x, nb = (int32_t)blockIdx.y;
  const int col = (threadIdx.x & 15) * 8, row0 = nb * 128 + (threadIdx.x >> 4);
  constexpr int es = XT == VQ_F32 ? 4 : 2;
  const int32_t end = min(a.rows, nb * 128 + 128);
  uint32_t big = 0;
  float f[8][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int32_t r = row0 + 16 * j;
    vqd::load_f32<XT, 8>((const char*)a.x + (int64_t)min(r, end - 1) * a.ldx * es, kb * kStep + col, a.k, f[j]);
#pragma unroll
    for (int k = 0; k < 8; ++k) big = max(big, vqd::abs_bits(f[j][k]));  // a row past the end repeats the last one
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) big = max(big, (uint32_t)__shfl_xor((int)big, o, 64));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = big;
  __syncthreads();
  const vqd::Q8Scale sc = vqd::f8_scale(max(max(part[0], part[1]), max(part[2], part[3])));
  const int64_t ld = vqi::q8_row_bytes(a.k);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int32_t r = row0 + 16 * j;
    if (r < end)
      *(uint2*)(a.q + (int64_t)r * ld + kb * kStep + col) =
          make_uint2(vqd::f8_pack4(f[j], sc), vqd::f8_pack4(f[j] + 4, sc));
  }
  if (threadIdx.x == 0) a.s[(int64_t)nb * gridDim.x + kb] = sc.s;
}

// ---------------------------------------------------------------- tiles

// 4 bytes per lane from `g` to LDS at the wavefront's `l` + 4 lane.
__device__ __forceinline__ void to_lds4(const float* g, uint8_t* l) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                   (__attribute__((address_space(3))) void*)l, 4, 0, 0);
}

// LDS of a tile: NB steps of its rows and its tokens' scales, the scales of the weights' blocks (two rows of at most 512),
// and the tokens' largest values of the 8-bit epilogue.
template <int BM, int BN, int NB>
constexpr int kTileLds = NB * ((BM + BN) * kStep + BM * 4);

// One tile: WM x WN wavefronts compute BM rows (row0 ..) by BN weight rows (with the gate: BN / 2 outputs).  Each
// wavefront's weight rows are 16 NI consecutive ones (8 NI outputs of gate and up rows with the gate), dealt to its NI
// blocks so that a lane ends with 4 NI (2 NI) consecutive outputs of one token.
// OUTQ: the outputs in 8 bits (with the gate, BN / 2 = 128 outputs: one block).
template <int BM, int BN, int WM, int WN, int NB, bool WIDE, bool GATED, bool SPLIT, bool OUTQ>
__device__ __forceinline__ void tile(const F8Args& a, int32_t row0, int32_t n0, uint8_t* lds, float* sbs, float* tops) {
  constexpr int kWaves = WM * WN;
  constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  constexpr int NO = GATED ? NI / 2 : NI;  // blocks of outputs
  constexpr int TL = BM / 8 / kWaves, WL = BN / 8 / kWaves;  // 8-row loads per wavefront and step
  constexpr int SG = (BM + 63) / 64;                         // groups of 64 token scales
  constexpr int kRows = (BM + BN) * kStep;
  constexpr int kBuf = kRows + BM * 4;
  constexpr int kLater = (NB - 2) * (TL + WL + 1);
  static_assert(NB >= 2 && kLater < 64, "the wait counter holds 6 bits");
  constexpr int kWaitNext = 0x0070 | (kLater & 15) | (kLater >> 4) << 14;  // and lgkmcnt(0)
  static_assert(TL * 8 * kWaves == BM && WL * 8 * kWaves == BN, "whole loads");
  static_assert(BM % 64 == 0 && SG <= kWaves, "each wavefront loads one group of scales");
  static_assert(!GATED || NI % 2 == 0, "gate and up blocks in one wavefront");
  static_assert(!OUTQ || (GATED && BN == 256 && WN * NO * 16 == 128), "a block of outputs per tile");

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int col = lane & 15, grp = lane >> 4;
  const int64_t ld = vqi::q8_row_bytes(a.k);
  const int32_t blocks = (int32_t)(ld / kStep);
  const int32_t end = min(a.m, row0 + BM);

  int32_t kt0 = 0, kt1 = blocks;
  if constexpr (SPLIT) {
    kt0 = (int32_t)((int64_t)blocks * blockIdx.y / a.splits);
    kt1 = (int32_t)((int64_t)blocks * (blockIdx.y + 1) / a.splits);
  }
  const int32_t n = kt1 - kt0;

  // this lane's 16-byte piece of every load: row p of the tile, chunk lane % 8 of its LDS row, which holds chunk
  // (lane % 8) ^ (p / 2 % 8) of the matrix row (reads of 16 rows at one chunk then fall on all 64 banks)
  const uint8_t* gt[TL];
  const uint8_t* gw[WL];
#pragma unroll
  for (int j = 0; j < TL; ++j) {
    const int p = (j * kWaves + wave) * 8 + (lane >> 3);
    gt[j] = a.q + (int64_t)min(row0 + p, end - 1) * ld + kt0 * kStep + (((lane & 7) ^ ((p >> 1) & 7)) * 16);
  }
#pragma unroll
  for (int j = 0; j < WL; ++j) {
    const int p = (j * kWaves + wave) * 8 + (lane >> 3);
    const int pw = p / (16 * NI), pj = p / 16 % NI, pi = p & 15;  // wavefront, its block, the block's row
    const int o = pw * 16 * NO + (pi >> 2) * 4 * NO + 4 * (pj % NO) + (pi & 3);
    const int64_t r = (int64_t)min(n0 + o, a.n - 1) + (GATED && pj >= NO ? a.n : 0);
    gw[j] = a.w + r * ld + kt0 * kStep + (((lane & 7) ^ ((p >> 1) & 7)) * 16);
  }
  const float* gs = a.s + (int64_t)kt0 * a.m + min(row0 + wave % SG * 64 + lane, end - 1);
  auto fetch = [&](int buf) {
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
    to_lds4(gs, lds + buf * kBuf + kRows + wave % SG * 256);  // some twice, the same values
    gs += a.m;
  };
#pragma unroll
  for (int b = 0; b < NB - 1; ++b)
    if (b < n) fetch(b);

  // the weights' scales of the steps: with the gate a row for each half, else one for each 128 weight rows
  const int32_t nblocks = (int32_t)vqi::f8_blocks(a.n);
  constexpr int kScaleRows = GATED || BN > 128 ? 2 : 1;
  for (int32_t i = threadIdx.x; i < n * kScaleRows; i += 64 * kWaves) {
    const int32_t r = i / n, k = i - r * n;
    const int32_t nb = GATED ? n0 / 128 + r * nblocks : min(n0 / 128 + r, nblocks - 1);
    sbs[r * 512 + k] = a.sw[(int64_t)nb * blocks + kt0 + k];
  }
  const float* const sb0 = sbs + (GATED ? 0 : (n0 % 128 + wn * 16 * NI) / 128 * 512);

  v4f acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  const int lt = (wm * MI * 16 + col) * kStep;
  const int lw = BM * kStep + (wn * NI * 16 + col) * kStep;
  const int c0 = (grp ^ ((col >> 1) & 7)) * 16;
  auto frag = [&](int at) { return join<WIDE>(*(const v4i*)(lds + at + c0), *(const v4i*)(lds + at + (c0 ^ 64))); };

  if (NB - 1 <= n) {
    __builtin_amdgcn_s_waitcnt(kWaitNext);  // this wavefront's part of the first step is in LDS
  } else {
    __builtin_amdgcn_s_waitcnt(0x0070);
  }
  __syncthreads();  // and everyone's, and the scales
  if (NB - 1 < n) fetch(NB - 1);
  int buf = 0;
  for (int32_t kt = 0; kt < n; ++kt) {
    const int at = buf * kBuf;
    Frag<WIDE> w[NI], t[2];
#pragma unroll
    for (int j = 0; j < NI; ++j) w[j] = frag(at + lw + j * 16 * kStep);
    t[0] = frag(at + lt);
    const float sg = sb0[kt], su = GATED ? sbs[512 + kt] : 0.f;
    float s[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) s[i] = *(const float*)(lds + at + kRows + (wm * MI * 16 + i * 16 + col) * 4);
    v4f p[2][NI];
    auto add = [&](int i) {
      const float s0 = s[i] * sg, s1 = s[i] * su;
#pragma unroll
      for (int j = 0; j < NI; ++j) {
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[i & 1][j][r], GATED && j >= NO ? s1 : s0, acc[i][j][r]);
        asm volatile("" : "+v"(acc[i][j]));  // here, and not after the step's last product
      }
    };
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (i + 1 < MI) t[(i + 1) & 1] = frag(at + lt + (i + 1) * 16 * kStep);
#pragma unroll
      for (int j = 0; j < NI; ++j) p[i & 1][j] = multiply<WIDE>(w[j], t[i & 1]);
      if (i > 0) add(i - 1);
      // the row's fragment on its way first, then each product with its share of the additions of the row before
      if (i + 1 < MI) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        __builtin_amdgcn_sched_group_barrier(0x008, WIDE ? 4 : 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 4 + (WIDE ? 4 : 0), 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    add(MI - 1);
    if (kt + 1 < n) {
      // its part of the next step is in LDS (steps after that may still be on their way), its last reads are done
      if (kt + NB - 1 < n) {
        __builtin_amdgcn_s_waitcnt(kWaitNext);
      } else {
        __builtin_amdgcn_s_waitcnt(0x0070);
      }
      meet();  // and everyone's: the next step may be read, this one overwritten
      if (kt + NB < n) fetch(buf);
      buf = buf + 1 == NB ? 0 : buf + 1;
    }
  }

  // outputs: lane = token row0 + .., 4 NO consecutive channels
  const int32_t nw = n0 + wn * 16 * NO + grp * 4 * NO;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int32_t m = row0 + wm * MI * 16 + i * 16 + col;
    float v[4 * NO];
#pragma unroll
    for (int j = 0; j < NO; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[4 * j + r] = acc[i][j][r];
    if constexpr (SPLIT) {
      if (m < end) store_run<4 * NO>(a.part, VQ_F32, ((int64_t)blockIdx.y * a.m + m) * a.n, nw, a.n, v);
    } else {
      if (a.bias) {
        float b[4 * NO];
        load_bias<4 * NO>(a.bias, nw, a.n, b);
#pragma unroll
        for (int r = 0; r < 4 * NO; ++r) v[r] += b[r];
      }
      if constexpr (GATED) {
        float u[4 * NO];
#pragma unroll
        for (int j = 0; j < NO; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) u[4 * j + r] = acc[i][NO + j][r];
        if (a.bias) {
          float b[4 * NO];
          load_bias<4 * NO>(a.bias + a.n, nw, a.n, b);
#pragma unroll
          for (int r = 0; r < 4 * NO; ++r) u[r] += b[r];
        }
#pragma unroll
        for (int r = 0; r < 4 * NO; ++r) v[r] = silu(v[r]) * u[r];
      }
      if constexpr (OUTQ) {
        uint32_t big = 0;
#pragma unroll
        for (int r = 0; r < 4 * NO; ++r) {
          if (nw + r >= a.n) v[r] = 0.f;
          acc[i][r / 4][r % 4] = v[r];
          big = max(big, vqd::abs_bits(v[r]));
        }
        big = max(big, (uint32_t)__shfl_xor((int)big, 16, 64));
        big = max(big, (uint32_t)__shfl_xor((int)big, 32, 64));
        if (grp == 0) tops[wn * BM + wm * MI * 16 + i * 16 + col] = __builtin_bit_cast(float, big);
      } else {
        if (m < end) store_run<4 * NO>(a.y, a.y_dtype, (int64_t)m * a.n, nw, a.n, v);
      }
    }
  }
  if constexpr (OUTQ) {
    __syncthreads();
    const int64_t ldq = vqi::q8_row_bytes(a.n);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int at = wm * MI * 16 + i * 16 + col;
      uint32_t big = 0;
#pragma unroll
      for (int k = 0; k < WN; ++k) big = max(big, __builtin_bit_cast(uint32_t, tops[k * BM + at]));
      const vqd::Q8Scale sc = vqd::f8_scale(big);
      uint32_t v[NO];
#pragma unroll
      for (int j = 0; j < NO; ++j) {
        const float f[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        v[j] = vqd::f8_pack4(f, sc);
      }
      if (row0 + at < end) {
        __builtin_memcpy(a.yq + (int64_t)(row0 + at) * ldq + nw, v, 4 * NO);
        if (wn == 0 && grp == 0) a.ys[(int64_t)(n0 / 128) * a.m + row0 + at] = sc.s;
      }
    }
  }
}

template <int BM, int BN, int WM, int WN, int NB, bool WIDE, bool GATED, bool SPLIT>
__global__ __launch_bounds__(64 * WM * WN) void f8_tile_kernel(F8Args a, int32_t nt, int32_t mt_count) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kTileLds<BM, BN, NB>];
  __shared__ float sbs[(GATED || BN > 128 ? 2 : 1) * 512];
  int32_t mt, nti;
  if (!place((int32_t)blockIdx.x, mt_count * nt, mt_count, nt, mt, nti)) return;
  tile<BM, BN, WM, WN, NB, WIDE, GATED, SPLIT, false>(a, mt * BM, nti * (GATED ? BN / 2 : BN), lds, sbs, nullptr);
}

// 8 wavefronts, one workgroup per CU: 256 x 256 tiles, or 128 x 256 ones where the operands go to fp16 (their fragments
// take twice the registers).  256 x 256: 128 rows only where the matrix's last tile has no more left, and in the last round
// over the 256 CUs if at most half of them have a tile in it: two half tiles for each then take half a round.
template <bool WIDE, bool GATED, bool OUTQ>
__global__ __launch_bounds__(512) void f8_big_kernel(F8Args a, int32_t nt, int32_t mt_count) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[WIDE ? kTileLds<128, 256, 3> : kTileLds<256, 256, 2>];
  __shared__ float sbs[2 * 512];
  __shared__ float tops[OUTQ ? 4 * (WIDE ? 128 : 256) : 1];
  const int32_t total = mt_count * nt;
  const int32_t id = (int32_t)blockIdx.x;
  int32_t mt, nti, part = 0;
  if constexpr (WIDE) {
    if (!place(id, total, mt_count, nt, mt, nti)) return;
    tile<128, 256, 2, 4, 3, true, GATED, false, OUTQ>(a, mt * 128, nti * (GATED ? 128 : 256), lds, sbs, tops);
  } else {
    const int32_t rest = total % 256;
    const int32_t full = rest <= 128 ? total - rest : total;  // ids from the next multiple of 8 on are halves
    const int32_t whole = (full + 7) / 8 * 8;
    const bool half = id >= whole;
    if (half) {
      const int32_t at = full + (id - whole) / 2;
      if (at >= total) return;
      part = (id - whole) & 1;
      tile_at(at, mt_count, nt, mt, nti);
    } else if (!place(id, full, mt_count, nt, mt, nti)) {
      return;
    }
    const int32_t row0 = mt * 256 + part * 128, n0 = nti * (GATED ? 128 : 256);
    if (row0 >= a.m) return;
    if (half || a.m - row0 <= 128) {
      tile<128, 256, 2, 4, 2, false, GATED, false, OUTQ>(a, row0, n0, lds, sbs, tops);
    } else {
      tile<256, 256, 2, 4, 2, false, GATED, false, OUTQ>(a, row0, n0, lds, sbs, tops);
    }
  }
}

// y = the sum of the K splits, in order, + bias: 4 outputs per thread.
__global__ __launch_bounds__(256) void f8_join_kernel(F8Args a) {
  const int32_t groups = (a.n + 3) / 4;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (int64_t)a.m * groups) return;
  const int32_t m = (int32_t)(id / groups);
  const int32_t n = (int32_t)(id - (int64_t)m * groups) * 4;
  const int64_t apart = (int64_t)a.m * a.n;
  const float* p = a.part + (int64_t)m * a.n + n;
  float v[4] = {0.f, 0.f, 0.f, 0.f}, b[4];
  if (n + 4 <= a.n) {
#pragma unroll 8
    for (int32_t k = 0; k < a.splits; ++k) {
      float f[4];
      __builtin_memcpy(f, p + k * apart, 16);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += f[r];
    }
  } else {
    for (int32_t k = 0; k < a.splits; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += n + r < a.n ? p[k * apart + r] : 0.f;
  }
  load_bias<4>(a.bias, n, a.n, b);
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] += b[r];
  store_run<4>(a.y, a.y_dtype, (int64_t)m * a.n, n, a.n, v);
}

// ---------------------------------------------------------------- few rows

// Few tokens: the weights are read once, straight into the matrix instruction's registers.  A workgroup of 8 wavefronts
// takes RT blocks of 16 weight rows (with the gate RT / 2 blocks of gate rows and as many of up rows) and up to 16 MT
// tokens; its wavefronts cut K, their sums meet in LDS.  Two sets of U steps are in registers, one on its way while the
// other is used; the steps of a last, partial set are loaded again from the last one and left out.
// XT >= 0: the tokens come as they are and each wavefront cuts its own part of K to 8 bits, in LDS, while its first weights
// are on their way: a block's scale needs no other wavefront, so there is no barrier and no launch in front.
template <int RT, int MT, bool GATED, int XT>
__global__ __launch_bounds__(512) void f8_few_kernel(F8Args a) {
  constexpr bool CUT = XT >= 0;
  static_assert(!CUT || MT == 1, "tokens of one block");
  static_assert(!GATED || RT % 2 == 0, "gate and up blocks");
  constexpr int NO = GATED ? RT / 2 : RT;
  constexpr int kTiles = RT * MT;
  constexpr int U = kTiles == 1 ? 4 : kTiles <= 4 ? 2 : 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // [8][kTiles][64] v4f, then the cut tokens

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, grp = lane >> 4;
  const int32_t n0 = (int32_t)blockIdx.x * 16 * NO;
  const int64_t ld = vqi::q8_row_bytes(a.k);
  const int32_t blocks = (int32_t)(ld / kStep);
  const int32_t k0 = (int32_t)((int64_t)blocks * wave / 8), k1 = (int32_t)((int64_t)blocks * (wave + 1) / 8);
  v4f* const red = (v4f*)lds;

  v4f acc[RT][MT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  if (k0 < k1) {
    const uint8_t* gw[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int64_t r = (int64_t)min(n0 + 16 * (i % NO) + row, a.n - 1) + (i >= NO ? a.n : 0);
      gw[i] = a.w + r * ld + grp * 16;
    }
    const uint8_t* gt[MT];
    const float* gs[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int32_t m = min(16 * j + row, a.m - 1);
      gt[j] = CUT ? nullptr : a.q + (int64_t)m * ld + grp * 16;
      gs[j] = CUT ? nullptr : a.s + m;
    }
    // the weights' scales of this wavefront's steps (64 at most), one per lane
    const int32_t nblocks = (int32_t)vqi::f8_blocks(a.n);
    const float* sw = a.sw + (int64_t)(n0 / 128) * blocks + min(k0 + lane, k1 - 1);
    const float sg = sw[0], su = GATED ? sw[(int64_t)nblocks * blocks] : 0.f;

    // the tokens' part of this wavefront, in chunks of 16: chunk c is columns 16 (c % 8) .. of step k0 + c / 8
    constexpr vq_dtype XD = CUT ? (vq_dtype)XT : VQ_F32;
    const int32_t chunks = (k1 - k0) * 8;
    float first[CUT ? 16 : 1];
    if constexpr (CUT) {
      // the first ones are asked for before the weights, which then arrive behind them
      if (lane < chunks) vqd::load_f32<XD, 16>(a.x, k0 * kStep + lane * 16, a.k, first);
      __builtin_amdgcn_sched_barrier(0);
    }

    v4i w[2][U][RT][2], t[2][CUT ? 1 : U][MT][2];
    float ts[2][CUT ? 1 : U][MT];
    auto load = [&](int set, int32_t at) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int32_t k = min(at + u, k1 - 1);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            w[set][u][i][h] = __builtin_nontemporal_load((const v4i*)(gw[i] + (int64_t)k * kStep + 64 * h));
        if constexpr (!CUT) {
#pragma unroll
          for (int j = 0; j < MT; ++j) {
#pragma unroll
            for (int h = 0; h < 2; ++h) t[set][u][j][h] = *(const v4i*)(gt[j] + (int64_t)k * kStep + 64 * h);
            ts[set][u][j] = gs[j][(int64_t)k * a.m];
          }
        }
      }
    };
    const int32_t sets = (k1 - k0 + U - 1) / U;
    load(0, k0);
    if (sets > 1) load(1, k0 + U);
    __builtin_amdgcn_sched_barrier(0);

    uint8_t* const xq = lds + 8 * kTiles * 1024 + (int64_t)k0 * a.m * (kStep + 4);  // [steps][m][128], [steps][m] scales
    float* const xs = (float*)(xq + (int64_t)(k1 - k0) * a.m * kStep);
    if constexpr (CUT) {
      for (int32_t m = 0; m < a.m; ++m) {
        const void* x = (const char*)a.x + (int64_t)m * a.ldx * (XD == VQ_F32 ? 4 : 2);
        for (int32_t c = lane; c < (chunks + 63) / 64 * 64; c += 64) {
          float f[16];
          if (m == 0 && c < 64) {
#pragma unroll
            for (int k = 0; k < 16; ++k) f[k] = first[k];
          } else if (c < chunks) {
            vqd::load_f32<XD, 16>(x, k0 * kStep + c * 16, a.k, f);
          }
          uint32_t big = 0;
#pragma unroll
          for (int k = 0; k < 16; ++k) big = max(big, vqd::abs_bits(f[k]));
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) big = max(big, (uint32_t)__shfl_xor((int)big, o, 64));
          if (c < chunks) {  // 8 lanes at once
            const vqd::Q8Scale sc = vqd::f8_scale(big);
            const int32_t at = (c >> 3) * a.m + m;
            *(uint4*)(xq + (int64_t)at * kStep + ((c & 7) ^ ((m >> 1) & 7)) * 16) =
                make_uint4(vqd::f8_pack4(f, sc), vqd::f8_pack4(f + 4, sc), vqd::f8_pack4(f + 8, sc), vqd::f8_pack4(f + 12, sc));
            if ((c & 7) == 0) xs[at] = sc.s;
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }

    const int32_t mine = min(row, a.m - 1);
    const int c0 = (grp ^ ((mine >> 1) & 7)) * 16;
    auto use = [&](int set, int32_t at) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (at + u >= k1) break;
        const float g = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sg), at + u - k0));
        const float h = GATED ? __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, su), at + u - k0)) : 0.f;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          Frag<true> tok;
          float s;
          if constexpr (CUT) {
            const uint8_t* p = xq + (int64_t)((at + u - k0) * a.m + mine) * kStep;
            tok = join<true>(*(const v4i*)(p + c0), *(const v4i*)(p + (c0 ^ 64)));
            s = xs[(at + u - k0) * a.m + mine];
          } else {
            tok = join<true>(t[set][u][j][0], t[set][u][j][1]);
            s = ts[set][u][j];
          }
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const v4f p = multiply<true>(join<true>(w[set][u][i][0], w[set][u][i][1]), tok);
            const float c = s * (GATED && i >= NO ? h : g);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[r], c, acc[i][j][r]);
          }
        }
      }
    };
    for (int32_t b = 0; b < sets; b += 2) {
      use(0, k0 + b * U);
      if (b + 2 < sets) load(0, k0 + (b + 2) * U);
      if (b + 1 < sets) {
        use(1, k0 + (b + 1) * U);
        if (b + 3 < sets) load(1, k0 + (b + 3) * U);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) red[(wave * kTiles + i * MT + j) * 64 + lane] = acc[i][j];
  __syncthreads();

  // lane: token lane % 16, channels 4 (lane / 16) .. + 3 of a block; the wavefronts share the blocks out
  for (int o = wave; o < NO * MT; o += 8) {
    const int j = o % MT, i = o / MT;
    const int32_t m = 16 * j + row;
    const int32_t n = n0 + 16 * i + 4 * grp;
    auto total = [&](int at) {
      v4f sum = red[at * 64 + lane];
#pragma unroll
      for (int v = 1; v < 8; ++v) sum += red[(v * kTiles + at) * 64 + lane];
      return sum;
    };
    const v4f sum = total(o);
    float v[4], b[4];
    load_bias<4>(a.bias, n, a.n, b);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = sum[r] + b[r];
    if constexpr (GATED) {
      const v4f up = total(o + NO * MT);
      load_bias<4>(a.bias ? a.bias + a.n : nullptr, n, a.n, b);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = silu(v[r]) * (up[r] + b[r]);
    }
    if (m < a.m) store_run<4>(a.y, a.y_dtype, (int64_t)m * a.n, n, a.n, v);
  }
}

// ---------------------------------------------------------------- launches

vq_status done() { return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP; }

// Blocks of 16 outputs per workgroup of the kernels that stream the weights: 4, 2 or 1, as many as leave most CUs a
// workgroup (with the gate a block is 32 weight rows).
inline int out_blocks(int32_t n, bool gated) {
  if (gated) return n / 32 >= 192 ? 2 : 1;
  return n / 64 >= 192 ? 4 : n / 32 > 144 ? 2 : 1;
}

constexpr size_t kCutLds = 64 * 1024;
constexpr size_t few_lds(int tiles, int32_t m, int32_t k, bool cut) {
  return (size_t)8 * tiles * 1024 + (cut ? (size_t)vqi::f8_blocks(k) * m * (kStep + 4) : 0);
}

template <int RT, int MT, bool GATED, int XT>
vq_status few(const F8Args& a, hipStream_t st, bool check_only) {
  constexpr int out = (GATED ? RT / 2 : RT) * 16;
  const int64_t blocks = ((int64_t)a.n + out - 1) / out;
  if (!vqi::grid_ok(blocks, 512)) return VQ_ERR_SHAPE;
  if (check_only) return VQ_OK;
  f8_few_kernel<RT, MT, GATED, XT><<<dim3((uint32_t)blocks), dim3(512), few_lds(RT * MT, a.m, a.k, XT >= 0), st>>>(a);
  return done();
}
template <int RT, bool GATED>
vq_status few_cut(const F8Args& a, hipStream_t st, bool check_only) {
  switch (a.x_dtype) {
    case VQ_F32: return few<RT, 1, GATED, VQ_F32>(a, st, check_only);
    case VQ_F16: return few<RT, 1, GATED, VQ_F16>(a, st, check_only);
    default: return few<RT, 1, GATED, VQ_BF16>(a, st, check_only);
  }
}

template <int BM, int BN, int WM, int WN, int NB, bool WIDE, bool GATED, bool SPLIT>
vq_status launch_tile(const F8Args& a, hipStream_t st, bool check_only) {
  const int out = GATED ? BN / 2 : BN;
  const int64_t mt = ((int64_t)a.m + BM - 1) / BM;
  const int64_t nt = ((int64_t)a.n + out - 1) / out;
  constexpr int kThreads = 64 * WM * WN;
  if (!vqi::grid_ok(mt * nt + 8, kThreads)) return VQ_ERR_SHAPE;
  if (check_only) return VQ_OK;
  const uint32_t blocks = (uint32_t)((mt * nt + 7) / 8 * 8);
  f8_tile_kernel<BM, BN, WM, WN, NB, WIDE, GATED, SPLIT>
      <<<dim3(blocks, SPLIT ? a.splits : 1), dim3(kThreads), 0, st>>>(a, (int32_t)nt, (int32_t)mt);
  return done();
}
vq_status launch_join(const F8Args& a, hipStream_t st) {
  const int64_t items = (int64_t)a.m * ((a.n + 3) / 4);  // few tiles: a small grid
  f8_join_kernel<<<dim3((uint32_t)((items + 255) / 256)), dim3(256), 0, st>>>(a);
  return done();
}
template <bool WIDE, bool GATED, bool OUTQ>
vq_status launch_big(const F8Args& a, hipStream_t st, bool check_only) {
  constexpr int rows = WIDE ? 128 : 256, out = GATED ? 128 : 256;
  const int64_t mt = ((int64_t)a.m + rows - 1) / rows;
  const int64_t nt = ((int64_t)a.n + out - 1) / out;
  const int64_t blocks = WIDE ? (mt * nt + 7) / 8 * 8 : mt * nt + 128 + 8;  // at most 128 tiles are cut in two
  if (!vqi::grid_ok(blocks, 512)) return VQ_ERR_SHAPE;
  if (check_only) return VQ_OK;
  f8_big_kernel<WIDE, GATED, OUTQ><<<dim3((uint32_t)blocks), dim3(512), 0, st>>>(a, (int32_t)nt, (int32_t)mt);
  return done();
}

// How a product is computed.
enum Way { kStreamed, k64x64, k128x128, k256x256 };
struct Plan {
  Way way;
  int32_t splits;  // cuts of K over the CUs
};
Plan plan(int32_t m, int32_t n, int32_t k, bool gated) {
  const int64_t steps = vqi::f8_blocks(k);
  if (m <= 16) return {kStreamed, 1};
  auto tiles = [&](int bm, int bn) { return (((int64_t)m + bm - 1) / bm) * (((int64_t)n + bn - 1) / bn); };
  auto cut = [&](int64_t t) {
    return steps < 56 || gated ? 1 : (int32_t)std::max<int64_t>(1, std::min<int64_t>(256 / t, steps / 8));
  };
  if (tiles(256, gated ? 128 : 256) >= 200) return {k256x256, 1};
  if (m <= 64) return {k64x64, cut(tiles(64, 64))};
  return {k128x128, cut(tiles(128, 128))};
}

}  // namespace

namespace vqi {

vq_status launch_f8_tokens(const F8QuantArgs& a, void* stream, bool check_only) {
  hipStream_t st = (hipStream_t)stream;
  const int64_t rows = ((int64_t)a.rows + 15) / 16, cols = (f8_blocks(a.k) + kQuantCols - 1) / kQuantCols;
  if (!grid_ok(rows, 256)) return VQ_ERR_SHAPE;
  if (check_only) return VQ_OK;
  const dim3 g((uint32_t)rows, (uint32_t)cols), b(256);
  switch (a.x_dtype) {
    case VQ_F32: f8_tokens_kernel<VQ_F32><<<g, b, 0, st>>>(a); break;
    case VQ_F16: f8_tokens_kernel<VQ_F16><<<g, b, 0, st>>>(a); break;
    default: f8_tokens_kernel<VQ_BF16><<<g, b, 0, st>>>(a);
  }
  return done();
}

vq_status launch_f8_weights(const F8QuantArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const int64_t kb = f8_blocks(a.k), nb = f8_blocks(a.rows);
  if (nb > 65535) return VQ_ERR_SHAPE;
  const dim3 g((uint32_t)kb, (uint32_t)nb), b(256);
  switch (a.x_dtype) {
    case VQ_F32: f8_weights_kernel<VQ_F32><<<g, b, 0, st>>>(a); break;
    case VQ_F16: f8_weights_kernel<VQ_F16><<<g, b, 0, st>>>(a); break;
    default: f8_weights_kernel<VQ_BF16><<<g, b, 0, st>>>(a);
  }
  return done();
}

int32_t f8_splits(int32_t m, int32_t n, int32_t k, bool gated) { return plan(m, n, k, gated).splits; }

bool f8_cuts_inside(int32_t m, int32_t n, int32_t k, bool gated) {
  const int tiles = out_blocks(n, gated) * (gated ? 2 : 1);
  return m <= 4 && plan(m, n, k, gated).way == kStreamed && few_lds(tiles, m, k, true) <= kCutLds;
}

bool f8_writes_q(int32_t m, int32_t n, int32_t k) { return plan(m, n, k, true).way == k256x256; }

vq_status launch_f8(const F8Args& a, void* stream, bool check_only) {
  hipStream_t st = (hipStream_t)stream;
  const Plan p = plan(a.m, a.n, a.k, a.gated);
  if (a.gated) {
    switch (p.way) {
      case kStreamed:
        if (!a.q) return out_blocks(a.n, true) == 2 ? few_cut<4, true>(a, st, check_only) : few_cut<2, true>(a, st, check_only);
        return out_blocks(a.n, true) == 2 ? few<4, 1, true, -1>(a, st, check_only) : few<2, 1, true, -1>(a, st, check_only);
      case k64x64: return launch_tile<64, 128, 2, 2, 2, true, true, false>(a, st, check_only);
      case k128x128: return launch_tile<128, 128, 2, 2, 2, true, true, false>(a, st, check_only);
      default:
        if (a.wide) return a.y ? launch_big<true, true, false>(a, st, check_only) : launch_big<true, true, true>(a, st, check_only);
        return a.y ? launch_big<false, true, false>(a, st, check_only) : launch_big<false, true, true>(a, st, check_only);
    }
  }
  switch (p.way) {
    case kStreamed:
      switch (out_blocks(a.n, false)) {
        case 4: return a.q ? few<4, 1, false, -1>(a, st, check_only) : few_cut<4, false>(a, st, check_only);
        case 2: return a.q ? few<2, 1, false, -1>(a, st, check_only) : few_cut<2, false>(a, st, check_only);
        default: return a.q ? few<1, 1, false, -1>(a, st, check_only) : few_cut<1, false>(a, st, check_only);
      }
    case k64x64: {
      if (a.splits == 1) return launch_tile<64, 64, 2, 2, 4, true, false, false>(a, st, check_only);
      const vq_status e = launch_tile<64, 64, 2, 2, 4, true, false, true>(a, st, check_only);
      return e != VQ_OK || check_only ? e : launch_join(a, st);
    }
    case k128x128: {
      if (a.splits == 1) return launch_tile<128, 128, 2, 2, 2, true, false, false>(a, st, check_only);
      const vq_status e = launch_tile<128, 128, 2, 2, 2, true, false, true>(a, st, check_only);
      return e != VQ_OK || check_only ? e : launch_join(a, st);
    }
    case k256x256: return a.wide ? launch_big<true, false, false>(a, st, check_only) : launch_big<false, false, false>(a, st, check_only);
  }
  return VQ_ERR_UNSUPPORTED;
}

}  // namespace vqi
