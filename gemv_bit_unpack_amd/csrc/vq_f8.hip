// The 8-bit float products: y[m][n] = sum_b s[b][m] sw[n / 128][b] sum_{k in block b} q[m][k] w[n][k] (+ bias[n]), with
// e4m3 values and one fp32 scale for each 128 columns of a token and each 128 x 128 block of the weights; the gated form
// y = silu(g) u of two such products; and the cutting of tokens and weights to e4m3.
//
// A block of K is one matrix instruction deep (16 x 16 x 128), so its sum leaves the matrix pipe once, in fp32, and is
// added to the output's fp32 sum with the product of its two scales: one fused multiply-add per output and block, beside
// 128 multiply-adds of the matrix pipe.  That is half of the vector pipe's time under the matrix pipe's whole.
//
// Weights that fill the memory's time bound it up to some hundred rows (one row of 28672 x 8192: 42 us, 5.6 TB/s; 128 of
// 8192 x 28672: 54 us, 4.3).  Smaller ones, from 17 rows on, take 2 to 4 times as long as their bytes: a CU has one tile or
// two, a step of which is a chain of loads, barrier, fragments and products (37 x 5003 x 4099: 14 us, the matrix pipe busy a
// tenth of it).  Prompts fill no pipe: 8192^3 takes 479 to 514 us (2.1 to 2.3 PFLOP/s; a library product with one scale for
// all 414 to 427), with the matrix pipe busy 52 % of the cycles, at 2.0 GHz, the vector pipe 41 % and wavefronts waiting for
// 29 % of theirs.
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
// before the first is used.  Bound by the bytes (4096 x 4096 in bf16: 12 us, 4.2 TB/s); few rows by the launch (4 us).
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
  vqd::Run<XT, 8> raw[kQuantCols];
#pragma unroll
  for (int c = 0; c < kQuantCols; ++c) raw[c] = vqd::load_run<XT, 8>(x, (b0 + c) * kStep + lane16 * 8, a.k);
#pragma unroll
  for (int c = 0; c < kQuantCols; ++c) {
    if (b0 + c >= blocks) break;
    float f[8];
    vqd::widen(raw[c], f);
    uint32_t big = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) big = max(big, vqd::abs_bits(f[k]));
    const vqd::Q8Scale sc = vqd::f8_scale(vqd::group_max<16>(big));
    const uint2 v = make_uint2(vqd::f8_pack4(f, sc), vqd::f8_pack4(f + 4, sc));
    *(uint2*)(a.q + (int64_t)row * ld + (b0 + c) * kStep + lane16 * 8) = v;
    if (lane16 == 0) a.s[(int64_t)(b0 + c) * a.rows + row] = sc.s;
  }
}

// Weights: a workgroup takes a block of 128 rows and columns, once for its largest value and once for its bytes.
template <vq_dtype XT>
__global__ __launch_bounds__(256) void f8_weights_kernel(F8QuantArgs a) {
  __shared__ uint32_t part[4];
  const int32_t blocks = (int32_t)vqi::f8_blocks(a.k);
  const int32_t nb = (int32_t)blockIdx.x / blocks, kb = (int32_t)blockIdx.x - nb * blocks;
  const int col = (threadIdx.x & 15) * 8, row0 = nb * 128 + (threadIdx.x >> 4);
  constexpr int es = XT == VQ_F32 ? 4 : 2;
  const int32_t end = min(a.rows, nb * 128 + 128);
  uint32_t big = 0;
  float f[8][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int32_t r = row0 + 16 * j;
    vqd::widen(vqd::load_run<XT, 8>((const char*)a.x + (int64_t)min(r, end - 1) * a.ldx * es, kb * kStep + col, a.k), f[j]);
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
  if (threadIdx.x == 0) a.s[blockIdx.x] = sc.s;
}

// ---------------------------------------------------------------- tiles

// 4 bytes per lane from `g` to LDS at the wavefront's `l` + 4 lane.
__device__ __forceinline__ void to_lds4(const float* g, uint8_t* l) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                   (__attribute__((address_space(3))) void*)l, 4, 0, 0);
}

// Bytes of a step in LDS: its rows and its tokens' scales (64 at least, what a wavefront's load brings).
constexpr int step_bytes(int bm, int bn) { return (bm + bn) * kStep + (bm < 64 ? 64 : bm) * 4; }

// One tile: KG groups of WM x WN wavefronts, each with its share of K and its own NB steps in LDS, compute BM rows (row0
// ..) by BN weight rows (with the gate: BN / 2 outputs).  Each wavefront's weight rows are 16 NI consecutive ones (8 NI
// outputs of gate and up rows with the gate), dealt to its NI blocks so that a lane ends with 4 NI (2 NI) consecutive
// outputs of one token.
// OUTQ: the outputs in 8 bits (with the gate, BN / 2 = 128 outputs: one block).
// lds: KG * NB steps.  sbs: the scales of the weights' blocks, two rows of at most 512.  tops: the tokens' largest values
// of the 8-bit epilogue.
template <int BM, int BN, int WM, int WN, int NB, int KG, bool WIDE, bool GATED, bool SPLIT, bool OUTQ>
__device__ __forceinline__ void tile(const F8Args& a, int32_t row0, int32_t n0, uint8_t* lds, float* sbs, float* tops) {
  constexpr int kWaves = WM * WN;
  constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  constexpr int NO = GATED ? NI / 2 : NI;  // blocks of outputs
  constexpr int TL = BM / 8 / kWaves, WL = BN / 8 / kWaves;  // 8-row loads per wavefront and step
  constexpr int SG = (BM + 63) / 64;                         // groups of 64 token scales
  constexpr int kRows = (BM + BN) * kStep;
  constexpr int kBuf = step_bytes(BM, BN);
  // steps in LDS: one is read while NB - 1 are on their way; vmcnt of a wavefront whose loads of one step more than the
  // next may be outstanding
  constexpr int kLater = (NB - 2) * (TL + WL + 1);
  static_assert(NB >= 2 && kLater < 64, "the wait counter holds 6 bits");
  constexpr int kWaitNext = 0x0070 | (kLater & 15) | (kLater >> 4) << 14;  // and lgkmcnt(0)
  static_assert(TL * 8 * kWaves == BM && WL * 8 * kWaves == BN, "whole loads");
  static_assert(SG <= kWaves, "each wavefront loads one group of scales");
  static_assert(!GATED || NI % 2 == 0, "gate and up blocks in one wavefront");
  static_assert(!OUTQ || (GATED && BN == 256 && WN * NO * 16 == 128), "a block of outputs per tile");
  // small tiles read the next step's fragments while they multiply this one's; larger ones have registers for its weights
  // and first token block only, asked for behind this step's last products (4096 x 14336 x 4096 270 -> 232 us, with the loads
  // to LDS no longer waited for)
  constexpr bool AHEAD = MI + NI <= 6;
  static_assert(KG == 1 || (KG == 2 && AHEAD && !SPLIT && !OUTQ && MI * NI * 1024 * kWaves <= NB * kBuf), "sums of two groups");

  const int lane = threadIdx.x & 63;
  const int all_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = all_wave % kWaves, group = all_wave / kWaves;
  lds += group * NB * kBuf;
  const int wm = wave / WN, wn = wave % WN;
  const int col = lane & 15, grp = lane >> 4;
  const int64_t ld = vqi::q8_row_bytes(a.k);
  const int32_t blocks = (int32_t)(ld / kStep);
  const int32_t end = min(a.m, row0 + BM);

  int32_t first = 0, last = blocks;
  if constexpr (SPLIT) {
    first = (int32_t)((int64_t)blocks * blockIdx.y / a.plan.splits);
    last = (int32_t)((int64_t)blocks * (blockIdx.y + 1) / a.plan.splits);
  }
  // steps of each group of wavefronts; the second may have one less
  const int32_t n = (last - first + KG - 1) / KG;
  const int32_t kt0 = first + group * n;
  const int32_t mine = KG == 1 ? n : min(n, last - kt0);

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
  // the weights' scales of the steps: with the gate a row for each half, else one for each 128 weight rows.  Asked for
  // before the first steps and put down behind them: no load waits for another
  const int32_t nblocks = (int32_t)vqi::f8_blocks(a.n);
  constexpr int kScaleRows = GATED || BN > 128 ? 2 : 1;
  constexpr int kThreads = 64 * kWaves * KG;
  constexpr int kPer = (512 + kThreads - 1) / kThreads;
  const int32_t all = last - first;
  float sv[kScaleRows][kPer];
#pragma unroll
  for (int r = 0; r < kScaleRows; ++r) {
    const int32_t nb = GATED ? n0 / 128 + r * nblocks : min(n0 / 128 + r, nblocks - 1);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      sv[r][i] = a.sw[(int64_t)nb * blocks + first + min((int32_t)threadIdx.x + i * kThreads, all - 1)];
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int b = 0; b < NB - 1; ++b)
    if (b < mine) fetch(b);
#pragma unroll
  for (int r = 0; r < kScaleRows; ++r)
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if ((int32_t)threadIdx.x + i * kThreads < all) sbs[r * 512 + threadIdx.x + i * kThreads] = sv[r][i];
  const float* const sb0 = sbs + (GATED ? 0 : (n0 % 128 + wn * 16 * NI) / 128 * 512) + (kt0 - first);

  v4f acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  const int lt = (wm * MI * 16 + col) * kStep;
  const int lw = BM * kStep + (wn * NI * 16 + col) * kStep;
  const int c0 = (grp ^ ((col >> 1) & 7)) * 16;
  auto frag = [&](int at) { return join<WIDE>(*(const v4i*)(lds + at + c0), *(const v4i*)(lds + at + (c0 ^ 64))); };
  auto token_scale = [&](int at, int i) { return *(const float*)(lds + at + kRows + (wm * MI * 16 + i * 16 + col) * 4); };
  auto add = [&](int i, const v4f (&p)[NI], float s, float sg, float su) {
    const float s0 = s * sg, s1 = s * su;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[j][r], GATED && j >= NO ? s1 : s0, acc[i][j][r]);
      asm volatile("" : "+v"(acc[i][j]));  // here, and not after the step's last product
    }
  };
  // its part of step kt is in LDS (steps after that may still be on their way), its last reads are done
  auto arrived = [&](int32_t kt) {
    if (kt + NB - 2 < mine) {
      __builtin_amdgcn_s_waitcnt(kWaitNext);
    } else {
      __builtin_amdgcn_s_waitcnt(0x0070);
    }
  };

  arrived(0);
  meet();  // and everyone's, and the scales
  if (NB - 1 < mine) fetch(NB - 1);
  int buf = 0;
  // the next step may be read, this one overwritten
  auto next = [&](int32_t kt) {
    arrived(kt + 1);
    meet();
    if (kt + NB < mine) fetch(buf);
    buf = buf + 1 == NB ? 0 : buf + 1;
  };
  if constexpr (AHEAD) {
    v4i rw[2][NI][2], rt[2][MI][2];
    float s[2][MI], sg[2], su[2];
    auto read = [&](int set, int32_t kt) {
      const int at = buf * kBuf;
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        rw[set][j][0] = *(const v4i*)(lds + at + lw + j * 16 * kStep + c0);
        rw[set][j][1] = *(const v4i*)(lds + at + lw + j * 16 * kStep + (c0 ^ 64));
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        rt[set][i][0] = *(const v4i*)(lds + at + lt + i * 16 * kStep + c0);
        rt[set][i][1] = *(const v4i*)(lds + at + lt + i * 16 * kStep + (c0 ^ 64));
        s[set][i] = token_scale(at, i);
      }
      sg[set] = sb0[kt];
      su[set] = GATED ? sb0[512 + kt] : 0.f;
    };
    auto step = [&](int set, int32_t kt) {
      if (kt + 1 < n) {
        next(kt);
        read(1 - set, min(kt + 1, mine - 1));
        __builtin_amdgcn_sched_barrier(0);
      }
      if (KG == 1 || kt < mine) {
        Frag<WIDE> w[NI];
#pragma unroll
        for (int j = 0; j < NI; ++j) w[j] = join<WIDE>(rw[set][j][0], rw[set][j][1]);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const Frag<WIDE> t = join<WIDE>(rt[set][i][0], rt[set][i][1]);
          v4f p[NI];
#pragma unroll
          for (int j = 0; j < NI; ++j) p[j] = multiply<WIDE>(w[j], t);
          add(i, p, s[set][i], sg[set], su[set]);
        }
      }
    };
    read(0, 0);
    int32_t kt = 0;
    for (; kt + 2 <= n; kt += 2) {
      step(0, kt);
      step(1, kt + 1);
    }
    if (kt < n) step(0, kt);
  } else {
    // a step's weights and first token block are asked for behind the last products of the step before
    static_assert(MI % 2 == 0, "the first token block's place is free by then");
    v4i rw[NI][2], rt[2];
    float s[MI], sg, su;
    auto head = [&](int32_t kt) {
      const int at = buf * kBuf;
#pragma unroll
      for (int h = 0; h < 2; ++h) rt[h] = *(const v4i*)(lds + at + lt + (c0 ^ (64 * h)));
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) rw[j][h] = *(const v4i*)(lds + at + lw + j * 16 * kStep + (c0 ^ (64 * h)));
#pragma unroll
      for (int i = 0; i < MI; ++i) s[i] = token_scale(at, i);
      sg = sb0[kt];
      su = GATED ? sb0[512 + kt] : 0.f;
    };
    auto step = [&](int32_t kt, bool more) {
      const int at = buf * kBuf;
      Frag<WIDE> w[NI], t[2];
#pragma unroll
      for (int j = 0; j < NI; ++j) w[j] = join<WIDE>(rw[j][0], rw[j][1]);
      t[0] = join<WIDE>(rt[0], rt[1]);
      v4f p[2][NI];
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if (i + 1 < MI) {
          t[(i + 1) & 1] = frag(at + lt + (i + 1) * 16 * kStep);
        } else if (more) {
          next(kt);
        }
#pragma unroll
        for (int j = 0; j < NI; ++j) p[i & 1][j] = multiply<WIDE>(w[j], t[i & 1]);
        if (i > 0) add(i - 1, p[(i - 1) & 1], s[i - 1], sg, su);
        // the row's fragment on its way first, then each product with its share of the additions of the row before
        if (i + 1 < MI) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          __builtin_amdgcn_sched_group_barrier(0x008, WIDE ? 4 : 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 4 + (WIDE ? 4 : 0), 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      const float sl = s[MI - 1], gl = sg, ul = su;
      if (more) {
        head(kt + 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      add(MI - 1, p[(MI - 1) & 1], sl, gl, ul);
    };
    head(0);
    for (int32_t kt = 0; kt + 1 < n; ++kt) step(kt, true);
    if (n > 0) step(n - 1, false);
  }
  if constexpr (KG == 2) {  // the second group's sums join the first's
    v4f* const sums = (v4f*)(lds + (1 - group) * NB * kBuf) + wave * MI * NI * 64 + lane;
    __builtin_amdgcn_s_waitcnt(0x0070);
    meet();  // no one reads a step any more
    if (group == 1) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) sums[(i * NI + j) * 64] = acc[i][j];
    }
    __syncthreads();
    if (group == 1) return;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] += sums[(i * NI + j) * 64];
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

template <int BM, int BN, int WM, int WN, int NB, int KG, bool WIDE, bool GATED, bool SPLIT>
__global__ __launch_bounds__(64 * WM * WN * KG) void f8_tile_kernel(F8Args a, int32_t nt, int32_t mt_count) {
  // one array: with more than one the compiler waits for all loads to LDS before each read of it
  __shared__ __attribute__((aligned(1024))) uint8_t lds[KG * NB * step_bytes(BM, BN) + (GATED || BN > 128 ? 4096 : 2048)];
  float* const sbs = (float*)(lds + KG * NB * step_bytes(BM, BN));
  int32_t mt, nti;
  if (!place((int32_t)blockIdx.x, mt_count * nt, mt_count, nt, mt, nti)) return;
  tile<BM, BN, WM, WN, NB, KG, WIDE, GATED, SPLIT, false>(a, mt * BM, nti * (GATED ? BN / 2 : BN), lds, sbs, nullptr);
}

// 8 wavefronts, one workgroup per CU: 256 x 256 tiles, or 128 x 256 ones for outputs in 8 bits, whose operands go to fp16
// (their fragments take twice the registers; their conversions take as much of the vector pipe, 57 % of the cycles, as the
// products of the matrix pipe, 45 %: 2048 tokens, 14336 pairs of 4096 columns 494 to 507 us).  256 x 256: 128 rows only where the matrix's last tile has no more left, and in the last round
// over the 256 CUs if at most half of them have a tile in it: two half tiles for each then take half a round.
template <bool GATED, bool OUTQ>
__global__ __launch_bounds__(512) void f8_big_kernel(F8Args a, int32_t nt, int32_t mt_count) {
  constexpr int kSteps = OUTQ ? 3 * step_bytes(128, 256) : 2 * step_bytes(256, 256);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kSteps + 4096 + (OUTQ ? 16 * 128 : 0)];
  float* const sbs = (float*)(lds + kSteps);
  const int32_t total = mt_count * nt;
  const int32_t id = (int32_t)blockIdx.x;
  int32_t mt, nti, part = 0;
  if constexpr (OUTQ) {
    if (!place(id, total, mt_count, nt, mt, nti)) return;
    tile<128, 256, 2, 4, 3, 1, true, GATED, false, true>(a, mt * 128, nti * 128, lds, sbs, sbs + 1024);
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
      tile<128, 256, 2, 4, 2, 1, false, GATED, false, false>(a, row0, n0, lds, sbs, nullptr);
    } else {
      tile<256, 256, 2, 4, 2, 1, false, GATED, false, false>(a, row0, n0, lds, sbs, nullptr);
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
    for (int32_t k = 0; k < a.plan.splits; ++k) {
      float f[4];
      __builtin_memcpy(f, p + k * apart, 16);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += f[r];
    }
  } else {
    for (int32_t k = 0; k < a.plan.splits; ++k)
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
// takes groups of RT blocks of 16 weight rows (with the gate RT / 2 blocks of gate rows and as many of up rows) one after
// the other, and 16 tokens at most; its wavefronts cut K, their sums meet in LDS.  Two sets of U steps are in registers, one
// on its way while the other is used, across the groups: the first steps of the next group are asked for before the sums
// of this one meet.  The steps of a last, partial set are the last one again and left out.
// Bound by the weights' bytes: 1 x 28672 x 8192 42 us, 5.6 TB/s.  A load takes 32 bytes of a lane's row in two pieces next
// to each other, so that both of a memory line's halves are asked for together, and without the hint that they are read
// once: with pieces 64 bytes apart and the hint 2 x 28672 x 5120 took 44 us, so 34.  Small products are bound by their chain
// of latencies: 1 x 4096 x 4096 7 us, 1 x 1024 x 1024 5.
// XT >= 0: the tokens come as they are and each wavefront cuts its own part of K to 8 bits, in LDS, once, while its first
// weights are on their way: a block's scale needs no other wavefront, so there is no barrier and no launch in front.
// SPLIT: workgroups cut K too (blockIdx.y), and their sums go to `part`.
template <int RT, bool GATED, bool SPLIT, int XT>
__global__ __launch_bounds__(512, 4) void f8_few_kernel(F8Args a, int32_t groups) {
  constexpr bool CUT = XT >= 0;
  static_assert(!GATED || (RT % 2 == 0 && !SPLIT), "gate and up blocks");
  constexpr int NO = GATED ? RT / 2 : RT;
  constexpr int U = CUT ? 4 / RT : 2 / RT;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // [8][RT][64] v4f, then the cut tokens

  // all arguments at once: each of their cache lines that is first read later would cost a small product half a microsecond
  asm volatile("" ::"s"(a.w), "s"(a.sw), "s"(a.y), "s"(a.plan.splits), "s"(groups));

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, grp = lane >> 4;
  const int64_t ld = vqi::q8_row_bytes(a.k);
  const int32_t blocks = (int32_t)(ld / kStep), nblocks = (int32_t)vqi::f8_blocks(a.n);
  int32_t first = 0, last = blocks;
  if constexpr (SPLIT) {
    first = (int32_t)((int64_t)blocks * blockIdx.y / a.plan.splits);
    last = (int32_t)((int64_t)blocks * (blockIdx.y + 1) / a.plan.splits);
  }
  const int32_t k0 = first + (last - first) * wave / 8, k1 = first + (last - first) * (wave + 1) / 8;
  const int32_t sets = (k1 - k0 + U - 1) / U;  // of each group; a short K leaves wavefronts without any
  const int32_t mine = min(row, a.m - 1);
  v4f* const red = (v4f*)lds;

  v4f acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};

  // the tokens' part of this wavefront in pieces of 16 columns: piece e is piece e % pieces of token e / pieces, columns
  // 16 (.. % 8) .. of step k0 + .. / 8.  The first ones are asked for before the weights, which then arrive behind them
  constexpr vq_dtype XD = CUT ? (vq_dtype)XT : VQ_F32;
  constexpr int kAhead = GATED || XT == VQ_F32 ? 1 : 2;  // what 128 registers hold
  const int32_t pieces = (k1 - k0) * 8, all = pieces * a.m;
  auto token_of = [&](int32_t e) { return a.m == 1 ? 0 : e / pieces; };  // one token: no division before its loads
  auto piece = [&](int32_t e) {
    const int32_t m = token_of(e), c = e - m * pieces;
    return vqd::load_run<XD, 16>((const char*)a.x + (int64_t)m * a.ldx * (XD == VQ_F32 ? 4 : 2), k0 * kStep + c * 16, a.k);
  };
  vqd::Run<XD, 16> raw[CUT ? kAhead : 1];
  if constexpr (CUT) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (lane + 64 * i < all) raw[i] = piece(lane + 64 * i);
    __builtin_amdgcn_sched_barrier(0);
  }

  v4i w[2][U][RT][2], t[2][CUT ? 1 : U][2];
  float ts[2][CUT ? 1 : U], sg[2], su[2];  // sg, su: the weights' scales of a set's steps, one per lane
  const uint8_t* gw[RT];
  const uint8_t* const gt = CUT ? nullptr : a.q + (int64_t)mine * ld + grp * 32;
  const float* sw = nullptr;
  int32_t ask_group = (int32_t)blockIdx.x, ask_set = 0;
  auto ask = [&](int set) {  // the next set of steps, of this group or the next
    if (ask_group >= groups) return;
    if (ask_set == 0) {
      const int32_t n0 = ask_group * 16 * NO;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int64_t r = (int64_t)min(n0 + 16 * (i % NO) + row, a.n - 1) + (i >= NO ? a.n : 0);
        gw[i] = a.w + r * ld + grp * 32;
      }
      sw = a.sw + (int64_t)(n0 / 128) * blocks;
    }
    const int32_t at = k0 + ask_set * U;
    sg[set] = sw[min(at + (lane & 3), k1 - 1)];
    if constexpr (GATED) su[set] = sw[(int64_t)nblocks * blocks + min(at + (lane & 3), k1 - 1)];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t k = min(at + u, k1 - 1);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[set][u][i][h] = *(const v4i*)(gw[i] + (int64_t)k * kStep + 16 * h);
      if constexpr (!CUT) {
#pragma unroll
        for (int h = 0; h < 2; ++h) t[set][u][h] = *(const v4i*)(gt + (int64_t)k * kStep + 16 * h);
        ts[set][u] = a.s[(int64_t)k * a.m + mine];
      }
    }
    if (++ask_set == sets) {
      ask_set = 0;
      ask_group += (int32_t)gridDim.x;
    }
  };
  if (sets > 0) {
    ask(0);
    ask(1);
  }
  __builtin_amdgcn_sched_barrier(0);

  // the workgroup's tokens [steps][m][128] and behind them their scales [steps][m]; each wavefront writes and reads its own
  uint8_t* const tokens = lds + 8 * RT * 1024;
  uint8_t* const xq = tokens + (int64_t)(k0 - first) * a.m * kStep;
  float* const xs = (float*)(tokens + (int64_t)(last - first) * a.m * kStep) + (int64_t)(k0 - first) * a.m;
  if constexpr (CUT) {
    for (int32_t e0 = 0; e0 < all; e0 += 64 * kAhead) {
      if (e0 > 0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (e0 + lane + 64 * i < all) raw[i] = piece(e0 + lane + 64 * i);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (e0 + 64 * i >= all) break;
        const int32_t e = e0 + lane + 64 * i;
        float f[16];
        vqd::widen(raw[i], f);
        uint32_t big = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) big = max(big, vqd::abs_bits(f[k]));
        big = vqd::group_max<8>(big);
        if (e < all) {  // 8 lanes at once
          const int32_t m = token_of(e), c = e - m * pieces;
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

  const int c0 = ((2 * grp) ^ ((mine >> 1) & 7)) * 16;
  auto use = [&](int set, int32_t at) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (at + u >= k1) break;
      auto scale = [&](float v) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), u)); };
      const float g = scale(sg[set]), h = GATED ? scale(su[set]) : 0.f;
      Frag<true> tok;
      float s;
      if constexpr (CUT) {
        const uint8_t* p = xq + (int64_t)((at + u - k0) * a.m + mine) * kStep;
        tok = join<true>(*(const v4i*)(p + c0), *(const v4i*)(p + (c0 ^ 16)));
        s = xs[(at + u - k0) * a.m + mine];
      } else {
        tok = join<true>(t[set][u][0], t[set][u][1]);
        s = ts[set][u];
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const v4f p = multiply<true>(join<true>(w[set][u][i][0], w[set][u][i][1]), tok);
        const float c = s * (GATED && i >= NO ? h : g);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][r] = __builtin_fmaf(p[r], c, acc[i][r]);
      }
    }
  };
  // The sums of a group meet and are stored.  The barriers are bare: loads stay on their way across them.
  auto finish = [&](int32_t group) {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the reads of the group before are done
    meet();
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      red[(wave * RT + i) * 64 + lane] = acc[i];
      acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);
    meet();
    // lane: token lane % 16, channels 4 (lane / 16) .. + 3 of a block; a wavefront for each block
    if (wave >= NO) return;
    auto total = [&](int at) {
      v4f sum = red[at * 64 + lane];
#pragma unroll
      for (int v = 1; v < 8; ++v) sum += red[(v * RT + at) * 64 + lane];
      return sum;
    };
    int32_t tok = row;
    asm volatile("" : "+v"(tok));  // its addresses are formed here, not kept in registers from the start
    const int32_t n = group * 16 * NO + 16 * wave + 4 * grp;
    const v4f sum = total(wave);
    float v[4], b[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = sum[r];
    if constexpr (SPLIT) {
      if (tok < a.m) store_run<4>(a.part, VQ_F32, ((int64_t)blockIdx.y * a.m + tok) * a.n, n, a.n, v);
    } else {
      if (a.bias) {
        load_bias<4>(a.bias, n, a.n, b);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += b[r];
      }
      if constexpr (GATED) {
        v4f up = total(wave + NO);
        if (a.bias) {
          load_bias<4>(a.bias + a.n, n, a.n, b);
#pragma unroll
          for (int r = 0; r < 4; ++r) up[r] += b[r];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = silu(v[r]) * up[r];
      }
      if (tok < a.m) store_run<4>(a.y, a.y_dtype, (int64_t)tok * a.n, n, a.n, v);
    }
  };

  int32_t group = (int32_t)blockIdx.x, at_set = 0;
  auto turn = [&](int set) {
    use(set, k0 + at_set * U);
    ask(set);
    if (++at_set == sets) {
      finish(group);
      at_set = 0;
      group += (int32_t)gridDim.x;
    }
  };
  if (sets == 0) {
    for (; group < groups; group += (int32_t)gridDim.x) finish(group);
  }
  while (group < groups) {
    turn(0);
    if (group < groups) turn(1);
  }
}

// ---------------------------------------------------------------- launches

vq_status done() { return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP; }

constexpr size_t kCutLds = 64 * 1024;
// Dynamic LDS of the streaming kernel: the wavefronts' sums, and the cut tokens of a workgroup's steps.
constexpr size_t few_lds(int rt, int32_t m, int32_t steps, bool cut) {
  return (size_t)8 * rt * 1024 + (cut ? (size_t)steps * m * (kStep + 4) : 0);
}

vq_status launch_join(const F8Args& a, hipStream_t st) {
  const int64_t items = (int64_t)a.m * ((a.n + 3) / 4);  // K is cut for few tiles only: a small grid
  f8_join_kernel<<<dim3((uint32_t)((items + 255) / 256)), dim3(256), 0, st>>>(a);
  return done();
}

// Workgroups of the streaming kernel: as many as the CUs hold at once, two each.
constexpr int32_t kFewWorkgroups = 512;

template <int RT, bool GATED, int XT>
vq_status few(const F8Args& a, hipStream_t st, bool check_only) {
  constexpr int out = (GATED ? RT / 2 : RT) * 16;
  if (check_only) return VQ_OK;  // a bounded grid
  const int32_t groups = (int32_t)(((int64_t)a.n + out - 1) / out);
  const size_t lds = few_lds(RT, a.m, (int32_t)((vqi::f8_blocks(a.k) + a.plan.splits - 1) / a.plan.splits), XT >= 0);
  const dim3 g((uint32_t)std::min(groups, std::max(kFewWorkgroups / a.plan.splits, 1)), (uint32_t)a.plan.splits), b(512);
  if constexpr (!GATED) {
    if (a.plan.splits > 1) {
      f8_few_kernel<RT, GATED, true, XT><<<g, b, lds, st>>>(a, groups);
      const vq_status e = done();
      return e != VQ_OK ? e : launch_join(a, st);
    }
  }
  f8_few_kernel<RT, GATED, false, XT><<<g, b, lds, st>>>(a, groups);
  return done();
}
template <int RT, bool GATED>
vq_status few_cut(const F8Args& a, hipStream_t st, bool check_only) {
  switch (a.x_dtype) {
    case VQ_F32: return few<RT, GATED, VQ_F32>(a, st, check_only);
    case VQ_F16: return few<RT, GATED, VQ_F16>(a, st, check_only);
    default: return few<RT, GATED, VQ_BF16>(a, st, check_only);
  }
}

template <int BM, int BN, int WM, int WN, int NB, int KG, bool WIDE, bool GATED, bool SPLIT>
vq_status launch_tile(const F8Args& a, hipStream_t st, bool check_only) {
  const int out = GATED ? BN / 2 : BN;
  const int64_t mt = ((int64_t)a.m + BM - 1) / BM;
  const int64_t nt = ((int64_t)a.n + out - 1) / out;
  constexpr int kThreads = 64 * WM * WN * KG;
  if (!vqi::grid_ok(mt * nt + 8, kThreads)) return VQ_ERR_SHAPE;
  if (check_only) return VQ_OK;
  const uint32_t blocks = (uint32_t)((mt * nt + 7) / 8 * 8);
  f8_tile_kernel<BM, BN, WM, WN, NB, KG, WIDE, GATED, SPLIT>
      <<<dim3(blocks, SPLIT ? a.plan.splits : 1), dim3(kThreads), 0, st>>>(a, (int32_t)nt, (int32_t)mt);
  return done();
}
template <bool GATED, bool OUTQ>
vq_status launch_big(const F8Args& a, hipStream_t st, bool check_only) {
  constexpr int rows = OUTQ ? 128 : 256, out = GATED ? 128 : 256;
  const int64_t mt = ((int64_t)a.m + rows - 1) / rows;
  const int64_t nt = ((int64_t)a.n + out - 1) / out;
  const int64_t blocks = OUTQ ? (mt * nt + 7) / 8 * 8 : mt * nt + 128 + 8;  // at most 128 tiles are cut in two
  if (!vqi::grid_ok(blocks, 512)) return VQ_ERR_SHAPE;
  if (check_only) return VQ_OK;
  f8_big_kernel<GATED, OUTQ><<<dim3((uint32_t)blocks), dim3(512), 0, st>>>(a, (int32_t)nt, (int32_t)mt);
  return done();
}

// ---------------------------------------------------------------- which way

// A way of computing a product and what it takes, in us: `start` for the launch and its ends, and for each round over the
// CUs `round` and then `step` for each step of K, the first of them with one workgroup on a CU, then two and three, as many
// as `together` (the LDS) says.  Fitted to 670 shapes of 1 to 4096 rows by 64 to 28672 columns and outputs, weights from
// memory, which they meet to 10 - 17 % (rms).  The way with the least of these times, or of reading the operands, is taken:
// over those shapes 1.8 % slower than the best of each (geometric mean), at the worst a third, of 15 us.  us, in the way that
// is taken and in others:
//   16-bit outputs: 37 x 5003 x 4099 11.4 in 32 x 32, 12.4 in 32 x 64, 13.4 in 64 x 64, 14.6 in 64 x 128 / 4;
//     256 x 4096 x 4096 13.5 in 64 x 64, 16.3 in 32 x 64; 512 x 4096 x 4096 18.9 in 64 x 128, 24.4 in 128 x 128, 24.6 in
//     64 x 64; 128 x 28672 x 8192 57.5 in 128 x 128, 64.8 in pairs of them, 68.3 in 64 x 128; 128 x 8192 x 28672 63 in
//     128 x 128 / 4, 70.3 / 3, 72 in 64 x 128 / 2; 512 x 14336 x 4096 41.3 in pairs of 128 x 128, 49 in 256 x 256, 55.7 in
//     64 x 128; 4096 x 14336 x 4096 232 in 256 x 256, 268 in pairs of 128 x 128
//   fp32 outputs: 512 x 4096 x 4096 27.7 in 64 x 128, 32 in 64 x 64, 41 in 128 x 128; 4096 x 14336 x 4096 457 in pairs of
//     128 x 128, 543 in 128 x 128
//   few rows, streamed and in tiles, tokens in 8 bits: 16 x 4096 x 4096 7.1 and 9.3, 8 x 28672 x 8192 53 and 46.7; cut
//     inside or by a launch in front: 1 x 4096 x 4096 7.4 and 3.3 + 6.3, 8 x 4096 x 4096 10.2 and 3.3 + 6.4
enum Way : int32_t { kStream1, kStream2, k32x32, k32x64, k64x64, k64x128, k128x128, k128x128Pair, k256x256, kWays };
struct Cost {
  int32_t bm, bm_log2, bn, bn_log2, groups_of_k, together;
  float start, round, step[3];
};
constexpr Cost kCosts[2][kWays] = {
    {{16, 4, 16, 4, 8, 2, 1.76f, 0.f, {0.82f, 1.79f}},
     {16, 4, 32, 5, 8, 2, 1.64f, 0.f, {1.33f, 2.61f}},
     {32, 5, 32, 5, 2, 2, 1.46f, 1.54f, {0.32f, 0.53f}},
     {32, 5, 64, 6, 1, 3, 1.13f, 1.94f, {0.26f, 0.43f, 0.52f}},
     {64, 6, 64, 6, 2, 1, 0.64f, 2.63f, {0.55f}},
     {64, 6, 128, 7, 1, 2, 0.91f, 2.52f, {0.44f, 0.85f}},
     {128, 7, 128, 7, 1, 1, 1.51f, 3.64f, {0.61f}},
     {128, 7, 128, 7, 1, 2, 1.24f, 4.19f, {0.71f, 1.11f}},
     {256, 8, 256, 8, 1, 1, 2.87f, 8.20f, {1.73f}}},
    // operands in fp16
    {{16, 4, 16, 4, 8, 2, 1.76f, 0.f, {0.82f, 1.79f}},
     {16, 4, 32, 5, 8, 2, 1.64f, 0.f, {1.33f, 2.61f}},
     {32, 5, 32, 5, 2, 2, 1.30f, 1.70f, {0.40f, 0.65f}},
     {32, 5, 64, 6, 1, 3, 0.14f, 2.85f, {0.35f, 0.62f, 0.66f}},
     {64, 6, 64, 6, 2, 1, 0.66f, 2.66f, {0.78f}},
     {64, 6, 128, 7, 1, 2, 0.00f, 3.34f, {0.69f, 1.54f}},
     {128, 7, 128, 7, 1, 1, 0.87f, 3.95f, {1.06f}},
     {128, 7, 128, 7, 1, 2, 1.27f, 4.65f, {1.11f, 1.89f}},
     {128, 7, 256, 8, 1, 1, 0.92f, 5.69f, {1.75f}}}};  // only where it writes its outputs in 8 bits
// Cutting tokens to 8 bits: inside the streaming kernel (its start, and for each 64 pieces of 16 columns of a wavefront),
// and in a launch of its own (and its bytes per us).
constexpr float kCutStart[2] = {1.45f, 1.44f}, kCutPiece = 0.9f, kQuantStart = 3.3f, kQuantRate = 4e6f;
constexpr float kCopyRate = 5.3e6f, kCopyStart = 2.0f;   // bytes per us of a large copy
constexpr float kJoinStart = 4.6f, kJoinRate = 4.5e6f;   // the launch that adds up a cut K (3.6 us, and one to win by)

int32_t ceil_div(int32_t a, int32_t b) { return (int32_t)(((uint32_t)a + (uint32_t)b - 1) / (uint32_t)b); }

// The parts of a product's cost that no way changes.
struct Shape {
  int32_t m, steps;
  int64_t outputs;  // weight rows
  float copy, out, parts;
  Shape(int32_t m_, int32_t n, int32_t k, bool gated, bool wide)
      : m(m_), steps((int32_t)vqi::f8_blocks(k)), outputs((int64_t)n * (gated ? 2 : 1)) {
    out = (float)m * (float)n * (wide ? 4.f : 2.f);
    parts = 8.f * (float)m * (float)n;
    copy = kCopyStart + ((float)outputs * (float)k + (float)m * (float)k + out) / kCopyRate;
  }
};
float cost(const Shape& s, int32_t way, int32_t splits, bool cut, bool wide) {
  const Cost& c = kCosts[wide][way];
  const float steps = (float)ceil_div(splits == 1 ? s.steps : ceil_div(s.steps, splits), c.groups_of_k);
  const int32_t columns = (int32_t)((s.outputs + c.bn - 1) >> c.bn_log2);
  float t = c.start;
  if (way <= kStream2) {
    // two workgroups on each CU, that take turns with the memory: parts of a round count as such
    const float rounds = (float)columns * (float)splits * (1.f / kFewWorkgroups);
    // cut inside, single blocks with eight steps of a wavefront or more keep their loads going, most of all whole sets of four:
    // of 28672 outputs with eight steps (K = 8192) 42 us and 48 in groups of two, with nine and ten 51 to 54 either way, with
    // twelve 72 and 77, with sixteen 92 and 101; with five 34 and 33
    const float going = cut && way == kStream1 && steps >= 8.f ? 0.8f : 1.f;
    t += steps * (rounds <= 0.5f ? c.step[0] : going * c.step[1] * std::max(rounds, 1.f));
    if (cut) t += kCutStart[way] + kCutPiece * 0.125f * (float)s.m * steps;
  } else {
    const int32_t rows = (int32_t)(((int64_t)s.m + c.bm - 1) >> c.bm_log2);
    const int64_t tiles = (int64_t)rows * columns * splits;
    if (way == k256x256 && !wide) {  // the last round in half tiles
      const int32_t rest = (int32_t)(tiles & 255);
      const float rounds = (float)(tiles >> 8) + (rest == 0 ? 0.f : rest <= 128 ? 0.55f : 1.f);
      t += rounds * (c.round + steps * c.step[0]);
    } else if (c.together == 1) {
      t += (float)((tiles + 255) >> 8) * (c.round + steps * c.step[0]);
    } else {
      const uint64_t per_cu = (uint64_t)(tiles + 255) >> 8, full = per_cu / c.together, rest = per_cu - full * c.together;
      t += (float)(full + (rest != 0)) * c.round + steps * (float)full * c.step[c.together - 1];
      if (rest) t += steps * c.step[rest - 1];
    }
  }
  // streamed weights come with their tokens, from the caches: 8 and 16 rows of 28672 x 8192 53 and 60 us, 46 in tiles
  t = std::max(t, way <= kStream2 ? s.copy * (1.f + (float)s.m * (1.f / 64)) : s.copy);
  return splits == 1 ? t : t + kJoinStart + ((float)splits * s.parts + s.out) / kJoinRate;
}

vq_status stream(const F8Args& a, hipStream_t st, bool check_only) {
  const bool two = a.plan.way == kStream2;
  if (a.gated) return a.plan.cut ? few_cut<2, true>(a, st, check_only) : few<2, true, -1>(a, st, check_only);
  if (two) return a.plan.cut ? few_cut<2, false>(a, st, check_only) : few<2, false, -1>(a, st, check_only);
  return a.plan.cut ? few_cut<1, false>(a, st, check_only) : few<1, false, -1>(a, st, check_only);
}

template <int BM, int BN, int WM, int WN, int NB, int KG, bool WIDE>
vq_status tiles(const F8Args& a, hipStream_t st, bool check_only) {
  if (a.gated) return launch_tile<BM, BN, WM, WN, NB, KG, WIDE, true, false>(a, st, check_only);
  if constexpr (KG == 1) {
    if (a.plan.splits > 1) {
      const vq_status e = launch_tile<BM, BN, WM, WN, NB, KG, WIDE, false, true>(a, st, check_only);
      return e != VQ_OK || check_only ? e : launch_join(a, st);
    }
  }
  return launch_tile<BM, BN, WM, WN, NB, KG, WIDE, false, false>(a, st, check_only);
}
template <bool WIDE>
vq_status run(const F8Args& a, hipStream_t st, bool check_only) {
  switch (a.plan.way) {
    case kStream1:
    case kStream2: return stream(a, st, check_only);
    case k32x32: return tiles<32, 32, 2, 1, 4, 2, WIDE>(a, st, check_only);
    case k32x64: return tiles<32, 64, 2, 2, 4, 1, WIDE>(a, st, check_only);
    case k64x64: return tiles<64, 64, 2, 2, 3, 2, WIDE>(a, st, check_only);
    case k64x128: return tiles<64, 128, 2, 4, 3, 1, WIDE>(a, st, check_only);
    case k128x128: return tiles<128, 128, 4, 2, 3, 1, WIDE>(a, st, check_only);
    case k128x128Pair: return tiles<128, 128, 2, 2, 2, 1, WIDE>(a, st, check_only);
    default:
      if constexpr (WIDE) {
        return a.y ? VQ_ERR_UNSUPPORTED : launch_big<true, true>(a, st, check_only);  // no plan has the first
      } else {
        return a.gated ? launch_big<true, false>(a, st, check_only) : launch_big<false, false>(a, st, check_only);
      }
  }
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
  const int64_t blocks = f8_blocks(a.k) * f8_blocks(a.rows);
  if (!grid_ok(blocks, 256)) return VQ_ERR_SHAPE;
  const dim3 g((uint32_t)blocks), b(256);
  switch (a.x_dtype) {
    case VQ_F32: f8_weights_kernel<VQ_F32><<<g, b, 0, st>>>(a); break;
    case VQ_F16: f8_weights_kernel<VQ_F16><<<g, b, 0, st>>>(a); break;
    default: f8_weights_kernel<VQ_BF16><<<g, b, 0, st>>>(a);
  }
  return done();
}

F8Plan f8_plan(int32_t m, int32_t n, int32_t k, bool gated, bool wide, bool may_cut) {
  const Shape shape(m, n, k, gated, wide);
  const int32_t steps = shape.steps;
  F8Plan best{-1, 1, false};
  float least = 0.f;
  const float quant = may_cut ? kQuantStart + 3.f * (float)m * (float)k / kQuantRate : 0.f;
  auto offer = [&](int32_t way, int32_t splits, bool cut) {
    const float t = cost(shape, way, splits, cut, wide) + (cut ? 0.f : quant);
    if (best.way < 0 || t < least) {
      least = t;
      best = F8Plan{way, splits, cut};
    }
  };
  for (int32_t way = 0; way < kWays; ++way) {
    const Cost& c = kCosts[wide][way];
    if (way <= kStream2) {
      if (m > 16 || (gated && way == kStream1)) continue;
      const int64_t groups = (shape.outputs + c.bn - 1) >> c.bn_log2;
      for (int32_t z = 1; z <= 16; z *= 2) {
        if (z > 1 && (gated || groups * z > kFewWorkgroups || steps / z < 8)) break;
        offer(way, z, false);
        if (may_cut && few_lds(way + 1, m, ceil_div(steps, z), true) <= kCutLds) offer(way, z, true);
      }
      continue;
    }
    if ((way == k256x256 && wide) || (c.bm > 64 && m <= 32)) continue;  // f8_big_plan; mostly empty tiles
    offer(way, 1, false);
    if (gated || c.groups_of_k > 1 || way == k256x256) continue;
    // K is cut where the tiles leave CUs without work, into four steps at least
    const int64_t t = (((int64_t)m + c.bm - 1) >> c.bm_log2) * ((shape.outputs + c.bn - 1) >> c.bn_log2);
    for (const int32_t z : {2, 3, 4, 6, 8, 12, 16}) {
      if (t * z > 300 || steps < 4 * z) break;
      offer(way, z, false);
    }
  }
  return best;
}

bool f8_big_plan(int32_t m, int32_t n, int32_t k, F8Plan& plan) {
  // what the hidden rows cost otherwise: written and read in fp32, written in 8 bits, in a launch of their own
  const float spared = kQuantStart + 9.f * (float)m * (float)n / kQuantRate;
  const Shape s(m, n, k, true, true);
  if (cost(s, k256x256, 1, false, true) > cost(s, plan.way, plan.splits, plan.cut, true) + spared) return false;
  plan = F8Plan{k256x256, 1, false};
  return true;
}

vq_status launch_f8(const F8Args& a, void* stream, bool check_only) {
  hipStream_t st = (hipStream_t)stream;
  return a.wide ? run<true>(a, st, check_only) : run<false>(a, st, check_only);
}

}  // namespace vqi
