// vq_rotate_heads: norms of the queries' and keys' heads and their rotary positions, one pass over both.
//
//   v = N(x) over a head's values (identity, RMS or centred, weight and bias)
//   pairs (a, b) of the rotated part:  a' = c (a cos t - b sin t),  b' = c (a sin t + b cos t),  t = position * frequency
//
// The angle is formed in fp64, in turns, where the product is off by 2^-53 of itself at most, and reduced there to an eighth
// of a turn: what is left goes to fp32 with an error of 2^-27 turns.  That is the larger one up to 2^26 turns (2^28 positions
// of a pair that turns by one radian each); at 2^40 positions the product's is 2^-16 turns, at 2^52 2^-4.  The sines of a
// workgroup's tokens are computed once, one pair per thread, and shared by all heads in LDS.
//
// A head is held by L lanes (a power of two), 16 values each: 8 pairs of the rotated part, or 16 values of the parts beside
// it.  Every value is read once and written once; the norm's sums go over the L lanes, up to 16 of them without LDS.
//
// Bound by the bytes: 8192 tokens, 64 + 8 heads of 128 in bf16, 302 MB, 58 us rotated (5.2 TB/s; a large copy reaches 5.1)
// and 65 us with norms, whose chain of sums the wavefronts of a CU do not quite hide.  A decode step is the launch and one
// chain position - sine - store: 4.2 to 4.6 us in a trace.
#include "vq_device.h"
#include "vq_f8_device.h"
#include "vq_q8_device.h"

namespace {

using vqi::HeadsArgs;

constexpr int kThreads = 256;
constexpr int kSines = 1024;  // pairs of all tokens of a workgroup
// Pairs of a token in LDS: whole pieces of 8, read as such.
constexpr int32_t pairs_of(int32_t rot) { return (rot / 2 + 7) / 8 * 8; }

// Sum over groups of `lanes` consecutive lanes, the same bits in all of them.
template <int CTRL>
__device__ __forceinline__ float other(float v) {
  return __builtin_bit_cast(float, vqd::other<CTRL>(__builtin_bit_cast(uint32_t, v)));
}
__device__ __forceinline__ float group_sum(float v, int lanes) {
  if (lanes > 1) v += other<vqd::kXor1>(v);
  if (lanes > 2) v += other<vqd::kXor2>(v);
  if (lanes > 4) v += other<vqd::kHalf>(v);
  if (lanes > 8) v += other<vqd::kRow>(v);
  if (lanes > 16) v += __shfl_xor(v, 16, 64);
  if (lanes > 32) v += __shfl_xor(v, 32, 64);
  return v;
}

// Where a lane's item lies in a head: 8 values from `a` on and 8 from `b` on, `na` and `nb` of them there.  Neighbouring
// lanes take neighbouring pieces of 8 of a part, and as many further on the other halves of their items, so that every load
// and store of a wavefront is one run.  `pair`, `pair_b`: the first pairs of the two halves (half layout: of the first four
// and the next four of the item's pairs), -1 beside the rotated part.
struct Item {
  int32_t a, b, na, nb, pair, pair_b;
};
__device__ __forceinline__ Item item_at(const HeadsArgs& h, int32_t i) {
  Item r{0, 0, 0, 0, -1, -1};
  const int32_t half = h.rot / 2, front = (h.start + 15) / 16, turned = (half + 7) / 8;
  int32_t from, end, items;
  if (i < front) {
    from = 0;
    end = h.start;
    items = front;
  } else if (i < front + turned) {
    i -= front;
    if (!h.interleaved) {
      r.pair = 8 * i;
      r.pair_b = r.pair + 4;
      r.a = h.start + r.pair;
      r.b = r.a + half;
      r.na = r.nb = min(8, half - r.pair);
      return r;
    }
    from = h.start;
    end = from + h.rot;
    items = turned;
    r.pair = 4 * i;
    r.pair_b = 4 * (i + items);
  } else {
    i -= front + turned;
    from = h.start + h.rot;
    end = h.dim;
    items = (end - from + 15) / 16;
  }
  r.a = from + 8 * i;
  r.b = r.a + 8 * items;
  r.na = i < items ? min(max(end - r.a, 0), 8) : 0;  // lanes beyond the last item hold nothing
  r.nb = i < items ? min(max(end - r.b, 0), 8) : 0;
  return r;
}
inline int32_t items_of(const HeadsArgs& h) {
  return (h.start + 15) / 16 + (h.rot / 2 + 7) / 8 + (h.dim - h.start - h.rot + 15) / 16;
}

template <vq_dtype XT>
struct Bits {
  static constexpr int kWords = XT == VQ_F32 ? 8 : 4;
  uint32_t v[2][kWords];
};
// `n` of 8 values at p; zeros behind.
template <vq_dtype XT>
__device__ __forceinline__ void load_bits(const char* p, int32_t n, uint32_t (&v)[Bits<XT>::kWords]) {
  constexpr int es = XT == VQ_F32 ? 4 : 2;
  if (n == 8) {
    __builtin_memcpy(v, p, 8 * es);
  } else {
#pragma unroll
    for (int k = 0; k < Bits<XT>::kWords; ++k) {
      if constexpr (XT == VQ_F32) {
        v[k] = k < n ? ((const uint32_t*)p)[k] : 0u;
      } else {
        v[k] = (2 * k < n ? ((const uint16_t*)p)[2 * k] : 0u) | (2 * k + 1 < n ? ((const uint16_t*)p)[2 * k + 1] : 0u) << 16;
      }
    }
  }
}
template <vq_dtype XT>
__device__ __forceinline__ float value(const uint32_t (&v)[Bits<XT>::kWords], int k) {
  if constexpr (XT == VQ_F32) {
    return __builtin_bit_cast(float, v[k]);
  } else {
    return vqd::x_to_f32<XT == VQ_F16 ? 0 : 1>(v[k / 2] >> (16 * (k & 1)));
  }
}
// `n` of 8 values of a vector at `at`; zeros behind.
__device__ __forceinline__ void load_vec(const void* p, vq_dtype t, int32_t at, int32_t n, float* f) {
  if (t == VQ_F32) {
    uint32_t v[8];
    load_bits<VQ_F32>((const char*)p + (int64_t)at * 4, n, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = value<VQ_F32>(v, k);
  } else {
    uint32_t v[4];
    load_bits<VQ_F16>((const char*)p + (int64_t)at * 2, n, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = t == VQ_F16 ? value<VQ_F16>(v, k) : value<VQ_BF16>(v, k);
  }
}
// 16 bytes, past the caches where STREAM.
template <bool STREAM>
__device__ __forceinline__ void store16(void* p, const uint32_t* v) {
  if constexpr (STREAM) {
    typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(2)));
    __builtin_nontemporal_store(u4{v[0], v[1], v[2], v[3]}, (u4*)p);
  } else {
    __builtin_memcpy(p, v, 16);
  }
}
template <bool STREAM>
__device__ __forceinline__ void store_part(char* row, vq_dtype t, int32_t at, int32_t n, const float* f) {
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = f[k];
  if (t == VQ_F32) {
    float* p = (float*)row + at;
    if (n == 8) {
      store16<STREAM>(p, (const uint32_t*)v);
      store16<STREAM>(p + 4, (const uint32_t*)v + 4);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) p[k] = v[k];
    }
  } else {
    uint16_t h[8];
    vqd::narrow<8>(v, t, h);
    uint16_t* p = (uint16_t*)row + at;
    if (n == 8) {
      uint32_t w[4];
      __builtin_memcpy(w, h, 16);
      store16<STREAM>(p, w);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) p[k] = h[k];
    }
  }
}

// A workgroup takes `tt` tokens (of batch * tokens, from blockIdx.x * tt on) and `per` heads (of queries and keys in a row,
// from blockIdx.y * per on).  Its groups of `lanes` lanes are dealt to the tokens, 256 / lanes / tt to each, and take its
// heads in turn, with the token's sines in registers and the next head on its way.  I items per lane.
template <int I, int NORM, vq_dtype XT, bool INTER>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadsArgs a, int32_t lanes, int32_t tt, int32_t per) {
  __shared__ __attribute__((aligned(16))) float cs[kSines], sn[kSines];
  const int64_t all = (int64_t)a.batch * a.tokens;
  const int64_t bt0 = (int64_t)blockIdx.x * tt;
  const int32_t here = (int32_t)min((int64_t)tt, all - bt0);
  const int32_t half = a.rot / 2, pairs = pairs_of(a.rot);
  const int32_t groups = kThreads / lanes / tt, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  const int32_t mine = group / groups, sub = group % groups;  // this group's token, and which of the token's groups it is
  const bool there = mine < here;  // idle groups go along: barriers, and sums over whole groups of lanes
  const int64_t bt = bt0 + (there ? mine : 0), b = bt / a.tokens, t = bt - b * a.tokens;
  constexpr int es = XT == VQ_F32 ? 4 : 2;
  const int ey = a.y_dtype == VQ_F32 ? 4 : 2;

  Item it[I];
#pragma unroll
  for (int n = 0; n < I; ++n) it[n] = item_at(a, lane + n * lanes);

  for (int32_t i = threadIdx.x; i < here * half; i += kThreads) {
    const int32_t tok = i / half, j = i - tok * half;
    const int64_t p_bt = bt0 + tok;
    const int64_t p_b = p_bt / a.tokens, at = p_b * a.pos_stride + (p_bt - p_b * a.tokens);
    const double p = a.pos_64 ? (double)((const int64_t*)a.positions)[at] : (double)((const int32_t*)a.positions)[at];
    const double turn = p * a.freqs[j];
    const double r = turn - __builtin_rint(turn);
    const double quarter = __builtin_rint(4.0 * r);
    float s, c;
    sincospif((float)(2.0 * (r - 0.25 * quarter)), &s, &c);  // up to a quarter of a half turn
    const int q = (int)quarter & 3;
    const float c1 = q & 1 ? s : c, s1 = q & 1 ? c : s;
    cs[tok * pairs + j] = (q == 1 || q == 2 ? -c1 : c1) * a.scale;
    sn[tok * pairs + j] = (q >= 2 ? -s1 : s1) * a.scale;
  }
  __syncthreads();
  float co[I][8], si[I][8];  // pairs past the part's end: what the array holds, for values that are not stored
#pragma unroll
  for (int n = 0; n < I; ++n) {
    const int32_t at = (there ? mine : 0) * pairs, p = at + max(it[n].pair, 0), q = at + max(it[n].pair_b, 0);
    __builtin_memcpy(co[n], cs + p, 16);
    __builtin_memcpy(co[n] + 4, cs + q, 16);
    __builtin_memcpy(si[n], sn + p, 16);
    __builtin_memcpy(si[n] + 4, sn + q, 16);
  }
  const float inv_d = 1.0f / (float)a.dim;

  for (int part = 0; part < 2; ++part) {
    const int32_t first = part ? a.heads[0] : 0;  // of this part, among all heads
    const int32_t h0 = max((int32_t)blockIdx.y * per - first, 0);
    const int32_t h1 = min(((int32_t)blockIdx.y + 1) * per - first, a.heads[part]);
    if (h0 >= h1) continue;
    const char* const x = (const char*)a.x[part] + (b * a.xs[part][0] + t * a.xs[part][1]) * es;
    char* const y = (char*)a.y[part] + (b * a.ys[part][0] + t * a.ys[part][1]) * ey;
    Bits<XT> raw[I];
    auto ask = [&](int32_t h) {  // a head past the last one is the first again
      const char* p = x + (int64_t)(h < h1 ? h : h0) * a.xs[part][2] * es;
#pragma unroll
      for (int n = 0; n < I; ++n) {
        load_bits<XT>(p + (int64_t)it[n].a * es, it[n].na, raw[n].v[0]);
        load_bits<XT>(p + (int64_t)it[n].b * es, it[n].nb, raw[n].v[1]);
      }
    };
    ask(h0 + sub);
    float w[NORM ? I : 1][16];
    if constexpr (NORM) {
#pragma unroll
      for (int n = 0; n < I; ++n) {
#pragma unroll
        for (int k = 0; k < 16; ++k) w[n][k] = 1.f;
        if (a.w[part]) {
          load_vec(a.w[part], a.w_dtype, it[n].a, it[n].na, w[n]);
          load_vec(a.w[part], a.w_dtype, it[n].b, it[n].nb, w[n] + 8);
#pragma unroll
          for (int k = 0; k < 16; ++k) w[n][k] += a.w_offset;
        }
      }
    }
    for (int32_t hp = h0; hp < h1; hp += groups) {
      const int32_t h = hp + sub;
      float f[I][16];
#pragma unroll
      for (int n = 0; n < I; ++n)
#pragma unroll
        for (int k = 0; k < 16; ++k) f[n][k] = value<XT>(raw[n].v[k / 8], k % 8);
      if (hp + groups < h1) ask(h + groups);
      if constexpr (NORM != VQ_NORM_NONE) {
        if constexpr (NORM == VQ_NORM_LAYER) {
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < I; ++n)
#pragma unroll
            for (int k = 0; k < 16; ++k) sum += f[n][k];  // zeros past the ends
          const float mean = group_sum(sum, lanes) * inv_d;
#pragma unroll
          for (int n = 0; n < I; ++n)
#pragma unroll
            for (int k = 0; k < 16; ++k) f[n][k] = k % 8 < (k < 8 ? it[n].na : it[n].nb) ? f[n][k] - mean : 0.f;
        }
        float sq = 0.f;
#pragma unroll
        for (int n = 0; n < I; ++n)
#pragma unroll
          for (int k = 0; k < 16; ++k) sq = __builtin_fmaf(f[n][k], f[n][k], sq);
        const float inv = 1.0f / __builtin_sqrtf(group_sum(sq, lanes) * inv_d + a.eps);
#pragma unroll
        for (int n = 0; n < I; ++n) {
          if (a.b[part]) {
            float bias[16];
            load_vec(a.b[part], a.w_dtype, it[n].a, it[n].na, bias);
            load_vec(a.b[part], a.w_dtype, it[n].b, it[n].nb, bias + 8);
#pragma unroll
            for (int k = 0; k < 16; ++k) f[n][k] = __builtin_fmaf(f[n][k] * inv, w[n][k], bias[k]);
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) f[n][k] = f[n][k] * inv * w[n][k];
          }
        }
      }
#pragma unroll
      for (int n = 0; n < I; ++n) {
        if (it[n].pair >= 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float u = INTER ? f[n][2 * k] : f[n][k], v = INTER ? f[n][2 * k + 1] : f[n][8 + k];
            (INTER ? f[n][2 * k] : f[n][k]) = __builtin_fmaf(u, co[n][k], -(v * si[n][k]));
            (INTER ? f[n][2 * k + 1] : f[n][8 + k]) = __builtin_fmaf(u, si[n][k], v * co[n][k]);
          }
        }
        if (there && h < h1) {
          char* p = y + (int64_t)h * a.ys[part][2] * ey;
          if (a.streams) {
            store_part<true>(p, a.y_dtype, it[n].a, it[n].na, f[n]);
            store_part<true>(p, a.y_dtype, it[n].b, it[n].nb, f[n] + 8);
          } else {
            store_part<false>(p, a.y_dtype, it[n].a, it[n].na, f[n]);
            store_part<false>(p, a.y_dtype, it[n].b, it[n].nb, f[n] + 8);
          }
        }
      }
    }
  }
}

template <int I, int NORM, vq_dtype XT>
void launch_t(const HeadsArgs& a, dim3 g, int32_t lanes, int32_t tt, int32_t per, hipStream_t st) {
  if (a.interleaved) heads_kernel<I, NORM, XT, true><<<g, dim3(kThreads), 0, st>>>(a, lanes, tt, per);
  else heads_kernel<I, NORM, XT, false><<<g, dim3(kThreads), 0, st>>>(a, lanes, tt, per);
}
template <int I, int NORM>
void launch(const HeadsArgs& a, dim3 g, int32_t lanes, int32_t tt, int32_t per, hipStream_t st) {
  switch (a.x_dtype) {
    case VQ_F32: launch_t<I, NORM, VQ_F32>(a, g, lanes, tt, per, st); break;
    case VQ_F16: launch_t<I, NORM, VQ_F16>(a, g, lanes, tt, per, st); break;
    default: launch_t<I, NORM, VQ_BF16>(a, g, lanes, tt, per, st);
  }
}

// Workgroups up to which a token's heads are spread over more lanes rather than taken in turn: two for each CU.
constexpr int64_t kWorkgroups = 512;

}  // namespace

namespace vqi {

vq_status launch_heads(const HeadsArgs& args, void* stream) {
  HeadsArgs a = args;
  hipStream_t st = (hipStream_t)stream;
  const int32_t items = items_of(a);
  int32_t lanes = 1;
  while (lanes < items && lanes < 64) lanes *= 2;
  if (items > 2 * lanes) return VQ_ERR_SHAPE;
  const int64_t all = (int64_t)a.batch * a.tokens;
  const int32_t heads = a.heads[0] + a.heads[1], groups = kThreads / lanes;
  // tokens of a workgroup: as many as leave each group of lanes so many heads at most, fit the sines' place and leave the CUs
  // work.  8192 tokens, 64 + 8 heads of 128, 4, 8 and 16 heads a group: rotated 59, 59 and 63 us (half a head 64, 69 and 74),
  // with norms, whose weights a group loads once, 77, 66 and 66
  const int32_t turns = a.norm == VQ_NORM_NONE ? 4 : 8;
  int32_t tt = groups, per = heads;
  while (tt > 1 && (tt * pairs_of(a.rot) > kSines || groups / tt * turns < heads || (all + tt - 1) / tt < kWorkgroups)) tt /= 2;
  if (tt == 1 && all < kWorkgroups) per = groups;  // one head for each group
  const int64_t gx = (all + tt - 1) / tt, gy = ((int64_t)heads + per - 1) / per;
  if (gy > 65535 || !grid_ok(gx * gy, kThreads)) return VQ_ERR_SHAPE;
  // one's output where the other is read or written: workgroups take the heads of both in any order
  if (a.heads[0] > 0 && a.heads[1] > 0 && (a.y[0] == a.y[1] || a.y[0] == a.x[1] || a.y[1] == a.x[0])) return VQ_ERR_UNSUPPORTED;
  // Outputs that the L2s (8 of 4 MB) would not hold for whoever reads them next go past them: 8192 tokens of 64 + 8 heads of
  // 128 in bf16, 151 MB each way, 74 us through the caches and 62 past them (with norms 75 and 67, half a head rotated 97 and
  // 73); 512 tokens of 32 + 8 heads 6.7 us either way
  a.streams = all * heads * a.dim * (a.y_dtype == VQ_F32 ? 4 : 2) > (int64_t)32 << 20;
  const dim3 g((uint32_t)gx, (uint32_t)gy);
  const bool two = items > lanes;
  switch (a.norm) {
    case VQ_NORM_NONE: two ? launch<2, VQ_NORM_NONE>(a, g, lanes, tt, per, st) : launch<1, VQ_NORM_NONE>(a, g, lanes, tt, per, st); break;
    case VQ_NORM_RMS: two ? launch<2, VQ_NORM_RMS>(a, g, lanes, tt, per, st) : launch<1, VQ_NORM_RMS>(a, g, lanes, tt, per, st); break;
    default: two ? launch<2, VQ_NORM_LAYER>(a, g, lanes, tt, per, st) : launch<1, VQ_NORM_LAYER>(a, g, lanes, tt, per, st);
  }
  return hipGetLastError() == hipSuccess ? VQ_OK : VQ_ERR_HIP;
}

}  // namespace vqi
