// Host side of the 8-bit float layers: argument checks, workspace layouts and the exported entry points vq_f8_*.
#include <algorithm>
#include <cstring>

#include "vq_host_checks.h"
#include "vq_internal.h"

namespace vqi {
namespace {

bool valid_k(int32_t k) { return k >= 1 && k <= kF8MaxK; }

// Most rows and outputs: the edge of the last tile is still an int32.
constexpr int32_t kMaxRows = INT32_MAX - 1024;

vq_status check_sizes(int32_t M, int32_t N, int32_t K, int32_t gated) {
  if (M < 0 || M > kMaxRows || N < 0 || N > (gated ? INT32_MAX / 2 : kMaxRows) || !valid_k(K)) return VQ_ERR_SHAPE;
  return gated == 0 || gated == 1 ? VQ_OK : VQ_ERR_UNSUPPORTED;
}

size_t part_bytes(int32_t m, int32_t n, const F8Plan& p) { return p.splits > 1 ? (size_t)p.splits * (size_t)m * (size_t)n * 4 : 0; }

// Most partial sums of a product of this shape, whatever the type of its outputs.
size_t most_part_bytes(int32_t m, int32_t n, int32_t k, bool gated) {
  if (m == 0 || n == 0) return 0;
  return std::max(part_bytes(m, n, f8_plan(m, n, k, gated, false, false)), part_bytes(m, n, f8_plan(m, n, k, gated, true, false)));
}

// A product of tokens that are cut to 8 bits on the way: inside it, or in front of it, into q and s; and its partial sums.
struct LinearWs {
  F8Plan plan;
  uint8_t* q;
  float* s;
  float* part;
  size_t bytes;
};
LinearWs linear_ws(int32_t m, int32_t n, int32_t k, bool gated, bool wide, void* base) {
  LinearWs w;
  std::memset(&w, 0, sizeof w);
  if (m == 0 || n == 0) return w;
  w.plan = f8_plan(m, n, k, gated, wide, true);
  Pieces p{(uint8_t*)base};
  w.q = (uint8_t*)p.take(w.plan.cut ? 0 : (size_t)m * (size_t)q8_row_bytes(k));
  w.s = (float*)p.take(w.plan.cut ? 0 : (size_t)m * (size_t)f8_blocks(k) * 4);
  w.part = (float*)p.take(part_bytes(m, n, w.plan));
  w.bytes = p.at;
  return w;
}
size_t most_linear_bytes(int32_t m, int32_t n, int32_t k, bool gated) {
  return std::max(linear_ws(m, n, k, gated, false, nullptr).bytes, linear_ws(m, n, k, gated, true, nullptr).bytes);
}

// Between the two products of an MLP: the hidden rows in fp32, or in 8 bits where the first product writes them so; and
// one piece that both products use in turn.  The gated product's sums are in fp32 for outputs of every type: the 8-bit
// instruction's move hidden values over the border of two e4m3 steps, and bf16 outputs were then off by 0.8e-3 to 1.4e-3
// (rms) beside the 1.7e-3 of their own rounding.  2048 x 4096 x 14336: 388 us with those, 571 to 597 without.
struct MlpWs {
  bool writes_q;
  float* h;
  uint8_t* hq;
  float* hs;
  LinearWs in, out;
  size_t bytes;
};
MlpWs mlp_ws(int32_t m, int32_t d, int32_t i, vq_dtype y_dtype, void* base) {
  MlpWs w;
  std::memset(&w, 0, sizeof w);
  if (m == 0) return w;
  w.in = linear_ws(m, i, d, true, true, nullptr);
  w.out = linear_ws(m, d, i, false, y_dtype == VQ_F32, nullptr);
  F8Plan big = w.in.plan;
  w.writes_q = f8_big_plan(m, i, d, big);
  Pieces p{(uint8_t*)base};
  w.h = (float*)p.take(w.writes_q ? 0 : (size_t)m * (size_t)i * 4);
  w.hq = (uint8_t*)p.take(w.writes_q ? (size_t)m * (size_t)q8_row_bytes(i) : 0);
  w.hs = (float*)p.take(w.writes_q ? (size_t)m * (size_t)f8_blocks(i) * 4 : 0);
  if (w.writes_q) {
    w.in.plan = big;  // its tokens are cut in front of it
    w.in.bytes = padded((size_t)m * (size_t)q8_row_bytes(d)) + padded((size_t)m * (size_t)f8_blocks(d) * 4);
    w.out.plan = f8_plan(m, d, i, false, y_dtype == VQ_F32, false);
    w.out.bytes = padded(part_bytes(m, d, w.out.plan));
  }
  void* const products = p.take(std::max(w.in.bytes, w.out.bytes));
  auto place = [&](LinearWs& l, int32_t k, int32_t n, bool tokens) {
    Pieces at{(uint8_t*)products};
    l.q = (uint8_t*)at.take(tokens ? (size_t)m * (size_t)q8_row_bytes(k) : 0);
    l.s = (float*)at.take(tokens ? (size_t)m * (size_t)f8_blocks(k) * 4 : 0);
    l.part = (float*)at.take(part_bytes(m, n, l.plan));
  };
  place(w.in, d, i, !w.in.plan.cut);
  place(w.out, i, d, !w.out.plan.cut && !w.writes_q);
  w.bytes = p.at;
  return w;
}

vq_status quantize(int32_t m, int32_t k, const void* x, vq_dtype t, int64_t ldx, uint8_t* q, float* s, void* stream,
                   bool check_only) {
  F8QuantArgs a;
  std::memset(&a, 0, sizeof a);
  a.rows = m;
  a.k = k;
  a.x = x;
  a.x_dtype = t;
  a.ldx = ldx;
  a.q = q;
  a.s = s;
  return launch_f8_tokens(a, stream, check_only);
}

F8Args product(int32_t m, int32_t n, int32_t k, const void* w, const float* sw, const void* bias, int32_t gated, void* y,
               vq_dtype y_dtype) {
  F8Args a;
  std::memset(&a, 0, sizeof a);
  a.m = m;
  a.n = n;
  a.k = k;
  a.w = (const uint8_t*)w;
  a.sw = sw;
  a.bias = (const uint16_t*)bias;
  a.gated = gated;
  a.y = y;
  a.y_dtype = y_dtype;
  a.wide = y_dtype == VQ_F32;
  return a;
}

// The product `a` of tokens x [m][k] that are cut to 8 bits on the way.
vq_status linear(F8Args a, const void* x, vq_dtype x_dtype, int64_t ldx, const LinearWs& ws, void* stream, bool check_only) {
  a.plan = ws.plan;
  a.part = ws.part;
  if (a.plan.cut) {
    a.x = x;
    a.x_dtype = x_dtype;
    a.ldx = ldx;
  } else {
    const vq_status st = quantize(a.m, a.k, x, x_dtype, ldx, ws.q, ws.s, stream, check_only);
    if (st != VQ_OK) return st;
    a.q = ws.q;
    a.s = ws.s;
  }
  return launch_f8(a, stream, check_only);
}

}  // namespace
}  // namespace vqi

using namespace vqi;

extern "C" {

vq_status vq_f8_quantize(int32_t rows, int32_t k, int32_t block_rows, const void* x, vq_dtype x_dtype, int64_t ldx, void* q,
                         float* s, void* stream) {
  if (rows < 0 || rows > kMaxRows || !valid_k(k) || ldx < k) return VQ_ERR_SHAPE;
  if (!valid_dtype(x_dtype) || (block_rows != 1 && block_rows != kF8Block)) return VQ_ERR_UNSUPPORTED;
  if (rows == 0) return VQ_OK;
  if (!x || !q || !s) return VQ_ERR_NULL;
  if (!aligned(x, size_of(x_dtype)) || !aligned(q, 16) || !aligned(s, 4)) return VQ_ERR_ALIGN;
  if (block_rows == 1) return quantize(rows, k, x, x_dtype, ldx, (uint8_t*)q, s, stream, false);
  F8QuantArgs a;
  std::memset(&a, 0, sizeof a);
  a.rows = rows;
  a.k = k;
  a.x = x;
  a.x_dtype = x_dtype;
  a.ldx = ldx;
  a.q = (uint8_t*)q;
  a.s = s;
  return launch_f8_weights(a, stream);
}

vq_status vq_f8_gemm_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t gated, size_t* nbytes) {
  if (!nbytes) return VQ_ERR_NULL;
  const vq_status st = check_sizes(M, N, K, gated);
  if (st != VQ_OK) return st;
  *nbytes = most_part_bytes(M, N, K, gated);
  return VQ_OK;
}

vq_status vq_f8_gemm(int32_t M, int32_t N, int32_t K, const void* q, const float* s, const void* w, const float* sw,
                     const void* bias, int32_t gated, void* y, vq_dtype y_dtype, void* workspace, size_t workspace_bytes,
                     void* stream) {
  const vq_status st = check_sizes(M, N, K, gated);
  if (st != VQ_OK) return st;
  if (!valid_dtype(y_dtype)) return VQ_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return VQ_OK;
  if (!q || !s || !w || !sw || !y) return VQ_ERR_NULL;
  if (!aligned(q, 16) || !aligned(w, 16) || !aligned(s, 4) || !aligned(sw, 4) || misaligned(bias, 2) ||
      !aligned(y, size_of(y_dtype)))
    return VQ_ERR_ALIGN;
  F8Args a = product(M, N, K, w, sw, bias, gated, y, y_dtype);
  a.q = (const uint8_t*)q;
  a.s = s;
  a.plan = f8_plan(M, N, K, gated, a.wide, false);
  if (workspace && a.plan.splits > 1) {
    if (workspace_bytes < part_bytes(M, N, a.plan)) return VQ_ERR_BUFFER_SIZE;
    if (!aligned(workspace, 256)) return VQ_ERR_ALIGN;
    a.part = (float*)workspace;
  } else {
    a.plan.splits = 1;
  }
  return launch_f8(a, stream);
}

vq_status vq_f8_linear_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t gated, size_t* nbytes) {
  if (!nbytes) return VQ_ERR_NULL;
  const vq_status st = check_sizes(M, N, K, gated);
  if (st != VQ_OK) return st;
  *nbytes = most_linear_bytes(M, N, K, gated);
  return VQ_OK;
}

vq_status vq_f8_linear(int32_t M, int32_t N, int32_t K, const void* x, vq_dtype x_dtype, int64_t ldx, const void* w,
                       const float* sw, const void* bias, int32_t gated, void* y, vq_dtype y_dtype, void* workspace,
                       size_t workspace_bytes, void* stream) {
  vq_status st = check_sizes(M, N, K, gated);
  if (st != VQ_OK) return st;
  if (ldx < K) return VQ_ERR_SHAPE;
  if (!valid_dtype(x_dtype) || !valid_dtype(y_dtype)) return VQ_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return VQ_OK;
  const LinearWs ws = linear_ws(M, N, K, gated, y_dtype == VQ_F32, workspace);
  if (!x || !w || !sw || !y || (!workspace && ws.bytes > 0)) return VQ_ERR_NULL;
  if (!aligned(x, size_of(x_dtype)) || !aligned(w, 16) || !aligned(sw, 4) || misaligned(bias, 2) ||
      !aligned(y, size_of(y_dtype)) || misaligned(workspace, 256))
    return VQ_ERR_ALIGN;
  if (workspace_bytes < ws.bytes) return VQ_ERR_BUFFER_SIZE;
  if (x == y) return VQ_ERR_UNSUPPORTED;  // tokens that are cut inside are read while outputs are stored
  const F8Args a = product(M, N, K, w, sw, bias, gated, y, y_dtype);
  if ((st = linear(a, x, x_dtype, ldx, ws, stream, true)) != VQ_OK) return st;
  return linear(a, x, x_dtype, ldx, ws, stream, false);
}

vq_status vq_f8_mlp_workspace_bytes(int32_t M, int32_t D, int32_t I, size_t* nbytes) {
  if (!nbytes) return VQ_ERR_NULL;
  if (M < 0 || M > kMaxRows || !valid_k(D) || !valid_k(I)) return VQ_ERR_SHAPE;
  *nbytes = 0;
  for (const vq_dtype t : {VQ_F16, VQ_BF16, VQ_F32}) *nbytes = std::max(*nbytes, mlp_ws(M, D, I, t, nullptr).bytes);
  return VQ_OK;
}

vq_status vq_f8_mlp(int32_t M, int32_t D, int32_t I, const void* x, vq_dtype x_dtype, int64_t ldx, const void* w_in,
                    const float* s_in, const void* w_out, const float* s_out, void* y, vq_dtype y_dtype, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (M < 0 || M > kMaxRows || !valid_k(D) || !valid_k(I) || ldx < D) return VQ_ERR_SHAPE;
  if (!valid_dtype(x_dtype) || !valid_dtype(y_dtype)) return VQ_ERR_UNSUPPORTED;
  if (M == 0) return VQ_OK;
  if (!x || !w_in || !s_in || !w_out || !s_out || !y || !workspace) return VQ_ERR_NULL;
  if (!aligned(x, size_of(x_dtype)) || !aligned(w_in, 16) || !aligned(w_out, 16) || !aligned(s_in, 4) ||
      !aligned(s_out, 4) || !aligned(y, size_of(y_dtype)) || !aligned(workspace, 256))
    return VQ_ERR_ALIGN;
  const MlpWs ws = mlp_ws(M, D, I, y_dtype, workspace);
  if (workspace_bytes < ws.bytes) return VQ_ERR_BUFFER_SIZE;
  F8Args gate = product(M, I, D, w_in, s_in, nullptr, 1, ws.writes_q ? nullptr : ws.h, VQ_F32);
  gate.yq = ws.hq;
  gate.ys = ws.hs;
  F8Args last = product(M, D, I, w_out, s_out, nullptr, 0, y, y_dtype);
  auto run = [&](bool check_only) {
    const vq_status st = linear(gate, x, x_dtype, ldx, ws.in, stream, check_only);
    if (st != VQ_OK) return st;
    if (!ws.writes_q) return linear(last, ws.h, VQ_F32, I, ws.out, stream, check_only);
    F8Args a = last;
    a.plan = ws.out.plan;
    a.part = ws.out.part;
    a.q = ws.hq;
    a.s = ws.hs;
    return launch_f8(a, stream, check_only);
  };
  const vq_status st = run(true);
  return st != VQ_OK ? st : run(false);
}

}  // extern "C"
