// Host side of the 8-bit operators: argument checks, workspace layouts and the exported
// entry points vq_q8_*, vq_expert_* and vq_block_norm.
#include <cstring>

#include "vq_internal.h"

namespace vqi {
namespace {

constexpr int64_t kMaxPairs = (int64_t)1 << 30;
constexpr int32_t kMaxExperts = 4096;

bool valid_dtype(vq_dtype t) { return t == VQ_F16 || t == VQ_BF16 || t == VQ_F32; }
size_t size_of(vq_dtype t) { return t == VQ_F32 ? 4 : 2; }
bool valid_k(int32_t k) { return k >= 1 && k <= kQ8MaxK; }
size_t padded(size_t n) { return (n + 255) / 256 * 256; }
bool misaligned(const void* p, size_t a) { return p && !aligned(p, a); }

// Consecutive 256-byte aligned pieces of a workspace.
struct Pieces {
  uint8_t* base;
  size_t at = 0;
  void* take(size_t n) {
    void* p = base ? base + at : nullptr;
    at += padded(n);
    return p;
  }
};

size_t part_bytes(int32_t m, int32_t n, int32_t k, int32_t* splits) {
  *splits = m > 0 && n > 0 ? q8_splits(m, n, k) : 1;
  return *splits > 1 ? (size_t)*splits * (size_t)m * (size_t)n * 4 : 0;
}

struct LinearWs {
  uint8_t* q;
  float* s;
  int32_t* part;
  int32_t splits;
  size_t bytes;
};
LinearWs linear_ws(int32_t m, int32_t n, int32_t k, void* base) {
  LinearWs w;
  Pieces p{(uint8_t*)base};
  w.q = (uint8_t*)p.take((size_t)m * (size_t)q8_row_bytes(k));
  w.s = (float*)p.take((size_t)m * 4);
  w.part = (int32_t*)p.take(part_bytes(m, n, k, &w.splits));
  w.bytes = m > 0 && n > 0 ? p.at : 0;
  return w;
}

struct ExpertsWs {
  int32_t *offsets, *rows, *pos;
  uint8_t *xq, *hq;
  float *xs, *hs, *h, *z;
  size_t bytes;
};
ExpertsWs experts_ws(int32_t tokens, int32_t top, int32_t experts, int32_t d, int32_t i, void* base) {
  ExpertsWs w;
  Pieces p{(uint8_t*)base};
  const size_t r = (size_t)tokens * (size_t)top;
  w.offsets = (int32_t*)p.take(((size_t)experts + 1) * 4);
  w.rows = (int32_t*)p.take(r * 4);
  w.pos = (int32_t*)p.take(r * 4);
  w.xq = (uint8_t*)p.take((size_t)tokens * (size_t)q8_row_bytes(d));
  w.xs = (float*)p.take((size_t)tokens * 4);
  w.h = (float*)p.take(r * (size_t)i * 4);
  w.hq = (uint8_t*)p.take(r * (size_t)q8_row_bytes(i));
  w.hs = (float*)p.take(r * 4);
  w.z = (float*)p.take(r * (size_t)d * 4);
  w.bytes = tokens > 0 ? p.at : 0;
  return w;
}

vq_status check_routing(int32_t tokens, int32_t top, int32_t experts) {
  if (tokens < 0 || top < 1 || experts < 1 || experts > kMaxExperts || (int64_t)tokens * top >= kMaxPairs)
    return VQ_ERR_SHAPE;
  return VQ_OK;
}

vq_status quantize(int32_t rows, int32_t k, const void* x, vq_dtype t, int64_t ldx, uint8_t* q, float* s,
                   void* stream, bool check_only = false) {
  NormArgs a;
  std::memset(&a, 0, sizeof a);
  a.rows = rows;
  a.dim = k;
  a.z = x;
  a.z_dtype = t;
  a.ldz = ldx;
  a.gate_rows = 1;
  a.q = q;
  a.s = s;
  return launch_norm(a, stream, check_only);
}

vq_status grouped(int32_t experts, int32_t max_rows, int32_t tokens, int32_t N, int32_t K, const int32_t* offsets,
                  const int32_t* rows, const void* q, const float* s, const void* w, const float* sw, const void* bias,
                  int32_t gated, void* y, vq_dtype y_dtype, void* stream, bool check_only = false) {
  if (experts < 1 || experts > kMaxExperts || max_rows < 0 || max_rows >= kMaxPairs || tokens < 0 || N < 0 ||
      N > INT32_MAX / 2 || !valid_k(K))
    return VQ_ERR_SHAPE;
  if (!valid_dtype(y_dtype) || (gated != 0 && gated != 1)) return VQ_ERR_UNSUPPORTED;
  if (max_rows == 0 || N == 0) return VQ_OK;
  if (tokens < (rows ? 1 : max_rows)) return VQ_ERR_SHAPE;
  if (!offsets || !q || !s || !w || !sw || !y) return VQ_ERR_NULL;
  if (!aligned(offsets, 4) || misaligned(rows, 4) || !aligned(q, 16) || !aligned(w, 16) || !aligned(s, 4) ||
      !aligned(sw, 4) || misaligned(bias, 2) || !aligned(y, size_of(y_dtype)))
    return VQ_ERR_ALIGN;
  Q8Args a;
  std::memset(&a, 0, sizeof a);
  a.m = max_rows;
  a.tokens = tokens;
  a.n = N;
  a.k = K;
  a.q = (const uint8_t*)q;
  a.s = s;
  a.w = (const uint8_t*)w;
  a.sw = sw;
  a.bias = (const uint16_t*)bias;
  a.y = y;
  a.y_dtype = y_dtype;
  a.experts = experts;
  a.offsets = offsets;
  a.rows = rows;
  a.gated = gated;
  a.splits = 1;
  return launch_q8(a, stream, check_only);
}

}  // namespace
}  // namespace vqi

using namespace vqi;

extern "C" {

int64_t vq_q8_row_bytes(int32_t k) { return k < 1 ? 0 : q8_row_bytes(k); }

vq_status vq_q8_quantize(int32_t rows, int32_t k, const void* x, vq_dtype x_dtype, int64_t ldx, void* q, float* s,
                         void* stream) {
  if (rows < 0 || !valid_k(k) || ldx < k) return VQ_ERR_SHAPE;
  if (!valid_dtype(x_dtype)) return VQ_ERR_UNSUPPORTED;
  if (rows == 0) return VQ_OK;
  if (!x || !q || !s) return VQ_ERR_NULL;
  if (!aligned(x, size_of(x_dtype)) || !aligned(q, 16) || !aligned(s, 4)) return VQ_ERR_ALIGN;
  return quantize(rows, k, x, x_dtype, ldx, (uint8_t*)q, s, stream);
}

vq_status vq_q8_gemm_workspace_bytes(int32_t M, int32_t N, int32_t K, size_t* nbytes) {
  if (!nbytes) return VQ_ERR_NULL;
  if (M < 0 || N < 0 || !valid_k(K)) return VQ_ERR_SHAPE;
  int32_t splits;
  *nbytes = part_bytes(M, N, K, &splits);
  return VQ_OK;
}

vq_status vq_q8_gemm(int32_t M, int32_t N, int32_t K, const void* q, const float* s, const void* w, const float* sw,
                     const void* bias, void* y, vq_dtype y_dtype, void* workspace, size_t workspace_bytes,
                     void* stream) {
  if (M < 0 || N < 0 || !valid_k(K)) return VQ_ERR_SHAPE;
  if (!valid_dtype(y_dtype)) return VQ_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return VQ_OK;
  if (!q || !s || !w || !sw || !y) return VQ_ERR_NULL;
  if (!aligned(q, 16) || !aligned(w, 16) || !aligned(s, 4) || !aligned(sw, 4) || misaligned(bias, 2) ||
      !aligned(y, size_of(y_dtype)))
    return VQ_ERR_ALIGN;
  Q8Args a;
  std::memset(&a, 0, sizeof a);
  a.m = a.tokens = M;
  a.n = N;
  a.k = K;
  a.q = (const uint8_t*)q;
  a.s = s;
  a.w = (const uint8_t*)w;
  a.sw = sw;
  a.bias = (const uint16_t*)bias;
  a.y = y;
  a.y_dtype = y_dtype;
  const size_t need = part_bytes(M, N, K, &a.splits);
  if (workspace && need > 0) {
    if (workspace_bytes < need) return VQ_ERR_BUFFER_SIZE;
    if (!aligned(workspace, 256)) return VQ_ERR_ALIGN;
    a.part = (int32_t*)workspace;
  } else {
    a.splits = 1;
  }
  return launch_q8(a, stream);
}

vq_status vq_q8_linear_workspace_bytes(int32_t M, int32_t N, int32_t K, size_t* nbytes) {
  if (!nbytes) return VQ_ERR_NULL;
  if (M < 0 || N < 0 || !valid_k(K)) return VQ_ERR_SHAPE;
  *nbytes = linear_ws(M, N, K, nullptr).bytes;
  return VQ_OK;
}

vq_status vq_q8_linear(int32_t M, int32_t N, int32_t K, const void* x, vq_dtype x_dtype, int64_t ldx, const void* w,
                       const float* sw, const void* bias, void* y, vq_dtype y_dtype, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || !valid_k(K) || ldx < K) return VQ_ERR_SHAPE;
  if (!valid_dtype(x_dtype) || !valid_dtype(y_dtype)) return VQ_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return VQ_OK;
  const bool one = M == 1 && K <= VQ_Q8_ONE_MAX_K;  // the kernel cuts the token itself
  if (!x || !w || !sw || !y || (!workspace && !one)) return VQ_ERR_NULL;
  if (!aligned(x, size_of(x_dtype)) || !aligned(w, 16) || !aligned(sw, 4) || misaligned(bias, 2) ||
      !aligned(y, size_of(y_dtype)) || misaligned(workspace, 256))
    return VQ_ERR_ALIGN;
  const LinearWs ws = linear_ws(M, N, K, workspace);
  if (workspace && workspace_bytes < ws.bytes) return VQ_ERR_BUFFER_SIZE;
  if (one) {
    OneArgs a;
    std::memset(&a, 0, sizeof a);
    a.n = N;
    a.k = K;
    a.slots = 1;
    a.x = x;
    a.x_dtype = x_dtype;
    a.w = (const uint8_t*)w;
    a.sw = sw;
    a.bias = (const uint16_t*)bias;
    a.y = y;
    a.y_dtype = y_dtype;
    return launch_q8_one(a, stream);
  }
  const vq_status st = quantize(M, K, x, x_dtype, ldx, ws.q, ws.s, stream);
  if (st != VQ_OK) return st;
  return vq_q8_gemm(M, N, K, ws.q, ws.s, w, sw, bias, y, y_dtype, ws.splits > 1 ? ws.part : nullptr,
                    ws.splits > 1 ? workspace_bytes : 0, stream);
}

vq_status vq_expert_plan(int32_t tokens, int32_t top, int32_t experts, const int32_t* ids, int32_t* offsets,
                         int32_t* rows, int32_t* pos, void* stream) {
  const vq_status st = check_routing(tokens, top, experts);
  if (st != VQ_OK) return st;
  if (!offsets || (tokens > 0 && (!ids || !rows || !pos))) return VQ_ERR_NULL;
  if (misaligned(ids, 4) || !aligned(offsets, 4) || misaligned(rows, 4) || misaligned(pos, 4)) return VQ_ERR_ALIGN;
  return launch_expert_plan(tokens, top, experts, ids, offsets, rows, pos, stream);
}

vq_status vq_q8_gemm_grouped(int32_t experts, int32_t max_rows, int32_t tokens, int32_t N, int32_t K,
                             const int32_t* offsets, const int32_t* rows, const void* q, const float* s, const void* w,
                             const float* sw, const void* bias, int32_t gated, void* y, vq_dtype y_dtype,
                             void* stream) {
  return grouped(experts, max_rows, tokens, N, K, offsets, rows, q, s, w, sw, bias, gated, y, y_dtype, stream);
}

vq_status vq_expert_combine(int32_t tokens, int32_t top, int32_t N, int32_t max_rows, const float* z,
                            const int32_t* pos, const float* p, void* y, vq_dtype y_dtype, void* stream) {
  if (tokens < 0 || top < 1 || (int64_t)tokens * top >= kMaxPairs || N < 0 || max_rows < 0) return VQ_ERR_SHAPE;
  if (!valid_dtype(y_dtype)) return VQ_ERR_UNSUPPORTED;
  if (tokens == 0 || N == 0) return VQ_OK;
  if ((max_rows > 0 && !z) || !pos || !p || !y) return VQ_ERR_NULL;
  if (misaligned(z, 4) || !aligned(pos, 4) || !aligned(p, 4) || !aligned(y, size_of(y_dtype))) return VQ_ERR_ALIGN;
  return launch_expert_combine(tokens, top, N, max_rows, z, pos, p, y, y_dtype, stream);
}

vq_status vq_q8_experts_workspace_bytes(int32_t tokens, int32_t top, int32_t experts, int32_t D, int32_t I,
                                        size_t* nbytes) {
  if (!nbytes) return VQ_ERR_NULL;
  const vq_status st = check_routing(tokens, top, experts);
  if (st != VQ_OK) return st;
  if (!valid_k(D) || !valid_k(I)) return VQ_ERR_SHAPE;
  *nbytes = experts_ws(tokens, top, experts, D, I, nullptr).bytes;
  return VQ_OK;
}

vq_status vq_q8_experts(int32_t tokens, int32_t top, int32_t experts, int32_t D, int32_t I, const void* x,
                        vq_dtype x_dtype, int64_t ldx, const int32_t* ids, const float* p, const void* w_in,
                        const float* s_in, const void* w_out, const float* s_out, void* y, vq_dtype y_dtype,
                        void* workspace, size_t workspace_bytes, void* stream) {
  vq_status st = check_routing(tokens, top, experts);
  if (st != VQ_OK) return st;
  if (!valid_k(D) || !valid_k(I) || ldx < D) return VQ_ERR_SHAPE;
  if (!valid_dtype(x_dtype) || !valid_dtype(y_dtype)) return VQ_ERR_UNSUPPORTED;
  if (tokens == 0) return VQ_OK;
  if (!x || !ids || !p || !w_in || !s_in || !w_out || !s_out || !y || !workspace) return VQ_ERR_NULL;
  if (!aligned(x, size_of(x_dtype)) || !aligned(ids, 4) || !aligned(p, 4) || !aligned(w_in, 16) ||
      !aligned(w_out, 16) || !aligned(s_in, 4) || !aligned(s_out, 4) || !aligned(y, size_of(y_dtype)) ||
      !aligned(workspace, 256))
    return VQ_ERR_ALIGN;
  const ExpertsWs ws = experts_ws(tokens, top, experts, D, I, workspace);
  if (workspace_bytes < ws.bytes) return VQ_ERR_BUFFER_SIZE;
  const int32_t pairs = tokens * top;
  if (tokens == 1 && top <= kQ8OneSlots) {  // no routing to sort: two launches, where the hidden rows fit LDS together
    OneArgs in, out;
    std::memset(&in, 0, sizeof in);
    in.slots = top;
    in.experts = experts;
    in.ids = ids;
    in.p = p;
    out = in;
    in.n = I;
    in.k = D;
    in.x = x;
    in.x_dtype = x_dtype;
    in.w = (const uint8_t*)w_in;
    in.sw = s_in;
    in.gated = 1;
    in.y = ws.h;
    in.y_dtype = VQ_F32;
    out.n = D;
    out.k = I;
    out.x = ws.h;
    out.x_dtype = VQ_F32;
    out.w = (const uint8_t*)w_out;
    out.sw = s_out;
    out.join = 1;
    out.y = y;
    out.y_dtype = y_dtype;
    if (q8_one_lds(top, D, false) <= kQ8OneLds && q8_one_lds(top, I, true) <= kQ8OneLds) {
      if ((st = launch_q8_one(in, stream)) != VQ_OK) return st;
      return launch_q8_one(out, stream);
    }
  }
  auto run = [&](bool check_only) {
    if (!check_only &&
        (st = launch_expert_plan(tokens, top, experts, ids, ws.offsets, ws.rows, ws.pos, stream)) != VQ_OK)
      return st;
    if ((st = quantize(tokens, D, x, x_dtype, ldx, ws.xq, ws.xs, stream, check_only)) != VQ_OK) return st;
    if ((st = grouped(experts, pairs, tokens, I, D, ws.offsets, ws.rows, ws.xq, ws.xs, w_in, s_in, nullptr, 1, ws.h,
                      VQ_F32, stream, check_only)) != VQ_OK)
      return st;
    if ((st = quantize(pairs, I, ws.h, VQ_F32, I, ws.hq, ws.hs, stream, check_only)) != VQ_OK) return st;
    if ((st = grouped(experts, pairs, pairs, D, I, ws.offsets, nullptr, ws.hq, ws.hs, w_out, s_out, nullptr, 0, ws.z,
                      VQ_F32, stream, check_only)) != VQ_OK)
      return st;
    return launch_expert_combine(tokens, top, D, pairs, ws.z, ws.pos, p, y, y_dtype, stream, check_only);
  };
  if ((st = run(true)) != VQ_OK) return st;
  return run(false);
}

vq_status vq_block_norm(const vq_norm_desc* desc, const void* z, const void* h, const void* post_w, const void* post_b,
                        const void* pre_w, const void* pre_b, const void* gate, void* r, void* x, void* q, float* s,
                        void* stream) {
  if (!desc) return VQ_ERR_NULL;
  const vq_norm_desc& d = *desc;
  if (d.rows < 0 || d.dim < 1 || d.dim > kNormMaxDim || d.ldz < d.dim || (h && d.ldh < d.dim) ||
      (gate && d.gate_rows < 1))
    return VQ_ERR_SHAPE;
  if (d.post < VQ_NORM_NONE || d.post > VQ_NORM_LAYER || d.pre < VQ_NORM_NONE || d.pre > VQ_NORM_LAYER)
    return VQ_ERR_UNSUPPORTED;
  if (!valid_dtype(d.z_dtype) || ((h || r) && !valid_dtype(d.h_dtype)) || (gate && !valid_dtype(d.gate_dtype)) ||
      (x && !valid_dtype(d.x_dtype)) || ((post_w || post_b || pre_w || pre_b) && !valid_dtype(d.w_dtype)))
    return VQ_ERR_UNSUPPORTED;
  if ((d.post == VQ_NORM_NONE && (post_w || post_b)) || (d.pre == VQ_NORM_NONE && (pre_w || pre_b)))
    return VQ_ERR_UNSUPPORTED;
  if (d.rows == 0) return VQ_OK;
  if (!z || (!r && !x && !q) || (q == nullptr) != (s == nullptr)) return VQ_ERR_NULL;
  if (!aligned(z, size_of(d.z_dtype)) || misaligned(h, size_of(d.h_dtype)) || misaligned(r, size_of(d.h_dtype)) ||
      misaligned(gate, size_of(d.gate_dtype)) || misaligned(x, size_of(d.x_dtype)) ||
      misaligned(post_w, size_of(d.w_dtype)) || misaligned(post_b, size_of(d.w_dtype)) ||
      misaligned(pre_w, size_of(d.w_dtype)) || misaligned(pre_b, size_of(d.w_dtype)) || misaligned(q, 16) ||
      misaligned(s, 4))
    return VQ_ERR_ALIGN;
  NormArgs a;
  std::memset(&a, 0, sizeof a);
  a.rows = d.rows;
  a.dim = d.dim;
  a.z = z;
  a.z_dtype = d.z_dtype;
  a.ldz = d.ldz;
  a.h = h;
  a.h_dtype = d.h_dtype;
  a.ldh = d.ldh;
  a.post = d.post;
  a.pre = d.pre;
  a.post_w = post_w;
  a.post_b = post_b;
  a.pre_w = pre_w;
  a.pre_b = pre_b;
  a.w_dtype = d.w_dtype;
  a.gate = gate;
  a.gate_dtype = d.gate_dtype;
  a.gate_rows = gate ? d.gate_rows : 1;
  a.eps = d.eps;
  a.w_offset = d.w_offset;
  a.res_scale = d.res_scale;
  a.gate_scale = d.gate_scale;
  a.combine = h || d.gate_scale != 1.0f;
  a.r = r;
  a.x = x;
  a.x_dtype = d.x_dtype;
  a.q = (uint8_t*)q;
  a.s = s;
  return launch_norm(a, stream);
}

}  // extern "C"
