// Host side of vq_rotate_heads: argument checks.
#include <cstring>

#include "vq_host_checks.h"
#include "vq_internal.h"

using namespace vqi;

namespace {

// Strides of one tensor: no negative ones (a view whose pointer is not its lowest address).
bool strides_ok(const int64_t* s) { return s[0] >= 0 && s[1] >= 0 && s[2] >= 0; }

// Outputs: rows of different heads, tokens and batches apart.
bool apart(const int64_t* s, int32_t batch, int32_t tokens, int32_t heads, int32_t dim) {
  return (batch <= 1 || s[0] >= dim) && (tokens <= 1 || s[1] >= dim) && (heads <= 1 || s[2] >= dim);
}

}  // namespace

extern "C" vq_status vq_rotate_heads(const vq_heads_desc* desc, const void* q, const void* k, const void* positions,
                                     const double* freqs, const void* q_w, const void* q_b, const void* k_w,
                                     const void* k_b, void* q_out, void* k_out, void* stream) {
  if (!desc) return VQ_ERR_NULL;
  const vq_heads_desc& d = *desc;
  if (d.batch < 0 || d.tokens < 0 || d.q_heads < 0 || d.k_heads < 0 || d.q_heads > VQ_HEADS_MAX || d.k_heads > VQ_HEADS_MAX ||
      d.dim < 1 || d.dim > VQ_HEADS_MAX_DIM || d.rot < 0 || d.rot % 2 != 0 || d.start < 0 || d.rot > d.dim ||
      d.start > d.dim - d.rot || d.position_stride < 0)
    return VQ_ERR_SHAPE;
  if (d.norm < VQ_NORM_NONE || d.norm > VQ_NORM_LAYER || (d.interleaved != 0 && d.interleaved != 1) ||
      (d.positions_64 != 0 && d.positions_64 != 1) || !valid_dtype(d.x_dtype) || !valid_dtype(d.y_dtype) ||
      ((q_w || q_b || k_w || k_b) && (d.norm == VQ_NORM_NONE || !valid_dtype(d.w_dtype))))
    return VQ_ERR_UNSUPPORTED;
  const int64_t* strides[2][2] = {{d.q_strides, d.q_out_strides}, {d.k_strides, d.k_out_strides}};
  const int32_t heads[2] = {d.q_heads, d.k_heads};
  const void* const in[2] = {q, k};
  void* const out[2] = {q_out, k_out};
  const bool any = d.batch > 0 && d.tokens > 0;
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0 || !any) continue;
    if (!strides_ok(strides[i][0]) || !strides_ok(strides[i][1]) ||
        !apart(strides[i][1], d.batch, d.tokens, heads[i], d.dim))
      return VQ_ERR_SHAPE;
    if (!in[i] || !out[i]) return VQ_ERR_NULL;
    if (!aligned(in[i], size_of(d.x_dtype)) || !aligned(out[i], size_of(d.y_dtype))) return VQ_ERR_ALIGN;
    // in place: every value is written where it was read
    if (in[i] == out[i] && (d.x_dtype != d.y_dtype || std::memcmp(strides[i][0], strides[i][1], 3 * sizeof(int64_t)) != 0))
      return VQ_ERR_UNSUPPORTED;
  }
  if (!any || heads[0] + heads[1] == 0) return VQ_OK;
  if (d.rot > 0 && (!positions || !freqs)) return VQ_ERR_NULL;
  if (misaligned(positions, d.positions_64 ? 8 : 4) || misaligned(freqs, 8) || misaligned(q_w, size_of(d.w_dtype)) ||
      misaligned(q_b, size_of(d.w_dtype)) || misaligned(k_w, size_of(d.w_dtype)) || misaligned(k_b, size_of(d.w_dtype)))
    return VQ_ERR_ALIGN;
  HeadsArgs a;
  std::memset(&a, 0, sizeof a);
  a.batch = d.batch;
  a.tokens = d.tokens;
  a.dim = d.dim;
  a.rot = d.rot;
  a.start = d.start;
  a.interleaved = d.interleaved;
  a.norm = d.norm;
  for (int i = 0; i < 2; ++i) {
    a.heads[i] = heads[i];
    a.x[i] = in[i];
    a.y[i] = out[i];
    std::memcpy(a.xs[i], strides[i][0], sizeof a.xs[i]);
    std::memcpy(a.ys[i], strides[i][1], sizeof a.ys[i]);
  }
  a.x_dtype = d.x_dtype;
  a.y_dtype = d.y_dtype;
  a.w_dtype = d.w_dtype;
  a.positions = positions;
  a.pos_64 = d.positions_64;
  a.pos_stride = d.position_stride;
  a.freqs = freqs;
  a.scale = d.scale;
  a.w[0] = q_w;
  a.b[0] = q_b;
  a.w[1] = k_w;
  a.b[1] = k_b;
  a.eps = d.eps;
  a.w_offset = d.w_offset;
  return launch_heads(a, stream);
}
