// Internal declarations shared by the host and device translation units of libvq.
#pragma once

#include <cstddef>
#include <cstdint>

#include <hip/hip_runtime_api.h>

#include "vq.h"

namespace vqi {

// Number of v-wide vectors per row; the last one may be partial.
inline int64_t num_vectors(int64_t in_features, int v) { return (in_features + v - 1) / v; }

// Bytes of one row of an index stream of `bits`-bit fields: 16-byte padded.
inline int64_t row_stride(int64_t in_features, int v, int bits) {
  if (bits == 0) return 0;
  const int64_t nbits = num_vectors(in_features, v) * bits;
  return 16 * ((nbits + 127) / 128);
}

// Validates the descriptor fields (not pointers) of a row-stream layer: VQ_OK or the error
// code (any other layout is VQ_ERR_UNSUPPORTED).
vq_status check_desc(const vq_desc* d);
// The same, also accepting the slice-bucketed layout where it is defined (v = 8,
// bits1 = 16, bits2 0 or 8, IN a multiple of 8, within the 32-bit offsets of its product).
vq_status check_desc_any(const vq_desc* d);

// Slice-bucketed layout: vectors per chunk, and the bytes of its prefix table (8 * chunks
// * N + 1 uint32 bucket offsets, padded to 256 bytes) ahead of the 32-bit bucket words.
constexpr int32_t kBucketChunk = 1024;
inline int64_t bucketed_chunks(const vq_desc& d) {
  return (num_vectors(d.in_features, 8) + kBucketChunk - 1) / kBucketChunk;
}
inline size_t bucketed_header_bytes(const vq_desc& d) {
  const size_t starts = (size_t)(8 * bucketed_chunks(d)) * (size_t)d.out_features + 1;
  return (starts * 4 + 255) / 256 * 256;
}

// Packed size in bytes of a validated descriptor.
inline size_t packed_size(const vq_desc& d) {
  if (d.layout == VQ_LAYOUT_BUCKETED)
    return bucketed_header_bytes(d) + 4 * (size_t)d.out_features * (size_t)num_vectors(d.in_features, 8);
  return (size_t)d.out_features *
         (size_t)(row_stride(d.in_features, d.v, d.bits1) + row_stride(d.in_features, d.v, d.bits2));
}

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Arguments of every product launch (gemv and gemm), after validation.
struct ProductArgs {
  int32_t n, in_features, v, bits1, bits2, nv;
  int32_t s1_words, s2_words;  // row strides in 32-bit words
  const uint32_t* packed1;     // stream 1
  const uint32_t* packed2;     // stream 2 or nullptr
  const uint16_t* cb1;         // fp16 bits [K1][v]
  const uint16_t* cb2;         // fp16 bits [K2][v] or nullptr
  const uint16_t* scale;       // fp16 bits [n] or nullptr
  const uint16_t* bias;        // fp16 bits [n] or nullptr
  const uint16_t* x;           // [M][in] fp16 / bf16 bits
  void* y;                     // [M][n]
  int32_t m;
  vq_dtype x_dtype, y_dtype;
};

// Validates a product call; on success fills `a`.  `max_m` bounds M (0: unbounded).
vq_status prepare_product(const vq_desc* desc, const void* packed, const void* cb1, const void* cb2,
                          const void* scale, const void* bias, const void* x, vq_dtype x_dtype, int32_t m, void* y,
                          vq_dtype y_dtype, int32_t max_m, ProductArgs* a);

// Launchers (defined in the .hip units).  Return VQ_OK or VQ_ERR_HIP / VQ_ERR_UNSUPPORTED.
vq_status launch_dequant(const vq_desc& d, const void* packed, const void* cb1, const void* cb2, const void* scale,
                         void* w, vq_dtype w_dtype, void* stream);
vq_status launch_gemv(const ProductArgs& a, void* stream);
// The codebook-sliced GEMV (65536-entry main book, v = 8, 1 <= M <= 16) that runs with a
// caller-owned workspace: whether the shape has that path and the workspace it needs (0:
// none), whether the pointers allow it, and the launch.
bool sliced_gemv_shape_ok(const vq_desc& d, int32_t m, vq_dtype x_dtype);
size_t sliced_gemv_workspace(const vq_desc& d, int32_t m, vq_dtype x_dtype);
bool sliced_gemv_pointers_ok(const ProductArgs& a);
// rht_signs: also the randomized Hadamard transform of x (forward, blocks of rht_block(IN))
// in the x pass; then the workspace is sliced_gemv_rht_workspace(...) bytes.
vq_status launch_gemv_sliced(const ProductArgs& a, void* workspace, void* stream, const uint8_t* rht_signs = nullptr);
size_t sliced_gemv_rht_workspace(const vq_desc& d, int32_t m, vq_dtype x_dtype);
// The product over the slice-bucketed layout (M = 1): whether the descriptor's sizes fit
// its 32-bit offsets, its workspace bytes, and the launch (packed1 = the prefix table,
// packed2 = the bucket words, nv = IN / 8).
bool bucketed_gemv_shape_ok(const vq_desc& d);
size_t bucketed_gemv_workspace(const vq_desc& d);
vq_status launch_gemv_bucketed(const ProductArgs& a, void* workspace, void* stream);
// The fixed device workspace of vq_gemv_noalloc: its size, and this GPU's copy (looked up
// on the first call on each device; no allocation).
size_t static_scratch_bytes();
vq_status static_scratch(void** ptr);
vq_status launch_gemm(const ProductArgs& a, void* stream);
// The prefill product for the same 65536-entry book (vq_gemm_ws): shape test, workspace
// bytes (0: none needed), pointer test and launch.
bool gather_gemm_shape_ok(const vq_desc& d, int32_t m, vq_dtype x_dtype);
size_t gather_gemm_workspace(const vq_desc& d, int32_t m, vq_dtype x_dtype);
bool gather_gemm_pointers_ok(const ProductArgs& a);
vq_status launch_gemm_gather(const ProductArgs& a, void* workspace, void* stream, const uint8_t* rht_signs = nullptr);
size_t gather_gemm_rht_workspace(const vq_desc& d, int32_t m, vq_dtype x_dtype);
// Passes shared by the workspace products: bf16 activations rewritten as fp16 times a
// power of two per batch row (x16 [M][IN], xexp [M]); and y = 2^e * scale * (sum of
// `nparts` fp32 partial sums [nparts][M][N], in order) + bias.
vq_status launch_x_to_f16(const ProductArgs& a, uint16_t* x16, int32_t* xexp, void* stream);
// The same pass with the forward randomized Hadamard transform first (IN a multiple of 16,
// at most 32768; VQ_ERR_UNSUPPORTED otherwise).
vq_status launch_x_rht_to_f16(const ProductArgs& a, const uint8_t* signs, uint16_t* x16, int32_t* xexp, void* stream);
constexpr int32_t kFusedRhtMaxIn = 32768;
vq_status launch_partials_finalize(const ProductArgs& a, const float* part, const int32_t* xexp, int nparts,
                                   void* stream);

// Affine-lattice layers (v = 4, one 8-bit field of four 2-bit codes per vector), after
// validation.
struct SvqArgs {
  int32_t n, in_features, nv, stride;  // stride: bytes per row of the code stream
  const uint8_t* packed;
  const uint16_t* a;      // fp16 bits [4][4], A[t][u]
  const uint16_t* b;      // fp16 bits [4]
  const uint16_t* scale;  // fp16 bits [n] or nullptr
  const uint16_t* bias;   // fp16 bits [n] or nullptr
  const uint16_t* x;      // [M][in] fp16 / bf16 bits
  void* y;                // [M][n]
  int32_t m;
  vq_dtype x_dtype, y_dtype;
  int32_t x_vec4;  // IN % 4 == 0 and x 8-byte aligned: x read one 4-vector per load
};
vq_status launch_svq_gemv(const SvqArgs& p, void* stream);
vq_status launch_svq_gemm(const SvqArgs& p, void* stream);
// Randomized Hadamard transform (validated arguments; n a multiple of 16, m >= 1).
int32_t rht_block(int32_t n);
vq_status launch_rht(int32_t m, int32_t n, const void* x, vq_dtype x_dtype, const uint8_t* signs, int32_t transpose,
                     void* y, vq_dtype y_dtype, void* stream);
vq_status launch_svq_dequant(const SvqArgs& p, void* w, vq_dtype w_dtype, void* stream);
// Residual VQ encode (validated arguments: IN % v == 0, N * IN / v >= 1, workspace of at
// least assign_workspace(d) bytes, 256-byte aligned).
size_t assign_workspace(const vq_desc& d);
vq_status launch_assign(const vq_desc& d, const void* w, vq_dtype w_dtype, const uint16_t* cb1, const uint16_t* cb2,
                        uint32_t* idx1, uint32_t* idx2, void* workspace, void* stream);

// ---- 8-bit operators (vq_q8_*, vq_expert_*, vq_block_norm) ----
// `check_only`: whether the launch would be made (VQ_ERR_SHAPE: its grid is too large), for calls of several launches that
// have to refuse before the first (of the products the grouped one).

// Whether a launch of `blocks` workgroups of `threads` stays inside the 32-bit grid.
inline bool grid_ok(int64_t blocks, int64_t threads) { return blocks >= 1 && blocks * threads <= 0xFFFFFFFFll; }

// Bytes of one row of an 8-bit matrix of k columns: whole 128-byte matrix steps, the pad zero.
constexpr int64_t q8_row_bytes(int64_t k) { return (k + 127) / 128 * 128; }
// Largest K of the products and longest row of the row pass, which one workgroup holds.  (An int32 sum would hold 131071
// products of magnitude 128 * 128.)
constexpr int32_t kQ8MaxK = 65536;
constexpr int32_t kNormMaxDim = 65536;

// The row pass between two layers (validated arguments; vq_norm.hip).
struct NormArgs {
  int32_t rows, dim;
  const void* z;
  vq_dtype z_dtype;
  int64_t ldz;  // elements
  const void* h;  // residual or nullptr
  vq_dtype h_dtype;  // also r's
  int64_t ldh;
  int32_t post, pre;  // vq_norm_kind
  const void *post_w, *post_b, *pre_w, *pre_b;  // [dim] or nullptr
  vq_dtype w_dtype;
  const void* gate;  // [ceil(rows / gate_rows)][dim] or nullptr
  vq_dtype gate_dtype;
  int32_t gate_rows;
  float eps, w_offset, res_scale, gate_scale;
  int32_t combine;  // a residual or a gate_scale other than 1
  void* r;          // [rows][dim] or nullptr
  void* x;          // [rows][dim] or nullptr
  vq_dtype x_dtype;
  uint8_t* q;  // [rows][q8_row_bytes(dim)] or nullptr
  float* s;    // [rows]
};
vq_status launch_norm(const NormArgs& a, void* stream, bool check_only = false);

// An 8-bit product, dense (experts == 0) or grouped by expert (validated arguments; vq_q8.hip).
struct Q8Args {
  int32_t m;         // dense: rows; grouped: bound of the sorted rows, offsets[experts] at most
  int32_t tokens;    // rows of q and s
  int32_t n;         // outputs (with the gate: w has 2 n rows)
  int32_t k;
  const uint8_t* q;  // [tokens][q8_row_bytes(k)]
  const float* s;    // [tokens]
  const uint8_t* w;  // dense [n][..], grouped [experts][n or 2 n][..]
  const float* sw;
  const uint16_t* bias;  // fp16 [n] / [experts][n or 2 n] or nullptr
  void* y;               // [m][n]
  vq_dtype y_dtype;
  int32_t experts;
  const int32_t* offsets;  // [experts + 1]
  const int32_t* rows;     // [m] token of each sorted row, or nullptr: the row itself
  int32_t gated;           // y = silu(g) u, g and u the two halves of w's rows
  int32_t* part;           // [splits][m][n] int32 partial sums (splits > 1)
  int32_t splits;
};
// K splits that a dense product of this shape uses; its workspace is splits * m * n int32 where splits > 1.
int32_t q8_splits(int32_t m, int32_t n, int32_t k);
vq_status launch_q8(const Q8Args& a, void* stream, bool check_only = false);

// Products of one token that is cut to 8 bits inside the kernel (vq_q8.hip): dense (experts == 0), the gated products of
// its `slots` experts (y fp32 [slots][n], x one row), or their joined outputs (join: x fp32 [slots][k], y [n]).
struct OneArgs {
  int32_t n, k, slots, experts;
  const void* x;
  vq_dtype x_dtype;
  const uint8_t* w;
  const float* sw;
  const uint16_t* bias;  // dense only
  const int32_t* ids;    // [slots]
  const float* p;        // [slots]
  int32_t gated, join;
  void* y;
  vq_dtype y_dtype;
};
// Most slots of the joined form, which keeps all their rows in LDS: 7 of up to 1024 columns, 6 of 2560, 5 of 4608, 4 of
// 7936, 3 of 13312, 2 of 24064.  More slots or longer rows take the grouped products.
constexpr int32_t kQ8OneSlots = 7;
constexpr size_t kQ8OneLds = 63 * 1024;       // most dynamic LDS of a workgroup
// Dynamic LDS of the form that takes `a`: the 8-bit rows and the wavefronts' sums, two blocks of them unless joined.
constexpr size_t q8_one_lds(int64_t slots, int32_t k, bool join) {
  return (join ? slots : 1) * ((size_t)q8_row_bytes(k) + 8 * 64 * 16 * (join ? 1 : 2));
}
static_assert(q8_one_lds(1, VQ_Q8_ONE_MAX_K, false) <= kQ8OneLds && q8_one_lds(1, VQ_Q8_ONE_MAX_K + 1, false) > kQ8OneLds,
              "the longest row that a dense product of one token keeps in LDS");
static_assert(q8_one_lds(kQ8OneSlots, 1, true) <= kQ8OneLds && q8_one_lds(kQ8OneSlots + 1, 1, true) > kQ8OneLds,
              "as many slots as some row length finds room for");
vq_status launch_q8_one(const OneArgs& a, void* stream);

// Routing (vq_experts.hip): ids [tokens * top] -> offsets [experts + 1], rows and pos [tokens * top].
vq_status launch_expert_plan(int32_t tokens, int32_t top, int32_t experts, const int32_t* ids, int32_t* offsets,
                             int32_t* rows, int32_t* pos, void* stream);
vq_status launch_expert_combine(int32_t tokens, int32_t top, int32_t n, int32_t rows, const float* z,
                                const int32_t* pos, const float* p, void* y, vq_dtype y_dtype, void* stream,
                                bool check_only = false);

// ---- 8-bit floats (vq_f8_*) and the heads' pass (vq_rotate_heads) ----
// Columns and weight rows of a block with one scale.
constexpr int32_t kF8Block = 128;
constexpr int32_t kF8MaxK = 65536;
constexpr int64_t f8_blocks(int64_t n) { return (n + kF8Block - 1) / kF8Block; }

// Rows or 128-row blocks of x [rows][k] to e4m3 with block scales (validated arguments; vq_f8.hip).
struct F8QuantArgs {
  int32_t rows, k;
  const void* x;
  vq_dtype x_dtype;
  int64_t ldx;  // elements
  uint8_t* q;   // [rows][q8_row_bytes(k)]
  float* s;     // tokens: [f8_blocks(k)][rows]; weights: [f8_blocks(rows)][f8_blocks(k)]
};
vq_status launch_f8_tokens(const F8QuantArgs& a, void* stream, bool check_only = false);
vq_status launch_f8_weights(const F8QuantArgs& a, void* stream);

// How a product is computed (vq_f8.hip): the way, how often K is cut over the CUs, and whether the tokens are cut to 8 bits
// inside the kernel.
struct F8Plan {
  int32_t way, splits;
  bool cut;
};
// A product with block scales (validated arguments; vq_f8.hip).
struct F8Args {
  int32_t m, n, k;   // n outputs (with the gate: w has 2 n rows)
  F8Plan plan;
  const uint8_t* q;  // [m][q8_row_bytes(k)] e4m3, unless plan.cut
  const float* s;    // [f8_blocks(k)][m]
  const void* x;     // plan.cut: [m][k]
  vq_dtype x_dtype;
  int64_t ldx;
  const uint8_t* w;      // [n or 2 n][q8_row_bytes(k)] e4m3
  const float* sw;       // [f8_blocks(n), twice with the gate][f8_blocks(k)]
  const uint16_t* bias;  // fp16 [n or 2 n] or nullptr
  int32_t gated;         // y = silu(g) u, g and u the two halves of w's rows
  int32_t wide;          // the products' operands go to fp16, for sums that are exact to fp32 (fp32 and 8-bit outputs)
  void* y;               // [m][n], or nullptr: yq and ys take the outputs in 8 bits
  vq_dtype y_dtype;
  uint8_t* yq;  // [m][q8_row_bytes(n)]
  float* ys;    // [f8_blocks(n)][m]
  float* part;  // [plan.splits][m][n] fp32 partial sums (splits > 1)
};
// The plan of a product of m >= 1 rows and n >= 1 outputs; may_cut: the tokens come as they are, and a plan that does not cut
// them inside pays for the launch that does.
F8Plan f8_plan(int32_t m, int32_t n, int32_t k, bool gated, bool wide, bool may_cut);
// A gated product (wide) whose outputs are to be cut to 8 bits, by `plan` as it is or, true, by one that writes them so (yq, ys).
bool f8_big_plan(int32_t m, int32_t n, int32_t k, F8Plan& plan);
vq_status launch_f8(const F8Args& a, void* stream, bool check_only = false);

// Norms and rotation of heads (validated arguments; vq_heads.hip).
struct HeadsArgs {
  int32_t batch, tokens, heads[2], dim, rot, start, interleaved, norm;
  const void* x[2];  // queries and keys: [batch][tokens][heads][dim]
  void* y[2];
  int64_t xs[2][3], ys[2][3];  // strides of batch, tokens and heads in elements
  vq_dtype x_dtype, y_dtype, w_dtype;
  const void* positions;
  int32_t pos_64;      // int64 positions, else int32
  int64_t pos_stride;  // of batch, in elements; 0: the same for all
  const double* freqs;  // [rot / 2] turns per position
  float scale;          // on the rotated values
  const void *w[2], *b[2];  // [dim] or nullptr
  float eps, w_offset;
  int32_t streams;  // set by launch_heads: outputs go past the caches
};
vq_status launch_heads(const HeadsArgs& a, void* stream);

}  // namespace vqi
