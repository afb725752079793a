// Internal interfaces between the front end of a layer's other operators (layer_api.cpp) and
// their kernels: linear attention with decay (mixer.hip), tokens sorted by expert and back
// (experts.hip), dropout (dropout.hip).
#pragma once

#include "internal.hpp"

namespace muon {

// ---- linear attention (mixer.hip) ----
// One walk over tokens:  out_r = p_scale sum_{s <= r} e^{g (r - s)} (a_r . b_s) c_s
//                                + o_scale e^{g (r + off)} a_r Z_0,
//   Z_n = e^{g n} Z_0 + u_scale sum_s e^{g (n - off - s)} b_s^T c_s   (dim x dim_v, fp32),
// where r counts a sequence's tokens from its first (off 1) or, reversed, from its last (off 0).
// Forward: a, b, c = q, k, v. Gradients: dq from (do, v, k), dk from (v, do, q) reversed, dv
// from (k, q, do) reversed.
constexpr int kMixChunk = 64;
struct MixArray {
  const void* p;
  int64_t sb, st, sh;     // batch, token and head strides in elements
  int32_t group;          // heads that share one of its own
};
struct MixRole {
  MixArray a, b, c;
  void* out;              // contiguous batch x tokens x heads x dim_v (walks with outputs)
  int32_t out_f32;        // fp32 whatever the operands' type (one of several partial sums)
  int32_t dim, dim_v;
  int32_t reversed;
  float p_scale, o_scale, u_scale;
  const float* z_in;      // null: zeros. One dim x dim_v array per (batch, head) and segment
  int64_t z_row, z_col;   // its strides
  float* z_out;           // null: not wanted. Contiguous rows
  int32_t first;          // index of its first workgroup among a (batch, head, segment)'s
};
struct MixParams {
  MixRole role[3];
  int32_t roles;
  int32_t per;            // workgroups of a (batch, head, segment): all roles' slices
  const float* log_decay;
  const int32_t* lengths; // null: tokens
  int32_t batch, heads, tokens;
  int32_t segments, segment;  // number, tokens of one (a multiple of the chunk)
  int32_t direct;             // every operand's rows are 16-byte aligned, apart, and a chunk spans at most 2^29 bytes
  int32_t walked;             // segments walked: all, or without the last one
  int32_t z_in_per_segment;   // z_in has an array for each segment, else one for the first
  int32_t z_out_per_segment;  // z_out too (a segment's own sum), else one from the last token's segment
};
struct MixTile { int dim, dim_v; };   // padded dim, dim_v slice of a workgroup
// out: with outputs (the main walk) or the segments' states alone
hipError_t launch_mix(bool f32, MixTile t, bool out, const MixParams& p, int64_t groups, hipStream_t st);
// Segment sums to the states before each segment, in place.
struct MixScan {
  struct One { const float* z0; float* z; int32_t n; } one[2];   // n: elements of a state
  int32_t count;
  const float* log_decay;
  const int32_t* lengths;
  int32_t batch, heads, tokens, segments, segment;
};
hipError_t launch_mix_scan(const MixScan& p, hipStream_t st);
// Sums of the fp32 partial gradients of heads that share one: out[row][kv][d] = sum_i part[row][kv group + i][d].
struct MixShare {
  struct One { const float* part; void* out; int32_t dim; } one[2];
  int32_t count, kv_heads, group, bf16;
  int64_t rows;
};
hipError_t launch_mix_share(const MixShare& p, hipStream_t st);
struct MixStep {
  const void *q, *k, *v;
  int64_t q_sb, q_sh, k_sb, k_sh, v_sb, v_sh;
  const float* log_decay;
  const float* z_in; float* z_out;
  void* out;
  float scale;
  int32_t batch, heads, group, dim, dim_v, lanes;  // lanes: threads across a workgroup's columns
};
hipError_t launch_mix_step(bool f32, const MixStep& p, hipStream_t st);

// ---- tokens by expert (experts.hip) ----
constexpr int kMaxExperts = 1024;
struct PlanParams {
  const void* ids; int32_t ids64;
  int64_t n;                             // choices: tokens x top
  int32_t experts, blocks;
  int32_t *order, *slots, *offsets;
  int32_t* counts;                       // blocks x (experts + 1): a block's choices by expert
};
hipError_t launch_expert_plan(const PlanParams& p, hipStream_t st);
struct RowsParams {
  const int32_t *slots, *offsets;
  const float* weights;                  // null: 1
  const void *in, *in2;
  void *out; float* dw;
  int64_t ld_in, ld_in2, ld_out;
  int64_t tokens;
  int32_t top, experts, dim;
  int32_t once;                          // the sorted rows are more than the caches keep: read past them
};
enum RowsOp : int { ROWS_DISPATCH = 0, ROWS_COMBINE = 1, ROWS_COMBINE_GRAD = 2 };
hipError_t launch_expert_rows(RowsOp op, bool f32, const RowsParams& p, hipStream_t st);

// ---- dropout (dropout.hip) ----
struct DropParams {
  const void *x, *residual;
  void* out;
  int64_t ld_x, ld_r, ld_o;
  int64_t rows, cols;
  uint64_t seed, offset;
  const uint64_t* counter;               // device: seed and offset; null: the two above
  uint32_t threshold;                    // of 65536: a 16-bit number below it drops its element
  float factor;
};
hipError_t launch_dropout(bool f32, const DropParams& p, hipStream_t st);

}  // namespace muon
