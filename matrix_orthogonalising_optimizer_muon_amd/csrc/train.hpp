// Internal interfaces between the front end of the training operators (train_api.cpp) and
// their kernels (ffn.hip, losses.hip).
#pragma once

#include "internal.hpp"

namespace muon {

// Gated feed-forward block (ffn.hip): one product kernel, out(m, n) = sum_k A(m, k) B(n, k).
constexpr int kActSilu = 0, kActGeluTanh = 1;
enum FfnEpi : int { FFN_STORE = 0, FFN_GATE = 1, FFN_DGATE = 2 };
enum FfnStage : int {
  FFN_STAGE_GATE = 0,   // h = act(x Wg^T) (x Wu^T); x, Wg, Wu K-contiguous
  FFN_STAGE_DOWN = 1,   // y = h Wd^T; both K-contiguous
  FFN_STAGE_DGATE = 2,  // dh = dy Wd, then dg, du, h; Wd K-strided
  FFN_STAGE_DX = 3,     // dx = [dg du] [Wg; Wu]; weights K-strided, two K segments
  FFN_STAGE_DW = 4,     // A^T B over the tokens; both K-strided
};
enum FfnTile : int {
  FFN_TILE_32 = 0,      // 32 x 32, four k-groups of one wave
  FFN_TILE_64 = 1,      // 64 x 64, two k-groups of 4 waves
  FFN_TILE_64x128 = 2,  // 4 waves
  FFN_TILE_128 = 3,     // 128 x 128, 4 waves
  FFN_TILE_128x256 = 4, // 8 waves; not fp32
  FFN_TILE_256 = 5,     // 256 x 256, 8 waves; not fp32
  FFN_TILE_COUNT = 6
};
// One of up to three products that share a launch (FFN_STAGE_DW: gate, up and down).
struct FfnProblem {
  const void* A; const void* B; void* C;
  int64_t lda, ldb, ldc;
  int64_t part0;          // its partial products' offset in a split's, in elements
  int32_t M, N;
  int32_t tiles_m, tiles_n;
};
struct FfnGemm {
  FfnProblem problem[3];  // FFN_STAGE_DW: A, B, C, their strides, M, N and tiles come from here
  int32_t problems;       // 0: the fields below
  const void* A;
  const void* B[2];       // operand; B[1]: Wu (FFN_GATE), or a second K segment (K-strided B)
  int64_t lda, ldb, ldb1; // row strides in elements (ldb1: of Wu in FFN_GATE); rows 16-byte aligned
  int32_t M, N;           // output rows and columns (FFN_GATE: columns of one of g, u)
  int32_t K;              // valid k: of a K-contiguous row, or rows of a K-strided operand (of each segment)
  int32_t KA;             // valid k of A's rows when A is K-contiguous (K, or its zero-padded size)
  int32_t tail;           // K mod BK of the last slice's K-contiguous operands, 0: whole
  int32_t slices0;        // slices of K segment 0
  int32_t slices;         // slices of all segments
  int32_t slices_per_split, splits;
  int32_t tiles_m, tiles_n, tiles;  // tiles: of all problems
  void* C[3];             // FFN_STORE: the output; FFN_GATE: h; FFN_DGATE: dg, du, h
  int64_t ldc;            // row stride of C (FFN_DGATE: of dg and du)
  int64_t Np;             // row stride of h, g and u
  float* gu;              // saved g and u, 32 x 8 blocks (FFN_GATE: null: not saved)
  float* part;            // fp32 partial products by split, then problem, rows of N rounded up to 8; null: one split
  int64_t part_split;     // elements of a split's
  int32_t act;
  int32_t c_bf16, accumulate;
};
hipError_t launch_ffn(FfnStage stage, bool f32, int tile, const FfnGemm& p, hipStream_t st);
// Matrices to copy into 16-byte aligned rows.
struct FfnCopies {
  static constexpr int kMost = 5;
  const void* src[kMost]; void* dst[kMost];
  int64_t lds[kMost], ldd[kMost], rows[kMost], block0[kMost];
  int32_t cols[kMost];
  int32_t n;
};
hipError_t launch_ffn_align(FfnCopies& c, bool f32, hipStream_t st);
hipError_t launch_ffn_zero(void* out, int64_t ld, int64_t rows, int64_t cols, bool bf16, hipStream_t st);

// Losses over vocabulary logits (losses.hip): one workgroup per row.
enum LossKind : int { LOSS_POLICY = 0, LOSS_DISTILL = 1 };
constexpr int kMaxTop = 1024;  // kept teacher entries per row
struct LossParams {
  const void* logits; int64_t ld;
  void* dlogits; int64_t ld_d;      // null: no gradient
  int64_t rows;
  int32_t vocab;
  float temperature, inv_temperature;
  const float* weights;             // null: 1
  const float* grad_rows;           // null: 1
  float* loss;                      // null: not written
  float* lse;                       // written, or read with lse_given; may be null otherwise
  int32_t lse_given, lse_pairs;     // pairs: [rows][2], the largest logit and the sum
  // policy
  const int64_t* targets;
  const float* old_logp; const float* advantages; const float* ref_logp;
  float clip_low, clip_high, kl_coef;
  float* logp;
  // distill
  const void* top_logits; int64_t ld_top;
  const void* ids; int64_t ld_ids;
  const float* top_lse;             // null: normalised over the kept entries
  int32_t top, top_bf16, ids64;
  // few rows: each in `splits` parts (at most 64) of `part` 16-byte vectors
  int32_t splits, part;
  float* stats;                     // [rows][splits] running maximum and sum
  float* own;                       // [rows] target logit, or [rows][top] kept entries' logits
};
hipError_t launch_loss(int loss, bool bf16, const LossParams& p, hipStream_t st);

}  // namespace muon
