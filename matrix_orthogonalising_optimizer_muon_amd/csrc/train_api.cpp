// C-ABI front end of the training operators beside the updates: argument validation, the
// workspace plan and the launches of the gated feed-forward block (forward, backward) and
// of the losses over vocabulary logits. The calls only read the context, so several
// threads may make them on one context at once.
#include "../../include/muon.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "frontend.hpp"
#include "train.hpp"

namespace muon {
namespace {

constexpr int64_t kMaxTokens = int64_t{1} << 24;
constexpr int64_t kMaxDim = int64_t{1} << 20;
constexpr int64_t kMaxLd = int64_t{1} << 21;   // a tile's 256 rows stay within 32-bit byte offsets
constexpr size_t kAlign = 256;

inline int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline int64_t cdiv(int64_t x, int64_t a) { return (x + a - 1) / a; }
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline bool dtype_ok(int d) { return d == MUON_F32 || d == MUON_BF16; }
inline int64_t size_of(int d) { return d == MUON_F32 ? 4 : 2; }
inline bool aligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// ---- gated feed-forward block ----

int validate(const muon_ffn* f, bool need_pointers) {
  if (!f || !dtype_ok(f->dtype)) return MUON_ERR_ARG;
  if (f->activation != MUON_ACT_SILU && f->activation != MUON_ACT_GELU_TANH) return MUON_ERR_ARG;
  if (f->tokens < 0 || f->tokens > kMaxTokens) return MUON_ERR_ARG;
  if (f->dim < 1 || f->dim > kMaxDim || f->hidden < 1 || f->hidden > kMaxDim) return MUON_ERR_ARG;
  auto ld_ok = [](int64_t ld, int64_t cols) { return ld >= cols && ld <= kMaxLd; };
  if (!ld_ok(f->ld_x, f->dim) || !ld_ok(f->ld_gate, f->dim) || !ld_ok(f->ld_up, f->dim) ||
      !ld_ok(f->ld_down, f->hidden))
    return MUON_ERR_ARG;
  const int64_t es = size_of(f->dtype);
  if (!aligned(f->x, es) || !aligned(f->w_gate, es) || !aligned(f->w_up, es) || !aligned(f->w_down, es))
    return MUON_ERR_ARG;
  if (need_pointers && ((f->tokens > 0 && !f->x) || !f->w_gate || !f->w_up || !f->w_down)) return MUON_ERR_ARG;
  return MUON_OK;
}

int validate(const muon_ffn* f, const muon_ffn_grads* g, bool need_pointers) {
  if (!dtype_ok(g->g_dtype) || (g->accumulate != 0 && g->accumulate != 1)) return MUON_ERR_ARG;
  auto ld_ok = [](int64_t ld, int64_t cols) { return ld >= cols && ld <= kMaxLd; };
  if (!ld_ok(g->ld_dy, f->dim) || (g->dx && !ld_ok(g->ld_dx, f->dim)) || (g->g_gate && !ld_ok(g->ld_g_gate, f->dim)) ||
      (g->g_up && !ld_ok(g->ld_g_up, f->dim)) || (g->g_down && !ld_ok(g->ld_g_down, f->hidden)))
    return MUON_ERR_ARG;
  const int64_t es = size_of(f->dtype), gs = size_of(g->g_dtype);
  if (!aligned(g->dy, es) || !aligned(g->dx, es) || !aligned(g->g_gate, gs) || !aligned(g->g_up, gs) ||
      !aligned(g->g_down, gs) || !aligned(g->saved, 16))
    return MUON_ERR_ARG;
  if (need_pointers && f->tokens > 0 && (!g->dy || !g->saved)) return MUON_ERR_ARG;
  return MUON_OK;
}

// Workspace, in order of use. Offsets are filled whether or not memory is there.
struct Arena {
  size_t at = 0;
  size_t take(size_t bytes) {
    const size_t here = at;
    at = align_up(at + bytes);
    return here;
  }
};

// An operand as the product kernel reads it: the caller's array where its rows are 16-byte
// aligned, else a copy in the workspace whose rows are.
struct Operand {
  const void* p = nullptr;
  int64_t ld = 0;
  bool copied = false;
  size_t off = 0;
  const void* src = nullptr;
  int64_t src_ld = 0, rows = 0, cols = 0;
};

Operand operand(const void* p, int64_t ld, int64_t rows, int64_t cols, int64_t es, Arena& a, bool copy = false) {
  Operand o;
  o.src = p; o.src_ld = ld; o.rows = rows; o.cols = cols;
  o.p = p; o.ld = ld;
  if (copy || !aligned(p, 16) || ld * es % 16 != 0) {
    o.copied = true;
    o.ld = round_up(cols, 16 / es);
    o.off = a.take(static_cast<size_t>(rows * o.ld * es));
  }
  return o;
}

// Tile and K split of one product: the cheapest by a model of measured parts. A workgroup
// takes kSliceUs per slice of K (128 bytes a row), by operand layout, tile and how many
// share a CU; the launch is as many rounds of resident workgroups as it takes; each round
// adds the fill of the ring and an epilogue in proportion to the tile (larger where it
// reads g and u); a split of K (plain outputs) adds the traffic of the fp32 partials and
// the joining launch. Measured over 845 launches of 15 problems, 64 to 16384 tokens; on
// these the model's choice takes 1.6% more than the best of all tiles and splits (mean),
// against 20 to 110% for the largest tile that fills the GPU (2048 tokens, 2048 x 8192: dx
// 292 us with 128 x 128 tiles, 130 us with 256 x 256 and four splits).
struct Shape {
  int tile = FFN_TILE_128, splits = 1;
  int64_t slices = 0, per_split = 0;
};
constexpr int kTileM[FFN_TILE_COUNT] = {32, 64, 64, 128, 128, 256}, kTileN[FFN_TILE_COUNT] = {32, 64, 128, 128, 256, 256};
struct Extent {
  int64_t M, cols;  // rows; columns the tiles cover (twice the output's for the gate stage)
};

enum Layout { BOTH_CONTIGUOUS = 0, B_STRIDED = 1, BOTH_STRIDED = 2 };
// [fp32][layout][tile][two workgroups a CU, one]; the two large tiles always have one.
constexpr float kSliceUs[2][3][FFN_TILE_COUNT][2] = {
    {{{0.190f, 0.114f}, {0.406f, 0.173f}, {0.669f, 0.329f}, {0.534f, 0.534f}, {0.815f, 0.815f}, {1.375f, 1.375f}},
     {{0.244f, 0.146f}, {0.424f, 0.213f}, {0.677f, 0.376f}, {0.537f, 0.537f}, {0.815f, 0.815f}, {1.332f, 1.332f}},
     {{0.309f, 0.179f}, {0.494f, 0.305f}, {0.663f, 0.411f}, {0.575f, 0.575f}, {0.886f, 0.886f}, {1.526f, 1.526f}}},
    {{{0.353f, 0.184f}, {1.106f, 0.553f}, {2.171f, 1.106f}, {2.143f, 2.143f}, {1e9f, 1e9f}, {1e9f, 1e9f}},
     {{0.415f, 0.260f}, {1.123f, 0.628f}, {1.932f, 1.123f}, {2.031f, 2.031f}, {1e9f, 1e9f}, {1e9f, 1e9f}},
     {{0.418f, 0.292f}, {1.017f, 0.582f}, {1.918f, 1.053f}, {2.084f, 2.084f}, {1e9f, 1e9f}, {1e9f, 1e9f}}}};
constexpr double kFillUs = 2.2, kEpilogueUs = 4.0, kDgateEpilogueUs = 35.2;  // per round; epilogues per 256 x 256
constexpr double kJoinUs = 2.7, kJoinBytesPerUs = 6.2e6;
constexpr int64_t kMaxPartBytes = int64_t{1} << 28;
constexpr int64_t kMinSplitSlices = 4;

// The products of one launch (same K), dgate: their epilogue.
Shape choose(bool f32, Layout layout, std::initializer_list<Extent> outputs, int64_t slices, bool may_split, bool dgate,
             int cus) {
  static const int per_cu[FFN_TILE_COUNT] = {2, 2, 2, 1, 1, 1};
  static const int try_splits[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32};
  Shape best;
  double best_us = 1e300;
  for (int t = 0; t < FFN_TILE_COUNT; ++t) {
    if (f32 && t >= FFN_TILE_128x256) continue;
    int64_t tiles = 0, elements = 0;
    for (const Extent& o : outputs) {
      tiles += cdiv(o.M, kTileM[t]) * cdiv(o.cols, kTileN[t]);
      elements += o.M * round_up(o.cols, 8);
    }
    const double area = kTileM[t] * kTileN[t] / 65536.0;
    for (const int want : try_splits) {
      if (want > 1 && (!may_split || slices / want < kMinSplitSlices)) break;
      const int64_t per = cdiv(slices, want), splits = cdiv(slices, per);
      const int64_t part = splits > 1 ? splits * elements * 4 : 0;
      if (part > kMaxPartBytes) break;
      const int64_t wgs = tiles * splits;
      const int64_t slots = static_cast<int64_t>(cus) * per_cu[t];
      const double us = cdiv(wgs, slots) * (per * static_cast<double>(kSliceUs[f32][layout][t][wgs <= cus]) + kFillUs +
                                            area * (dgate ? kDgateEpilogueUs : kEpilogueUs)) +
                        (part ? kJoinUs + 2.0 * part / kJoinBytesPerUs : 0.0);
      if (us < best_us) {
        best_us = us;
        best.tile = t;
        best.splits = static_cast<int>(splits);
        best.slices = slices;
        best.per_split = per;
      }
    }
  }
  return best;
}

// Everything muon_ffn_forward / muon_ffn_backward launch, from the sizes and alignments.
struct FfnPlan {
  int64_t es = 2, bk = 64, Hp = 0;
  Operand x, wg, wu, wd, dy;
  size_t off_h = 0, off_dg = 0, off_part = 0, bytes = 0;
  Shape gate, down, dgate, dx, dw;
};

size_t part_bytes(const Shape& s, int64_t elements) {
  return s.splits > 1 ? static_cast<size_t>(s.splits) * elements * 4 : 0;
}

FfnPlan plan_of(const muon_ffn* f, const muon_ffn_grads* g, int cus) {
  FfnPlan p;
  const bool f32 = f->dtype == MUON_F32;
  p.es = size_of(f->dtype);
  p.bk = 128 / p.es;
  p.Hp = round_up(f->hidden, 64);
  const int64_t T = f->tokens, D = f->dim, F = f->hidden;
  if (T == 0) return p;  // nothing is launched on tiles
  Arena a;
  const size_t inter = static_cast<size_t>(T * p.Hp * p.es);
  // a backward reads x for the gradients of gate and up alone, and gate and up for dx alone
  const bool need_x = !g || g->g_gate || g->g_up, need_gate_up = !g || g->dx;
  if (need_x) p.x = operand(f->x, f->ld_x, T, D, p.es, a);
  p.wd = operand(f->w_down, f->ld_down, D, F, p.es, a);
  if (need_gate_up) {
    p.wg = operand(f->w_gate, f->ld_gate, F, D, p.es, a);
    p.wu = operand(f->w_up, f->ld_up, F, D, p.es, a);
  }
  if (g && g->dx && p.wg.ld != p.wu.ld) {
    // dx reads them as the two K segments of one operand: one row stride
    if (!p.wg.copied) p.wg = operand(f->w_gate, f->ld_gate, F, D, p.es, a, true);
    if (!p.wu.copied) p.wu = operand(f->w_up, f->ld_up, F, D, p.es, a, true);
  }
  p.off_h = a.take(inter);
  size_t part = 0;
  if (!g) {
    p.gate = choose(f32, BOTH_CONTIGUOUS, {{T, 2 * p.Hp}}, cdiv(D, p.bk), false, false, cus);  // h's padding is written too
    p.down = choose(f32, BOTH_CONTIGUOUS, {{T, D}}, cdiv(F, p.bk), true, false, cus);
    part = part_bytes(p.down, T * round_up(D, 8));
  } else {
    p.dy = operand(g->dy, g->ld_dy, T, D, p.es, a);
    p.off_dg = a.take(2 * inter);  // dg and du side by side in each row: one operand of dx
    p.dgate = choose(f32, B_STRIDED, {{T, p.Hp}}, cdiv(D, p.bk), false, true, cus);
    p.dx = choose(f32, B_STRIDED, {{T, D}}, 2 * (p.Hp / p.bk), true, false, cus);
    if (g->dx) part = part_bytes(p.dx, T * round_up(D, 8));
    // the weight gradients wanted, in one launch
    const Extent fd{g->g_gate ? F : 0, D}, fu{g->g_up ? F : 0, D}, df{g->g_down ? D : 0, F};
    p.dw = choose(f32, BOTH_STRIDED, {fd, fu, df}, cdiv(T, p.bk), true, false, cus);
    part = std::max(part, part_bytes(p.dw, (fd.M + fu.M) * round_up(D, 8) + df.M * round_up(F, 8)));
  }
  p.off_part = a.take(part);
  p.bytes = a.at;
  return p;
}

hipError_t settle(std::initializer_list<Operand*> operands, char* ws, bool f32, hipStream_t st) {
  FfnCopies c;
  c.n = 0;
  for (Operand* o : operands) {
    if (!o->copied) continue;
    o->p = ws + o->off;
    c.src[c.n] = o->src; c.lds[c.n] = o->src_ld;
    c.dst[c.n] = ws + o->off; c.ldd[c.n] = o->ld;
    c.rows[c.n] = o->rows; c.cols[c.n] = static_cast<int32_t>(o->cols);
    ++c.n;
  }
  return launch_ffn_align(c, f32, st);
}

FfnGemm product(const Shape& s, int64_t M, int64_t N, int64_t cols, int64_t K, int act) {
  FfnGemm q;
  std::memset(&q, 0, sizeof(q));
  q.M = static_cast<int32_t>(M);
  q.N = static_cast<int32_t>(N);
  q.K = q.KA = static_cast<int32_t>(K);
  q.slices0 = q.slices = static_cast<int32_t>(s.slices);
  q.slices_per_split = static_cast<int32_t>(s.per_split);
  q.splits = s.splits;
  q.tiles_m = static_cast<int32_t>(cdiv(M, kTileM[s.tile]));
  q.tiles_n = static_cast<int32_t>(cdiv(cols, kTileN[s.tile]));
  q.tiles = q.tiles_m * q.tiles_n;
  q.act = act;
  return q;
}

// A plain output: its type, and where the partial products of a K split go.
void output(FfnGemm& q, const Shape& s, char* part, int64_t part_split, bool bf16, bool accumulate) {
  q.c_bf16 = bf16;
  q.accumulate = accumulate;
  if (s.splits > 1) {
    q.part = reinterpret_cast<float*>(part);
    q.part_split = part_split;
  }
}

// One more product of a launch.
void add(FfnGemm& q, const Shape& s, const void* A, int64_t lda, const void* B, int64_t ldb, void* C, int64_t ldc,
         int64_t M, int64_t N) {
  FfnProblem& o = q.problem[q.problems];
  o.A = A; o.lda = lda;
  o.B = B; o.ldb = ldb;
  o.C = C; o.ldc = ldc;
  o.M = static_cast<int32_t>(M);
  o.N = static_cast<int32_t>(N);
  o.tiles_m = static_cast<int32_t>(cdiv(M, kTileM[s.tile]));
  o.tiles_n = static_cast<int32_t>(cdiv(N, kTileN[s.tile]));
  o.part0 = q.part_split;
  q.part_split += M * round_up(N, 8);
  q.tiles += o.tiles_m * o.tiles_n;
  ++q.problems;
}

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return MUON_OK;
  return !ws || have < need || !aligned(ws, kAlign) ? MUON_ERR_WORKSPACE : MUON_OK;
}

// ---- losses ----

// A workgroup of 256 threads a row: 2^32 threads is past what a launch takes.
constexpr int64_t kMaxRows = (int64_t{1} << 24) - 1;
constexpr int64_t kMaxLogitsLd = int64_t{1} << 36;

// Whether two row sets of one shape (strides in elements, at least cols) share an element:
// apart as address ranges, or columns side by side in rows of one stride.
bool overlap(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t rows, int64_t cols, int64_t es) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  const uintptr_t na = static_cast<uintptr_t>(((rows - 1) * lda + cols) * es);
  const uintptr_t nb = static_cast<uintptr_t>(((rows - 1) * ldb + cols) * es);
  if (pa + na <= pb || pb + nb <= pa) return false;
  if (lda != ldb) return true;
  const uintptr_t row = static_cast<uintptr_t>(lda * es), width = static_cast<uintptr_t>(cols * es);
  const uintptr_t shift = (pb > pa ? pb - pa : pa - pb) % row;
  return shift < width || shift + width > row;
}

// What the workspace's size depends on.
int validate_sizes(const muon_logits* l) {
  if (!l || !dtype_ok(l->dtype)) return MUON_ERR_ARG;
  if (l->rows < 0 || l->rows > kMaxRows || l->vocab < 1 || l->vocab > (int64_t{1} << 28)) return MUON_ERR_ARG;
  if ((l->lse_given != 0 && l->lse_given != 1) || (l->lse_pairs != 0 && l->lse_pairs != 1)) return MUON_ERR_ARG;
  return MUON_OK;
}

int validate(const muon_logits* l) {
  if (validate_sizes(l) != MUON_OK) return MUON_ERR_ARG;
  if (l->ld < l->vocab || (l->dlogits && l->ld_d < l->vocab)) return MUON_ERR_ARG;
  if (!std::isfinite(l->temperature) || !(l->temperature > 0.0f) || !std::isfinite(2.0f / l->temperature))
    return MUON_ERR_ARG;
  const int64_t es = size_of(l->dtype);
  if (!aligned(l->logits, es) || !aligned(l->dlogits, es)) return MUON_ERR_ARG;
  if (l->rows > 0 && (!l->logits || (l->lse_given && !l->lse))) return MUON_ERR_ARG;
  // row strides whose byte offsets stay within 64 bits
  if (l->ld > kMaxLogitsLd || (l->dlogits && l->ld_d > kMaxLogitsLd)) return MUON_ERR_ARG;
  // in place only as a whole: the same rows
  if (l->dlogits && l->dlogits == l->logits && l->ld_d != l->ld) return MUON_ERR_ARG;
  if (l->dlogits && l->rows > 0 && l->dlogits != l->logits &&
      overlap(l->logits, l->ld, l->dlogits, l->ld_d, l->rows, l->vocab, es))
    return MUON_ERR_ARG;
  return MUON_OK;
}

// Few long rows: one workgroup a row leaves most CUs idle, so each row is split until there
// are about as many workgroups as CUs, with at least kMinPart vectors (16 bytes) a part. It
// costs a launch, so it is for rows of kMinSplit columns or more: 16 rows of 152064 bf16
// columns take 25.8 us unsplit and 9.2 us (3.9 + 5.3) split, but 77 rows of 32003 fp32 columns
// 10.5 us unsplit and 13.8 us split. On the two sides of the border (98303 columns unsplit, 98304
// split; us, bf16 then fp32): 1 row 12.8 / 6.8, 14.6 / 6.4; 16 rows 14.6 / 7.4, 15.5 / 8.2; 64 rows
// 15.8 / 11.8, 21.2 / 17.5; 128 rows 16.7 / 20.1, 26.8 / 30.4. So the border is too high for few rows and
// the rule too wide above about 100 rows, where a row has only two parts; no border between
// 32003 and 98304 has been measured.
constexpr int kMinPart = 1024;
constexpr int64_t kMinSplit = 98304;
struct LossSplit {
  int splits = 1, part = 0;
  size_t stats = 0, bytes = 0;   // bytes of the parts' statistics; workspace in all
};
LossSplit split_of(const muon_logits* l, int own_per_row, int cus) {
  LossSplit s;
  const int64_t vectors = l->vocab * size_of(l->dtype) / 16;
  if (l->rows == 0 || 2 * l->rows > cus || l->vocab < kMinSplit || !(l->dlogits || !l->lse_given)) return s;
  const int64_t want = std::min<int64_t>({cus / l->rows, vectors / kMinPart, 64});
  if (want < 2) return s;
  s.part = static_cast<int>(cdiv(vectors, want));
  s.splits = static_cast<int>(cdiv(vectors, s.part));
  if (s.splits < 2) { s.splits = 1; return s; }
  s.stats = align_up(static_cast<size_t>(l->rows) * s.splits * 8);
  s.bytes = s.stats + align_up(static_cast<size_t>(l->rows) * own_per_row * 4);
  return s;
}
void apply(const LossSplit& s, LossParams& p, void* ws) {
  p.splits = s.splits;
  p.part = s.part;
  p.stats = static_cast<float*>(ws);
  p.own = s.splits > 1 ? reinterpret_cast<float*>(static_cast<char*>(ws) + s.stats) : nullptr;
}

LossParams params(const muon_logits* l) {
  LossParams p;
  std::memset(&p, 0, sizeof(p));
  p.logits = l->logits; p.ld = l->ld;
  p.dlogits = l->dlogits; p.ld_d = l->ld_d;
  p.rows = l->rows;
  p.vocab = static_cast<int32_t>(l->vocab);
  p.temperature = l->temperature;
  p.inv_temperature = 1.0f / l->temperature;
  p.weights = l->weights; p.grad_rows = l->grad_rows;
  p.loss = l->loss; p.lse = l->lse; p.lse_given = l->lse_given; p.lse_pairs = l->lse_pairs;
  return p;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

int muon_ffn_workspace_size(muon_ctx* ctx, const muon_ffn* f, const muon_ffn_grads* g, size_t* workspace,
                            size_t* saved) {
  try {
    if (!ctx || (!workspace && !saved)) return MUON_ERR_ARG;
    int rc = validate(f, false);
    if (rc == MUON_OK && g) rc = validate(f, g, false);
    if (rc != MUON_OK) return rc;
    const FfnPlan p = plan_of(f, g, ctx_cus(ctx));
    if (workspace) *workspace = p.bytes;
    if (saved) *saved = static_cast<size_t>(2 * round_up(f->tokens, 32) * p.Hp * 4);
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

int muon_ffn_forward(muon_ctx* ctx, const muon_ffn* f, void* y, int64_t ld_y, void* saved, void* workspace,
                     size_t workspace_bytes, void* stream) {
  try {
    if (!ctx) return MUON_ERR_ARG;
    int rc = validate(f, true);
    if (rc != MUON_OK) return rc;
    if (ld_y < f->dim || ld_y > kMaxLd || !aligned(y, size_of(f->dtype)) || !aligned(saved, 16)) return MUON_ERR_ARG;
    if (f->tokens == 0) return MUON_OK;
    if (!y) return MUON_ERR_ARG;
    FfnPlan p = plan_of(f, nullptr, ctx_cus(ctx));
    rc = check_workspace(workspace, workspace_bytes, p.bytes);
    if (rc != MUON_OK) return rc;
    if (ctx_device(ctx) < 0) return MUON_ERR_DEVICE;
    DeviceGuard dg(ctx_device(ctx));
    if (!dg.ok) return MUON_ERR_HIP;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    const bool f32 = f->dtype == MUON_F32;
    MUON_HIP(settle({&p.x, &p.wg, &p.wu, &p.wd}, ws, f32, st));
    const int64_t T = f->tokens, D = f->dim, F = f->hidden;

    FfnGemm q = product(p.gate, T, F, 2 * p.Hp, D, f->activation);
    q.A = p.x.p; q.lda = p.x.ld;
    q.B[0] = p.wg.p; q.ldb = p.wg.ld;
    q.B[1] = p.wu.p; q.ldb1 = p.wu.ld;
    q.tail = static_cast<int32_t>(D % p.bk);
    q.C[0] = ws + p.off_h;
    q.ldc = q.Np = p.Hp;
    q.gu = static_cast<float*>(saved);
    MUON_HIP(launch_ffn(FFN_STAGE_GATE, f32, p.gate.tile, q, st));

    q = product(p.down, T, D, D, F, f->activation);
    q.A = ws + p.off_h; q.lda = p.Hp;
    q.B[0] = p.wd.p; q.ldb = p.wd.ld;
    q.tail = static_cast<int32_t>(F % p.bk);
    q.C[0] = y; q.ldc = ld_y;
    output(q, p.down, ws + p.off_part, T * round_up(D, 8), !f32, false);
    MUON_HIP(launch_ffn(FFN_STAGE_DOWN, f32, p.down.tile, q, st));
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

int muon_ffn_backward(muon_ctx* ctx, const muon_ffn* f, const muon_ffn_grads* g, void* workspace,
                      size_t workspace_bytes, void* stream) {
  try {
    if (!ctx || !g) return MUON_ERR_ARG;
    int rc = validate(f, true);
    if (rc == MUON_OK) rc = validate(f, g, true);
    if (rc != MUON_OK) return rc;
    FfnPlan p = plan_of(f, g, ctx_cus(ctx));
    rc = f->tokens > 0 ? check_workspace(workspace, workspace_bytes, p.bytes) : MUON_OK;
    if (rc != MUON_OK) return rc;
    if (ctx_device(ctx) < 0) return MUON_ERR_DEVICE;
    DeviceGuard dg(ctx_device(ctx));
    if (!dg.ok) return MUON_ERR_HIP;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const bool f32 = f->dtype == MUON_F32, gb = g->g_dtype == MUON_BF16;
    const int64_t T = f->tokens, D = f->dim, F = f->hidden;
    if (T == 0) {  // no tokens: the weight gradients are zero, or stay as they are
      if (g->accumulate) return MUON_OK;
      if (g->g_gate) MUON_HIP(launch_ffn_zero(g->g_gate, g->ld_g_gate, F, D, gb, st));
      if (g->g_up) MUON_HIP(launch_ffn_zero(g->g_up, g->ld_g_up, F, D, gb, st));
      if (g->g_down) MUON_HIP(launch_ffn_zero(g->g_down, g->ld_g_down, D, F, gb, st));
      return MUON_OK;
    }
    char* ws = static_cast<char*>(workspace);
    MUON_HIP(settle({&p.x, &p.wg, &p.wu, &p.wd, &p.dy}, ws, f32, st));
    char *h = ws + p.off_h, *dgp = ws + p.off_dg, *dup = dgp + p.Hp * p.es, *part = ws + p.off_part;

    FfnGemm q = product(p.dgate, T, F, p.Hp, D, f->activation);
    q.A = p.dy.p; q.lda = p.dy.ld;
    q.B[0] = p.wd.p; q.ldb = p.wd.ld;
    q.tail = static_cast<int32_t>(D % p.bk);
    q.C[0] = dgp; q.C[1] = dup; q.C[2] = h;
    q.ldc = 2 * p.Hp;
    q.Np = p.Hp;
    q.gu = const_cast<float*>(static_cast<const float*>(g->saved));
    MUON_HIP(launch_ffn(FFN_STAGE_DGATE, f32, p.dgate.tile, q, st));

    if (g->dx) {
      q = product(p.dx, T, D, D, F, f->activation);
      q.slices0 = static_cast<int32_t>(p.Hp / p.bk);
      q.A = dgp; q.lda = 2 * p.Hp; q.KA = static_cast<int32_t>(2 * p.Hp);
      q.B[0] = p.wg.p; q.ldb = p.wg.ld;
      q.B[1] = p.wu.p;
      q.C[0] = g->dx; q.ldc = g->ld_dx;
      output(q, p.dx, part, T * round_up(D, 8), !f32, false);
      MUON_HIP(launch_ffn(FFN_STAGE_DX, f32, p.dx.tile, q, st));
    }
    if (g->g_gate || g->g_up || g->g_down) {
      q = product(p.dw, 0, 0, 0, T, f->activation);
      if (g->g_gate) add(q, p.dw, dgp, 2 * p.Hp, p.x.p, p.x.ld, g->g_gate, g->ld_g_gate, F, D);
      if (g->g_up) add(q, p.dw, dup, 2 * p.Hp, p.x.p, p.x.ld, g->g_up, g->ld_g_up, F, D);
      if (g->g_down) add(q, p.dw, p.dy.p, p.dy.ld, h, p.Hp, g->g_down, g->ld_g_down, D, F);
      output(q, p.dw, part, q.part_split, gb, g->accumulate);
      MUON_HIP(launch_ffn(FFN_STAGE_DW, f32, p.dw.tile, q, st));
    }
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

int muon_loss_workspace_size(muon_ctx* ctx, const muon_logits* l, int top, size_t* bytes) {
  try {
    if (!ctx || !bytes || validate_sizes(l) != MUON_OK || top < 0 || top > MUON_MAX_TOP) return MUON_ERR_ARG;
    *bytes = split_of(l, top > 0 ? top : 1, ctx_cus(ctx)).bytes;
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

int muon_policy_loss(muon_ctx* ctx, const muon_logits* l, const muon_policy* t, void* workspace, size_t workspace_bytes,
                     void* stream) {
  try {
    if (!ctx || !t) return MUON_ERR_ARG;
    const int rc = validate(l);
    if (rc != MUON_OK) return rc;
    if (!std::isfinite(t->clip_low) || !std::isfinite(t->clip_high) || !std::isfinite(t->kl_coef) ||
        t->clip_low < 0.0f || t->clip_high < 0.0f || t->clip_low > 1.0f)
      return MUON_ERR_ARG;
    if (t->kl_coef != 0.0f && l->rows > 0 && !t->ref_logp) return MUON_ERR_ARG;
    if (l->rows > 0 && (!t->targets || !t->old_logp || !t->advantages)) return MUON_ERR_ARG;
    if (l->rows == 0) return MUON_OK;
    const LossSplit s = split_of(l, 1, ctx_cus(ctx));
    const int wrc = check_workspace(workspace, workspace_bytes, s.bytes);
    if (wrc != MUON_OK) return wrc;
    if (ctx_device(ctx) < 0) return MUON_ERR_DEVICE;
    DeviceGuard dg(ctx_device(ctx));
    if (!dg.ok) return MUON_ERR_HIP;
    LossParams p = params(l);
    apply(s, p, workspace);
    p.targets = t->targets;
    p.old_logp = t->old_logp; p.advantages = t->advantages;
    p.ref_logp = t->kl_coef != 0.0f ? t->ref_logp : nullptr;
    p.clip_low = t->clip_low; p.clip_high = t->clip_high; p.kl_coef = t->kl_coef;
    p.logp = t->logp;
    MUON_HIP(launch_loss(LOSS_POLICY, l->dtype == MUON_BF16, p, static_cast<hipStream_t>(stream)));
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

int muon_distill_loss(muon_ctx* ctx, const muon_logits* l, const muon_distill* t, void* workspace,
                      size_t workspace_bytes, void* stream) {
  try {
    if (!ctx || !t) return MUON_ERR_ARG;
    const int rc = validate(l);
    if (rc != MUON_OK) return rc;
    if (t->top < 1 || t->top > MUON_MAX_TOP || t->ld_top < t->top || t->ld_ids < t->top) return MUON_ERR_ARG;
    if (!dtype_ok(t->top_dtype) || (t->id_dtype != MUON_I32 && t->id_dtype != MUON_I64)) return MUON_ERR_ARG;
    if (l->rows > 0 && (!t->top_logits || !t->top_ids)) return MUON_ERR_ARG;
    if (!aligned(t->top_logits, size_of(t->top_dtype)) || !aligned(t->top_ids, 4)) return MUON_ERR_ARG;
    if (l->rows == 0) return MUON_OK;
    const LossSplit s = split_of(l, t->top, ctx_cus(ctx));
    const int wrc = check_workspace(workspace, workspace_bytes, s.bytes);
    if (wrc != MUON_OK) return wrc;
    if (ctx_device(ctx) < 0) return MUON_ERR_DEVICE;
    DeviceGuard dg(ctx_device(ctx));
    if (!dg.ok) return MUON_ERR_HIP;
    LossParams p = params(l);
    apply(s, p, workspace);
    p.top_logits = t->top_logits; p.ld_top = t->ld_top;
    p.ids = t->top_ids; p.ld_ids = t->ld_ids;
    p.top_lse = t->top_lse;
    p.top = t->top; p.top_bf16 = t->top_dtype == MUON_BF16; p.ids64 = t->id_dtype == MUON_I64;
    MUON_HIP(launch_loss(LOSS_DISTILL, l->dtype == MUON_BF16, p, static_cast<hipStream_t>(stream)));
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

}  // extern "C"
