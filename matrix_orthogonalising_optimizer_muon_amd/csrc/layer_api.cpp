// C-ABI front end of a layer's operators beside the feed-forward block: linear attention with
// decay, tokens sorted by expert and back, dropout. Argument validation, workspace plans and
// launches. The calls only read the context, so several threads may make them on one context.
#include "../../include/muon.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "frontend.hpp"
#include "layer.hpp"

namespace muon {
namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxTokens = (int64_t{1} << 24) - 1;  // a workgroup of 256 threads each: 2^32 threads is past what a launch takes
constexpr int64_t kMaxLd = int64_t{1} << 36;

inline int64_t cdiv(int64_t x, int64_t a) { return (x + a - 1) / a; }
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline bool dtype_ok(int d) { return d == MUON_F32 || d == MUON_BF16; }
inline int64_t size_of(int d) { return d == MUON_F32 ? 4 : 2; }
// Rows whose byte offsets stay within 63 bits.
inline bool span_ok(int64_t rows, int64_t ld) { return ld <= kMaxLd && (rows <= 1 || ld <= (int64_t{1} << 60) / rows); }
inline bool aligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return MUON_OK;
  return !ws || have < need || !aligned(ws, kAlign) ? MUON_ERR_WORKSPACE : MUON_OK;
}

// ---- linear attention ----

bool strides_ok(const int64_t (&s)[3]) {
  for (const int64_t x : s)
    if (x < 0 || x > kMaxLd) return false;  // times 2^24 tokens and 4 bytes: within 63 bits
  return true;
}

int validate_sizes(const muon_mix* m) {
  if (!m || !dtype_ok(m->dtype)) return MUON_ERR_ARG;
  if (m->batch < 0 || m->batch > (int64_t{1} << 20) || m->tokens < 0 || m->tokens > (int64_t{1} << 24)) return MUON_ERR_ARG;
  if (m->heads < 1 || m->heads > 65536 || m->kv_heads < 1 || m->heads % m->kv_heads != 0) return MUON_ERR_ARG;
  if (m->batch * m->heads > (int64_t{1} << 18)) return MUON_ERR_ARG;
  if (m->dim < 1 || m->dim > MUON_MIX_MAX_DIM || m->dim_v < 1 || m->dim_v > MUON_MIX_MAX_DIM) return MUON_ERR_ARG;
  return MUON_OK;
}

int validate(const muon_mix* m) {
  if (validate_sizes(m) != MUON_OK || !std::isfinite(m->scale)) return MUON_ERR_ARG;
  if (!strides_ok(m->q_strides) || !strides_ok(m->k_strides) || !strides_ok(m->v_strides)) return MUON_ERR_ARG;
  const int64_t es = size_of(m->dtype);
  if (!aligned(m->q, es) || !aligned(m->k, es) || !aligned(m->v, es) || !aligned(m->log_decay, 4) || !aligned(m->state, 4) ||
      !aligned(m->lengths, 4))
    return MUON_ERR_ARG;
  if (m->batch > 0 && !m->log_decay) return MUON_ERR_ARG;
  if (m->batch * m->tokens > 0 && (!m->q || !m->k || !m->v)) return MUON_ERR_ARG;
  return MUON_OK;
}

int validate(const muon_mix* m, const muon_mix_grads* g) {
  const int64_t es = size_of(m->dtype);
  if (!strides_ok(g->do_strides)) return MUON_ERR_ARG;
  if (!aligned(g->d_o, es) || !aligned(g->dq, es) || !aligned(g->dk, es) || !aligned(g->dv, es) || !aligned(g->d_final, 4) ||
      !aligned(g->d_state, 4))
    return MUON_ERR_ARG;
  if (m->batch * m->tokens > 0 && !g->d_o) return MUON_ERR_ARG;
  return MUON_OK;
}

// How a (batch, head) is divided: dim_v slices and segments of tokens.
struct MixPlan {
  MixTile tile{64, 64};
  int64_t bh = 0;
  int segments = 1, segment = kMixChunk;
  size_t off_rev = 0, off_dk = 0, off_dv = 0, bytes = 0;  // workspace: states, states of the reversed walk, partial dk, dv
};

// Times of a walk in us, [fp32][dim 64, 128, 256][slice 32, 64, 128]: a chunk and the start and end of the walk with
// outputs, then of the one that only sums a segment's state. Measured with one workgroup on every CU (the second:
// on every other one), 4 to 32 chunks.
struct MixTime {
  float chunk, ends, sum_chunk, sum_ends;
};
constexpr MixTime kMixTime[2][3][3] = {
    {{{1.5f, 5.4f, 0.8f, 5.8f}, {2.0f, 5.5f, 1.0f, 7.0f}, {}},
     {{2.0f, 5.6f, 1.0f, 6.5f}, {2.75f, 7.2f, 1.35f, 6.1f}, {4.3f, 9.4f, 2.0f, 8.9f}},
     {{4.0f, 6.1f, 1.8f, 7.1f}, {5.0f, 9.0f, 2.4f, 9.5f}, {}}},
    {{{3.2f, 6.0f, 0.9f, 6.0f}, {4.8f, 7.7f, 1.5f, 6.0f}, {}},
     {{5.2f, 8.7f, 1.6f, 5.6f}, {8.0f, 9.9f, 3.0f, 7.0f}, {}},
     {{11.2f, 9.1f, 3.6f, 7.6f}, {16.0f, 8.0f, 6.0f, 8.0f}, {}}}};

// A walk over all tokens with wide slices reads and computes least. More workgroups come from narrower slices
// (scores and weighted operands are computed once a slice) or from segments (k and v are read twice, two more
// launches, the states' traffic): the cheapest of both by the measured times. 128 (batch, head)s of 128 x
// 128, 2048 tokens, forward: slices of 64 109 us, of 128 132 us, two segments of those 139 us; gradients (three
// walks): 329, 252 and 304 us. 16 of them, 65536 tokens: 32 segments with slices of 128 460 us, 16 486 us, 8 758 us; slices of 64
// with 32 segments 552 us.
MixPlan plan_of(const muon_mix* m, const muon_mix_grads* g, int cus) {
  MixPlan p;
  p.bh = m->batch * m->heads;
  const bool f32 = m->dtype == MUON_F32;
  const int wide = g ? std::max(m->dim, m->dim_v) : m->dim_v, deep = g ? wide : m->dim;
  const int di = deep <= 64 ? 0 : deep <= 128 ? 1 : 2;
  p.tile.dim = 64 << di;
  const int64_t chunks = std::max<int64_t>(cdiv(m->tokens, kMixChunk), 1);
  const int64_t state = int64_t{4} * m->dim * m->dim_v;
  const bool back = g && (g->dk || g->dv || g->d_state);
  const int sums = g ? (g->dq ? 1 : 0) + (back ? 1 : 0) : 1;   // directions whose segments' states are summed
  double best = 1e300;
  for (int vi = 0; vi < 3; ++vi) {
    const MixTime& t = kMixTime[f32][di][vi];
    const int nv = 32 << vi;
    if (t.chunk == 0.0f || (vi > 0 && nv >= 2 * wide)) continue;
    const int64_t v_slices = cdiv(m->dim_v, nv);
    const int64_t per = !g ? v_slices
                           : std::max<int64_t>(((g->dq ? 1 : 0) + (g->dk ? 1 : 0)) * cdiv(m->dim, nv) + (g->dv || g->d_state ? v_slices : 0), 1);
    int64_t last = 0;
    for (int64_t want = 1; want <= 256 && want <= chunks; want += std::max<int64_t>(1, want / 8)) {
      const int64_t each = cdiv(chunks, want), segments = cdiv(chunks, each);
      if (segments == last) continue;
      last = segments;
      // segments are for walks that leave CUs idle
      if (segments > 1 && (p.bh * segments * state > (int64_t{1} << 30) || p.bh * per > 2 * cus)) break;
      // a last round that leaves CUs idle costs less than a whole one
      auto rounds = [&](int64_t groups, double slots) {
        const double r = groups / slots, whole = std::floor(r);
        return r <= 1.0 ? 1.0 : whole + (r > whole ? 0.5 + 0.5 * (r - whole) : 0.0);
      };
      double us = rounds(p.bh * per * segments, cus) * (each * static_cast<double>(t.chunk) + t.ends);
      if (segments > 1)
        us += rounds(p.bh * sums * v_slices * (segments - 1), 1.3 * cus) * (each * static_cast<double>(t.sum_chunk) + t.sum_ends) + 4.0 +
              2.0 * sums * p.bh * segments * state / 4e6;
      if (us < best) {
        best = us;
        p.tile.dim_v = nv;
        p.segment = static_cast<int>(each * kMixChunk);
        p.segments = static_cast<int>(segments);
      }
    }
  }
  if (p.segments > 1) {
    const size_t z = align_up(static_cast<size_t>(p.bh * p.segments * state));
    p.off_rev = z;
    p.bytes = g ? 2 * z : z;
  }
  if (g && m->heads != m->kv_heads) {
    const int64_t rows = m->batch * m->tokens * m->heads;
    p.off_dk = p.bytes;
    if (g->dk) p.bytes += align_up(static_cast<size_t>(rows * m->dim * 4));
    p.off_dv = p.bytes;
    if (g->dv) p.bytes += align_up(static_cast<size_t>(rows * m->dim_v * 4));
  }
  return p;
}

MixArray array(const void* p, const int64_t (&s)[3], int group) { return {p, s[0], s[1], s[2], group}; }

// Whether the direct loads can take an array: rows of whole 16-byte pieces at 16-byte addresses that do not
// overlap, a chunk of them within 2^29 bytes (the kernels' offsets and their marker of what lies outside need that).
bool direct(const MixArray& a, int dim, int64_t es) {
  const int64_t tok = a.st * es;
  return aligned(a.p, 16) && a.sb * es % 16 == 0 && tok % 16 == 0 && a.sh * es % 16 == 0 && dim * es % 16 == 0 &&
         tok >= dim * es && tok * kMixChunk <= (int64_t{1} << 29);
}

MixParams params(const muon_mix* m, const MixPlan& pl) {
  MixParams p;
  std::memset(&p, 0, sizeof(p));
  p.log_decay = m->log_decay;
  p.lengths = m->lengths;
  p.batch = static_cast<int32_t>(m->batch);
  p.heads = m->heads;
  p.tokens = static_cast<int32_t>(m->tokens);
  p.segments = p.walked = pl.segments;
  p.segment = pl.segment;
  return p;
}

MixRole& add(MixParams& p, const MixPlan& pl, const MixArray& a, const MixArray& b, const MixArray& c, void* out, int dim,
             int dim_v) {
  MixRole& r = p.role[p.roles++];
  r.a = a; r.b = b; r.c = c;
  r.out = out;
  r.dim = dim; r.dim_v = dim_v;
  r.p_scale = r.o_scale = r.u_scale = 1.0f;
  r.z_row = dim_v; r.z_col = 1;
  r.first = p.per;
  p.per += static_cast<int32_t>(cdiv(dim_v, pl.tile.dim_v));   // its slices
  return r;
}

hipError_t walk(bool f32, const MixPlan& pl, bool out, const MixParams& p, hipStream_t st) {
  return launch_mix(f32, pl.tile, out, p, pl.bh * p.per * p.walked, st);
}

// ---- tokens by expert ----

int validate_sizes(const muon_experts* e) {
  if (!e || e->tokens < 0 || e->tokens > kMaxTokens || e->top < 1 || e->top > MUON_MAX_CHOICES) return MUON_ERR_ARG;
  if (e->tokens * e->top > (int64_t{1} << 25) || e->experts < 1 || e->experts > MUON_MAX_EXPERTS) return MUON_ERR_ARG;
  if (e->reserved != 0) return MUON_ERR_ARG;
  return MUON_OK;
}

// Workgroups of a plan. One (a launch less) while it is quick; then 512 choices each, at most 128, and at most 32768
// counters, which every workgroup adds up. Times in us, choices x experts: 1025 x 64: one 6.2, more 7.1; 2048 x 64:
// one 8.4, more 7.3; 2048 x 1024: one 9.2, more 11.7; 16384 x 64: 512 a workgroup 7.6, 1024 10.9, 2048 13.2; 65536 x
// 1024: 128 workgroups 30, 64 21, 32 19.
int plan_blocks(const muon_experts* e) {
  const int64_t n = e->tokens * e->top;
  if (n <= 1536 + 2 * e->experts) return 1;
  return static_cast<int>(std::min<int64_t>({cdiv(n, 512), 128, 32768 / (e->experts + 1)}));
}
size_t plan_bytes(const muon_experts* e) {
  const int blocks = plan_blocks(e);
  return blocks > 1 ? align_up(static_cast<size_t>(blocks) * (e->experts + 1) * 4) : 0;
}

int validate_rows(const muon_experts* e, int64_t dim, int dtype) {
  if (validate_sizes(e) != MUON_OK || !dtype_ok(dtype) || dim < 1 || dim > (int64_t{1} << 20)) return MUON_ERR_ARG;
  if (!aligned(e->slots, 4) || !aligned(e->offsets, 4)) return MUON_ERR_ARG;
  return e->tokens > 0 && (!e->slots || !e->offsets) ? MUON_ERR_ARG : MUON_OK;
}
bool rows_ok(const void* p, int64_t ld, int64_t dim, int dtype, bool needed) {
  return ld >= dim && span_ok(int64_t{1} << 25, ld) && aligned(p, size_of(dtype)) && (p || !needed);
}

RowsParams rows_params(const muon_experts* e, int64_t dim, int dtype) {
  RowsParams p;
  std::memset(&p, 0, sizeof(p));
  p.slots = e->slots;
  p.offsets = e->offsets;
  p.tokens = e->tokens;
  p.top = e->top;
  p.experts = e->experts;
  p.dim = static_cast<int32_t>(dim);
  p.once = e->tokens * e->top * dim * size_of(dtype) > (int64_t{128} << 20);  // half the 256 MB cache
  return p;
}

// ---- dropout ----

// Whether two row sets of one shape share an element without being the same rows.
bool overlaps(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t rows, int64_t cols, int64_t es) {
  if (a == b && (lda == ldb || rows == 1)) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  const uintptr_t na = static_cast<uintptr_t>(((rows - 1) * lda + cols) * es);
  const uintptr_t nb = static_cast<uintptr_t>(((rows - 1) * ldb + cols) * es);
  if (pa + na <= pb || pb + nb <= pa) return false;
  if (lda != ldb) return true;
  const uintptr_t row = static_cast<uintptr_t>(lda * es), width = static_cast<uintptr_t>(cols * es);
  const uintptr_t shift = (pb > pa ? pb - pa : pa - pb) % row;
  return shift < width || shift + width > row;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

int muon_mix_workspace_size(muon_ctx* ctx, const muon_mix* m, const muon_mix_grads* g, size_t* bytes) {
  try {
    if (!ctx || !bytes || validate_sizes(m) != MUON_OK) return MUON_ERR_ARG;
    *bytes = plan_of(m, g, ctx_cus(ctx)).bytes;
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

int muon_mix_forward(muon_ctx* ctx, const muon_mix* m, void* o, float* final_state, void* workspace, size_t workspace_bytes,
                     void* stream) {
  try {
    if (!ctx) return MUON_ERR_ARG;
    int rc = validate(m);
    if (rc != MUON_OK) return rc;
    if (!aligned(o, size_of(m->dtype)) || !aligned(final_state, 4) || (m->batch * m->tokens > 0 && !o)) return MUON_ERR_ARG;
    if (m->batch == 0 || (m->tokens == 0 && !final_state)) return MUON_OK;
    const MixPlan pl = plan_of(m, nullptr, ctx_cus(ctx));
    rc = check_workspace(workspace, workspace_bytes, pl.bytes);
    if (rc != MUON_OK) return rc;
    if (ctx_device(ctx) < 0) return MUON_ERR_DEVICE;
    DeviceGuard dg(ctx_device(ctx));
    if (!dg.ok) return MUON_ERR_HIP;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const bool f32 = m->dtype == MUON_F32;
    const int group = m->heads / m->kv_heads;
    const MixArray q = array(m->q, m->q_strides, 1), k = array(m->k, m->k_strides, group), v = array(m->v, m->v_strides, group);
    float* z = static_cast<float*>(workspace);
    MixParams p = params(m, pl);
    const int64_t es = size_of(m->dtype);
    p.direct = direct(q, m->dim, es) && direct(k, m->dim, es) && direct(v, m->dim_v, es);
    if (pl.segments > 1) {
      MixParams s = p;
      add(s, pl, q, k, v, nullptr, m->dim, m->dim_v).z_out = z;
      s.z_out_per_segment = 1;
      s.walked = pl.segments - 1;
      MUON_HIP(walk(f32, pl, false, s, st));
      MixScan c;
      std::memset(&c, 0, sizeof(c));
      c.one[0] = {m->state, z, m->dim * m->dim_v};
      c.count = 1;
      c.log_decay = m->log_decay; c.lengths = m->lengths;
      c.batch = p.batch; c.heads = p.heads; c.tokens = p.tokens; c.segments = p.segments; c.segment = p.segment;
      MUON_HIP(launch_mix_scan(c, st));
    }
    MixRole& r = add(p, pl, q, k, v, o, m->dim, m->dim_v);
    r.p_scale = r.o_scale = m->scale;
    r.z_in = pl.segments > 1 ? z : m->state;
    r.z_out = final_state;
    p.z_in_per_segment = pl.segments > 1;
    MUON_HIP(walk(f32, pl, true, p, st));
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

int muon_mix_backward(muon_ctx* ctx, const muon_mix* m, const muon_mix_grads* g, void* workspace, size_t workspace_bytes,
                      void* stream) {
  try {
    if (!ctx || !g) return MUON_ERR_ARG;
    int rc = validate(m);
    if (rc == MUON_OK) rc = validate(m, g);
    if (rc != MUON_OK) return rc;
    if (m->batch == 0 || (!g->dq && !g->dk && !g->dv && !g->d_state) || (m->tokens == 0 && !g->d_state)) return MUON_OK;
    const MixPlan pl = plan_of(m, g, ctx_cus(ctx));
    rc = check_workspace(workspace, workspace_bytes, pl.bytes);
    if (rc != MUON_OK) return rc;
    if (ctx_device(ctx) < 0) return MUON_ERR_DEVICE;
    DeviceGuard dg(ctx_device(ctx));
    if (!dg.ok) return MUON_ERR_HIP;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const bool f32 = m->dtype == MUON_F32;
    const int group = m->heads / m->kv_heads;
    const MixArray q = array(m->q, m->q_strides, 1), k = array(m->k, m->k_strides, group), v = array(m->v, m->v_strides, group);
    const MixArray d_o = array(g->d_o, g->do_strides, 1);
    char* ws = static_cast<char*>(workspace);
    float *z = reinterpret_cast<float*>(ws), *zr = reinterpret_cast<float*>(ws + pl.off_rev);
    const bool back = g->dk || g->dv || g->d_state;
    MixParams p = params(m, pl);
    const int64_t es = size_of(m->dtype);
    p.direct = direct(q, m->dim, es) && direct(k, m->dim, es) && direct(v, m->dim_v, es) && direct(d_o, m->dim_v, es);
    if (pl.segments > 1) {
      MixParams s = p;
      MixScan c;
      std::memset(&c, 0, sizeof(c));
      if (g->dq) {
        add(s, pl, q, k, v, nullptr, m->dim, m->dim_v).z_out = z;
        c.one[c.count++] = {m->state, z, m->dim * m->dim_v};
      }
      if (back) {
        MixRole& r = add(s, pl, k, q, d_o, nullptr, m->dim, m->dim_v);
        r.z_out = zr;
        r.reversed = 1;
        r.u_scale = m->scale;
        c.one[c.count++] = {g->d_final, zr, m->dim * m->dim_v};
      }
      s.z_out_per_segment = 1;
      s.walked = pl.segments - 1;
      MUON_HIP(walk(f32, pl, false, s, st));
      c.log_decay = m->log_decay; c.lengths = m->lengths;
      c.batch = p.batch; c.heads = p.heads; c.tokens = p.tokens; c.segments = p.segments; c.segment = p.segment;
      MUON_HIP(launch_mix_scan(c, st));
      p.z_in_per_segment = 1;
    }
    if (g->dq) {
      MixRole& r = add(p, pl, d_o, v, k, g->dq, m->dim_v, m->dim);
      r.p_scale = r.o_scale = m->scale;
      r.z_in = pl.segments > 1 ? z : m->state;
      r.z_row = 1;
      r.z_col = m->dim_v;
    }
    if (g->dk) {
      MixRole& r = add(p, pl, v, d_o, q, group > 1 ? static_cast<void*>(ws + pl.off_dk) : g->dk, m->dim_v, m->dim);
      r.out_f32 = group > 1;
      r.reversed = 1;
      r.p_scale = r.u_scale = m->scale;
      r.z_in = pl.segments > 1 ? zr : g->d_final;
      r.z_row = 1;
      r.z_col = m->dim_v;
    }
    MixParams alone = p;                         // d_state without dv: the walk that makes no outputs
    alone.roles = alone.per = 0;
    if (g->dv || g->d_state) {
      MixRole& r = add(g->dv ? p : alone, pl, k, q, d_o, !g->dv ? nullptr : group > 1 ? static_cast<void*>(ws + pl.off_dv) : g->dv, m->dim, m->dim_v);
      r.out_f32 = group > 1;
      r.reversed = 1;
      r.p_scale = r.u_scale = m->scale;
      r.z_in = pl.segments > 1 ? zr : g->d_final;
      r.z_out = g->d_state;
    }
    if (p.roles > 0) MUON_HIP(walk(f32, pl, true, p, st));
    if (alone.roles > 0) MUON_HIP(walk(f32, pl, false, alone, st));
    if (group > 1 && m->tokens > 0 && (g->dk || g->dv)) {
      MixShare s;
      std::memset(&s, 0, sizeof(s));
      if (g->dk) s.one[s.count++] = {reinterpret_cast<float*>(ws + pl.off_dk), g->dk, m->dim};
      if (g->dv) s.one[s.count++] = {reinterpret_cast<float*>(ws + pl.off_dv), g->dv, m->dim_v};
      s.kv_heads = m->kv_heads;
      s.group = group;
      s.bf16 = !f32;
      s.rows = m->batch * m->tokens;
      MUON_HIP(launch_mix_share(s, st));
    }
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

int muon_mix_step(muon_ctx* ctx, const muon_mix* m, void* o, float* new_state, void* stream) {
  try {
    if (!ctx) return MUON_ERR_ARG;
    const int rc = validate(m);
    if (rc != MUON_OK) return rc;
    if (m->tokens != 1 || m->lengths || !aligned(o, size_of(m->dtype)) || !aligned(new_state, 4)) return MUON_ERR_ARG;
    if (m->batch > 0 && (!m->state || !o || !new_state)) return MUON_ERR_ARG;
    const uintptr_t a = reinterpret_cast<uintptr_t>(m->state), b = reinterpret_cast<uintptr_t>(new_state);
    const uintptr_t bytes = static_cast<uintptr_t>(m->batch * m->heads * m->dim * m->dim_v * 4);
    if (a != b && a < b + bytes && b < a + bytes) return MUON_ERR_ARG;
    if (m->batch == 0) return MUON_OK;
    if (ctx_device(ctx) < 0) return MUON_ERR_DEVICE;
    DeviceGuard dg(ctx_device(ctx));
    if (!dg.ok) return MUON_ERR_HIP;
    MixStep p;
    std::memset(&p, 0, sizeof(p));
    p.q = m->q; p.k = m->k; p.v = m->v;
    p.q_sb = m->q_strides[0]; p.q_sh = m->q_strides[2];
    p.k_sb = m->k_strides[0]; p.k_sh = m->k_strides[2];
    p.v_sb = m->v_strides[0]; p.v_sh = m->v_strides[2];
    p.log_decay = m->log_decay;
    p.z_in = m->state; p.z_out = new_state;
    p.out = o;
    p.scale = m->scale;
    p.batch = static_cast<int32_t>(m->batch); p.heads = m->heads; p.group = m->heads / m->kv_heads;
    p.dim = m->dim; p.dim_v = m->dim_v;
    // All columns a workgroup where states fill the CUs: rows that are not whole cache lines would share them with another
    // workgroup's. 4096 states, 64 columns or all, us: 16 x 256: 55.5 or 29.1; 64 x 256: 110 or 104; 128 x 128: 107 or 105;
    // 40 x 72: 33 or 21; 33 x 129: 56 or 33. Fewer states: 64, or 32 where that leaves CUs idle (16 of 128 x 128, 32, 64 and
    // 128 columns: 4.5, 4.9, 5.9 us).
    const int64_t states = m->batch * m->heads;
    const int all = static_cast<int>(cdiv(m->dim_v, 4));
    p.lanes = states >= ctx_cus(ctx) ? all : states * cdiv(m->dim_v, 64) < ctx_cus(ctx) ? 8 : 16;
    p.lanes = std::min(p.lanes, all);
    MUON_HIP(launch_mix_step(m->dtype == MUON_F32, p, static_cast<hipStream_t>(stream)));
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

int muon_expert_plan_workspace_size(muon_ctx* ctx, const muon_experts* e, size_t* bytes) {
  try {
    if (!ctx || !bytes || validate_sizes(e) != MUON_OK) return MUON_ERR_ARG;
    *bytes = plan_bytes(e);
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

int muon_expert_plan(muon_ctx* ctx, const muon_experts* e, void* workspace, size_t workspace_bytes, void* stream) {
  try {
    if (!ctx || validate_sizes(e) != MUON_OK) return MUON_ERR_ARG;
    if (e->id_dtype != MUON_I32 && e->id_dtype != MUON_I64) return MUON_ERR_ARG;
    if (!aligned(e->ids, e->id_dtype == MUON_I64 ? 8 : 4) || !aligned(e->order, 4) || !aligned(e->slots, 4) || !aligned(e->offsets, 4))
      return MUON_ERR_ARG;
    if (!e->offsets || (e->tokens > 0 && (!e->ids || !e->order || !e->slots))) return MUON_ERR_ARG;
    const int rc = check_workspace(workspace, workspace_bytes, plan_bytes(e));
    if (rc != MUON_OK) return rc;
    if (ctx_device(ctx) < 0) return MUON_ERR_DEVICE;
    DeviceGuard dg(ctx_device(ctx));
    if (!dg.ok) return MUON_ERR_HIP;
    PlanParams p;
    std::memset(&p, 0, sizeof(p));
    p.ids = e->ids;
    p.ids64 = e->id_dtype == MUON_I64;
    p.n = e->tokens * e->top;
    p.experts = e->experts;
    p.blocks = plan_blocks(e);
    p.order = e->order; p.slots = e->slots; p.offsets = e->offsets;
    p.counts = static_cast<int32_t*>(workspace);
    MUON_HIP(launch_expert_plan(p, static_cast<hipStream_t>(stream)));
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

int muon_expert_dispatch(muon_ctx* ctx, const muon_experts* e, const void* token, int64_t ld_token, void* sorted,
                         int64_t ld_sorted, int64_t dim, int dtype, void* stream) {
  try {
    if (!ctx || validate_rows(e, dim, dtype) != MUON_OK) return MUON_ERR_ARG;
    const bool any = e->tokens > 0;
    if (!rows_ok(token, ld_token, dim, dtype, any) || !rows_ok(sorted, ld_sorted, dim, dtype, any)) return MUON_ERR_ARG;
    if (!any) return MUON_OK;
    if (ctx_device(ctx) < 0) return MUON_ERR_DEVICE;
    DeviceGuard dg(ctx_device(ctx));
    if (!dg.ok) return MUON_ERR_HIP;
    RowsParams p = rows_params(e, dim, dtype);
    p.in = token; p.ld_in = ld_token;
    p.out = sorted; p.ld_out = ld_sorted;
    MUON_HIP(launch_expert_rows(ROWS_DISPATCH, dtype == MUON_F32, p, static_cast<hipStream_t>(stream)));
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

int muon_expert_combine(muon_ctx* ctx, const muon_experts* e, const void* sorted, int64_t ld_sorted, const float* weights,
                        void* token, int64_t ld_token, int64_t dim, int dtype, void* stream) {
  try {
    if (!ctx || validate_rows(e, dim, dtype) != MUON_OK) return MUON_ERR_ARG;
    const bool any = e->tokens > 0;
    if (!rows_ok(token, ld_token, dim, dtype, any) || !rows_ok(sorted, ld_sorted, dim, dtype, any) || !aligned(weights, 4))
      return MUON_ERR_ARG;
    if (!any) return MUON_OK;
    if (ctx_device(ctx) < 0) return MUON_ERR_DEVICE;
    DeviceGuard dg(ctx_device(ctx));
    if (!dg.ok) return MUON_ERR_HIP;
    RowsParams p = rows_params(e, dim, dtype);
    p.weights = weights;
    p.in = sorted; p.ld_in = ld_sorted;
    p.out = token; p.ld_out = ld_token;
    MUON_HIP(launch_expert_rows(ROWS_COMBINE, dtype == MUON_F32, p, static_cast<hipStream_t>(stream)));
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

int muon_expert_combine_backward(muon_ctx* ctx, const muon_experts* e, const void* d_token, int64_t ld_token,
                                 const void* sorted, int64_t ld_sorted, const float* weights, void* d_sorted,
                                 int64_t ld_d_sorted, float* d_weights, int64_t dim, int dtype, void* stream) {
  try {
    if (!ctx || validate_rows(e, dim, dtype) != MUON_OK) return MUON_ERR_ARG;
    const bool any = e->tokens > 0;
    if (!rows_ok(d_token, ld_token, dim, dtype, any) || !aligned(weights, 4) || !aligned(d_weights, 4)) return MUON_ERR_ARG;
    if ((d_weights && !rows_ok(sorted, ld_sorted, dim, dtype, any)) || (d_sorted && !rows_ok(d_sorted, ld_d_sorted, dim, dtype, any)))
      return MUON_ERR_ARG;
    if (!any || (!d_sorted && !d_weights)) return MUON_OK;
    if (ctx_device(ctx) < 0) return MUON_ERR_DEVICE;
    DeviceGuard dg(ctx_device(ctx));
    if (!dg.ok) return MUON_ERR_HIP;
    RowsParams p = rows_params(e, dim, dtype);
    p.weights = weights;
    p.in = d_token; p.ld_in = ld_token;
    p.in2 = sorted; p.ld_in2 = ld_sorted;
    p.out = d_sorted; p.ld_out = ld_d_sorted;
    p.dw = d_weights;
    MUON_HIP(launch_expert_rows(ROWS_COMBINE_GRAD, dtype == MUON_F32, p, static_cast<hipStream_t>(stream)));
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

int muon_dropout(muon_ctx* ctx, const muon_drop* d, void* stream) {
  try {
    if (!ctx || !d || !dtype_ok(d->dtype)) return MUON_ERR_ARG;
    if (d->rows < 0 || d->rows >= (int64_t{1} << 31) || d->cols < 1 || d->cols > (int64_t{1} << 34)) return MUON_ERR_ARG;
    if (d->rows > (int64_t{1} << 34) / d->cols || !(d->p >= 0.0f && d->p <= 1.0f)) return MUON_ERR_ARG;
    const int64_t es = size_of(d->dtype);
    auto ld_ok = [&](int64_t ld) { return ld >= d->cols && span_ok(d->rows, ld); };
    if (!ld_ok(d->ld_x) || !ld_ok(d->ld_out) || (d->residual && !ld_ok(d->ld_residual))) return MUON_ERR_ARG;
    if (!aligned(d->x, es) || !aligned(d->residual, es) || !aligned(d->out, es) || !aligned(d->counter, 8)) return MUON_ERR_ARG;
    if (d->rows == 0) return MUON_OK;
    if (!d->x || !d->out) return MUON_ERR_ARG;
    if (overlaps(d->out, d->ld_out, d->x, d->ld_x, d->rows, d->cols, es) ||
        (d->residual && overlaps(d->out, d->ld_out, d->residual, d->ld_residual, d->rows, d->cols, es)))
      return MUON_ERR_ARG;
    if (ctx_device(ctx) < 0) return MUON_ERR_DEVICE;
    DeviceGuard dg(ctx_device(ctx));
    if (!dg.ok) return MUON_ERR_HIP;
    DropParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = d->x; p.residual = d->residual; p.out = d->out;
    p.ld_x = d->ld_x; p.ld_r = d->ld_residual; p.ld_o = d->ld_out;
    p.rows = d->rows; p.cols = d->cols;
    // rows that follow each other are one
    if (d->ld_x == d->cols && d->ld_out == d->cols && (!d->residual || d->ld_residual == d->cols)) {
      p.cols = d->rows * d->cols;
      p.rows = 1;
    }
    p.seed = d->seed; p.offset = d->offset; p.counter = d->counter;
    p.threshold = static_cast<uint32_t>(std::floor(static_cast<double>(d->p) * 65536.0 + 0.5));
    p.factor = p.threshold < 65536 ? 65536.0f / static_cast<float>(65536 - p.threshold) : 0.0f;
    MUON_HIP(launch_dropout(d->dtype == MUON_F32, p, static_cast<hipStream_t>(stream)));
    return MUON_OK;
  } catch (...) {
    return MUON_ERR_HIP;
  }
}

}  // extern "C"
