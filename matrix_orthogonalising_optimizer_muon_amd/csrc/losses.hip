// Losses over vocabulary logits, each with its gradient: the clipped policy loss with a KL
// term, and distillation from a teacher's top logits.
//
// Row r, z = logits / tau, q = softmax(z), lse = log sum exp z, upstream gradient u_r:
//   policy:  lp = z_t - lse, rho = exp(lp - old),
//            l = -min(rho A, clip(rho, 1 - cl, 1 + ch) A) + beta (exp(ref - lp) - (ref - lp) - 1)
//            dl/dlp = -(rho A where min takes it, else 0) + beta (1 - exp(ref - lp))
//            dlogits_v = w u dl/dlp ([v = t] - q_v) / tau
//   distill: p_j = exp(t_j / tau - L) for the kept entries (id i_j), P = sum p,
//            l = sum_j p_j (log p_j - z_{i_j} + lse)
//            dlogits_v = w u (P q_v - sum_{j: i_j = v} p_j) / tau
//
// One workgroup per row. The first pass keeps each thread's running maximum m and sum s of
// exp(z - m) over its columns (one rescale per 16 values), joined in a fixed order; the second
// writes the gradient. All of it in fp32; exp((z - m) c) is formed from the difference, so
// that rows of the type's lowest values stay exact, and q = e / s.
//
// Bound by HBM: the logits read once, the gradient written once. 4096 x 151936 bf16, a fifth of
// the rows without weight: 437-445 us, 5.1 TB/s (a copy reaches 5.1); 2048 x 152064 with 64 kept
// entries: 271-278 us, 4.3 TB/s, where one row a CU at a time leaves the last of 7.2 rounds partly
// idle. The arithmetic (two exponentials a column, about 17 instructions) takes some 18 us a row of
// 152064 on a CU and hides behind the row's 30 us of traffic.
#include <type_traits>

#include "mfma_util.hpp"
#include "train.hpp"

namespace muon {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// 16 bytes at any element alignment (one instruction; the address may straddle lines).
template <int A>
struct Chunk;
template <>
struct Chunk<2> {
  typedef u32x4 T __attribute__((aligned(2)));
};
template <>
struct Chunk<4> {
  typedef u32x4 T __attribute__((aligned(4)));
};

template <typename E>
struct Row {
  static constexpr int VEC = 16 / sizeof(E);
  typedef typename Chunk<sizeof(E)>::T C;
  static __device__ __forceinline__ u32x4 load(const E* p) { return *reinterpret_cast<const C*>(p); }
  static __device__ __forceinline__ void unpack(const u32x4& w, float (&v)[VEC]) {
    if constexpr (sizeof(E) == 4) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(w[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
      }
    }
  }
  static __device__ __forceinline__ E to(float f) {
    if constexpr (sizeof(E) == 4) return f;
    else return __builtin_bit_cast(unsigned short, static_cast<__bf16>(f));
  }
  static __device__ __forceinline__ float from(E e) {
    if constexpr (sizeof(E) == 4) return e;
    else return __uint_as_float(static_cast<unsigned int>(e) << 16);
  }
  static __device__ __forceinline__ void store(E* p, const float (&v)[VEC]) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (sizeof(E) == 4) w[e] = __float_as_uint(v[e]);
      else w[e] = to(v[2 * e]) | (static_cast<unsigned int>(to(v[2 * e + 1])) << 16);
    }
    *reinterpret_cast<C*>(p) = w;
  }
};

// Running maximum and sum of exp2((x - m) c). A maximum of -inf stands for nothing seen
// yet (or only masked columns): differences are then taken from 0, so that exp2 gives 0.
struct Stat {
  float m, s;
};
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, float c) {
  const float m = fmaxf(a.m, b.m), at = base_of(m);
  return {m, a.s * __builtin_amdgcn_exp2f((a.m - at) * c) + b.s * __builtin_amdgcn_exp2f((b.m - at) * c)};
}

// Reductions over 16 lanes by lane permutes within the vector instruction (neighbours,
// pairs, halves of 8, halves of 16; every lane ends with the result), the rest of a wave by
// two shuffles. No contraction in the sums: fused with the product that made v, the first addition
// would round each lane's own product differently from its neighbour's, and the lanes would end
// with different last bits.
template <int CTRL>
__device__ __forceinline__ float permuted(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float max16(float v) {
  v = fmaxf(v, permuted<0xB1>(v));   // lanes 1 0 3 2
  v = fmaxf(v, permuted<0x4E>(v));   // lanes 2 3 0 1
  v = fmaxf(v, permuted<0x141>(v));  // mirrored in 8
  return fmaxf(v, permuted<0x140>(v));  // mirrored in 16
}
__device__ __forceinline__ float sum16(float v) {
#pragma clang fp contract(off)
  v += permuted<0xB1>(v);
  v += permuted<0x4E>(v);
  v += permuted<0x141>(v);
  return v + permuted<0x140>(v);
}
__device__ __forceinline__ float max64(float v) {
  v = max16(v);
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum64(float v) {
#pragma clang fp contract(off)
  v = sum16(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Joined over the workgroup, in a fixed order; every thread receives the result. The maximum
// first, then one rescale and the sum (joining pairs of statistics step by step took 1.4 us
// of a row's 34). `lds`: at least 16 entries that this call alone uses, so that one barrier
// is enough.
template <int THREADS>
__device__ __forceinline__ Stat join_all(Stat v, float c, Stat* lds) {
  const int lane = threadIdx.x & 63;
  float m = max64(v.m);
  const float s = sum64(v.s * __builtin_amdgcn_exp2f((v.m - base_of(m)) * c));
  if (lane == 0) lds[threadIdx.x >> 6] = Stat{m, s};
  __syncthreads();
  const Stat x = (lane & 15) < THREADS / 64 ? lds[lane & 15] : Stat{-INFINITY, 0.0f};
  m = max16(x.m);
  return {m, sum16(x.s * __builtin_amdgcn_exp2f((x.m - base_of(m)) * c))};
}
template <int THREADS>
__device__ __forceinline__ float sum_all(float v, float* lds) {
  const int lane = threadIdx.x & 63;
  v = sum64(v);
  if (lane == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return sum16((lane & 15) < THREADS / 64 ? lds[lane & 15] : 0.0f);
}

// exp(d) - 1 without cancellation: the series for small d (next term d^6 / 720 below
// 2^-24 of the result for |d| < 0.1), else the exponential.
__device__ __forceinline__ float expm1_f(float d) {
  if (fabsf(d) < 0.1f)
    return d * (1.0f + d * (0.5f + d * (0.16666667f + d * (0.041666668f + d * 0.0083333338f))));
  return __builtin_amdgcn_exp2f(d * kLog2e) - 1.0f;
}

struct Shared {
  Stat row[16], teacher[16];
  float mass[16], loss[16];
};

// Few long rows: every row is split into p.splits parts of p.part vectors, one workgroup
// each. This kernel leaves each part's running maximum and sum, and the row's own logits
// (the target's, or the kept entries'), which a gradient in place may overwrite, in the
// workspace; loss_kernel with SPLIT joins them and does the rest.
template <typename E, int LOSS, int THREADS>
__global__ __launch_bounds__(THREADS) void loss_parts(const LossParams p) {
  using R = Row<E>;
  __shared__ Stat lds[16];
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x / p.splits;
  const int part = blockIdx.x - static_cast<int>(r) * p.splits;
  const int V = p.vocab;
  const E* z = static_cast<const E*>(p.logits) + r * p.ld;
  if (p.weights && p.weights[r] == 0.0f) return;
  if (LOSS == LOSS_POLICY && (p.targets[r] < 0 || p.targets[r] >= V)) return;
  if (part == 0) {
    float* own = p.own + r * (LOSS == LOSS_POLICY ? 1 : p.top);
    if constexpr (LOSS == LOSS_POLICY) {
      if (tid == 0) own[0] = R::from(z[p.targets[r]]);
    } else {
      for (int j = tid; j < p.top; j += THREADS) {
        const int64_t id = p.ids64 ? static_cast<const int64_t*>(p.ids)[r * p.ld_ids + j]
                                   : static_cast<const int32_t*>(p.ids)[r * p.ld_ids + j];
        own[j] = id >= 0 && id < V ? R::from(z[id]) : 0.0f;
      }
    }
  }
  if (p.lse_given) return;
  const float c = p.inv_temperature * kLog2e;
  const int full = V / R::VEC;
  const int first = part * p.part, last = min(full, first + p.part);
  Stat st{-INFINITY, 0.0f};
#pragma unroll 4
  for (int i = first + tid; i < last; i += THREADS) {
    float v[R::VEC];
    R::unpack(R::load(z + static_cast<int64_t>(i) * R::VEC), v);
    float mx = st.m;
#pragma unroll
    for (int e = 0; e < R::VEC; ++e) mx = fmaxf(mx, v[e]);
    const float at = base_of(mx);
    float s = st.s * __builtin_amdgcn_exp2f((st.m - at) * c);
#pragma unroll
    for (int e = 0; e < R::VEC; ++e) s += __builtin_amdgcn_exp2f((v[e] - at) * c);
    st = {mx, s};
  }
  const int tail = full * R::VEC + tid;
  if (part == p.splits - 1 && tail < V) {
    const float v = R::from(z[tail]);
    st = join(st, Stat{v, v == v ? 1.0f : v}, c);
  }
  st = join_all<THREADS>(st, c, lds);
  if (tid == 0) {
    p.stats[(r * p.splits + part) * 2] = st.m;
    p.stats[(r * p.splits + part) * 2 + 1] = st.s;
  }
}

// NV > 0: the row stays in registers between the passes, NV 16-byte vectors a thread, and is
// read once. NV == 0: the second pass reads it again (rows too long to hold). SPLIT: the
// second pass of one part of a row, after loss_parts. SAFE: the row has more than
// SAFE x THREADS vectors.
template <typename E, int LOSS, int THREADS, int NV, int SAFE, bool SPLIT = false>
__global__ __launch_bounds__(THREADS) void loss_kernel(const LossParams p) {
  static_assert(!SPLIT || NV == 0, "a part is read again");
  using R = Row<E>;
  constexpr int VEC = R::VEC;
  constexpr int KT = LOSS == LOSS_DISTILL ? (kMaxTop + THREADS - 1) / THREADS : 1;  // kept entries a thread takes
  __shared__ Shared sh;
  __shared__ __attribute__((aligned(16))) int col[LOSS == LOSS_DISTILL ? kMaxTop : 4];   // the kept entries' columns, -1: absent
  __shared__ float p_of[LOSS == LOSS_DISTILL ? kMaxTop : 1];    // their teacher probabilities p, then loss terms
  __shared__ float lp_of[LOSS == LOSS_DISTILL ? kMaxTop : 1];   // log2 p, then the student's logit
  __shared__ float fix_of[LOSS == LOSS_DISTILL ? kMaxTop : 1];  // the column's sum of p (-1: absent, or not the column's first)
  __shared__ int head[LOSS == LOSS_DISTILL ? THREADS : 1];      // entries by the thread that writes their column
  __shared__ int next_of[LOSS == LOSS_DISTILL ? kMaxTop : 1];

  const int tid = threadIdx.x;
  const int64_t r = SPLIT ? blockIdx.x / p.splits : blockIdx.x;
  const int part = SPLIT ? static_cast<int>(blockIdx.x - r * p.splits) : 0;
  const int V = p.vocab;
  const E* z = static_cast<const E*>(p.logits) + r * p.ld;
  E* d = p.dlogits ? static_cast<E*>(p.dlogits) + r * p.ld_d : nullptr;
  const float c = p.inv_temperature * kLog2e;
  // the row's scalars, requested together
  const float w = p.weights ? p.weights[r] : 1.0f;
  const float up = p.grad_rows ? p.grad_rows[r] : 1.0f;
  float adv = 0.0f, old_logp = 0.0f, ref_logp = 0.0f;
  int64_t target = 0;
  if constexpr (LOSS == LOSS_POLICY) {
    target = p.targets[r];
    adv = p.advantages[r];
    old_logp = p.old_logp[r];
    if (p.ref_logp) ref_logp = p.ref_logp[r];
  }
  const int full = V / VEC;                 // whole vectors
  const int v0 = SPLIT ? part * p.part : 0, v1 = SPLIT ? min(full, v0 + p.part) : full;  // this workgroup's
  const bool last_part = !SPLIT || part == p.splits - 1;
  // the column behind the whole vectors that this thread takes
  const int tail = last_part ? full * VEC + tid : V;
  const bool first = tid == 0 && part == 0;  // writes the row's scalars

  // A row that takes no part (weight 0, or no target) is not read.
  if (w == 0.0f || target < 0 || target >= V) {
    if (first) {
      if (p.loss) p.loss[r] = 0.0f;
      if (!p.lse_given && p.lse) {
        if (p.lse_pairs) p.lse[2 * r] = p.lse[2 * r + 1] = 0.0f;
        else p.lse[r] = 0.0f;
      }
      if (LOSS == LOSS_POLICY && p.logp) p.logp[r] = 0.0f;
    }
    if (d) {
      float zero[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) zero[e] = 0.0f;
      for (int i = v0 + tid; i < v1; i += THREADS) R::store(d + static_cast<int64_t>(i) * VEC, zero);
      if (tail < V) d[tail] = R::to(0.0f);
    }
    return;
  }

  // The teacher's entries are requested before the row and decoded after it (loads return in
  // order): their columns' logits, their normaliser and mass and the repeated columns are
  // dealt with while the row is on its way. Ids as two words, the upper one of a 32-bit id
  // being itself.
  unsigned int id_lo[KT], id_hi[KT], t_word[KT];
  if constexpr (LOSS == LOSS_DISTILL) {
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const int j = min(k * THREADS + tid, p.top - 1);
      const char* id = static_cast<const char*>(p.ids) + (r * p.ld_ids + j) * (p.ids64 ? 8 : 4);
      id_lo[k] = *reinterpret_cast<const unsigned int*>(id);
      id_hi[k] = *reinterpret_cast<const unsigned int*>(id + (p.ids64 ? 4 : 0));
      const int64_t t = r * p.ld_top + j;
      if (p.top_bf16) t_word[k] = static_cast<const unsigned short*>(p.top_logits)[t];
      else t_word[k] = static_cast<const unsigned int*>(p.top_logits)[t];
    }
  }
  const float zl = R::from(z[min(tail, V - 1)]);
  float zt = 0.0f;
  if constexpr (LOSS == LOSS_POLICY) zt = SPLIT ? p.own[r] : R::from(z[target]);
  u32x4 row[NV > 0 ? NV : 1];
  if constexpr (NV > 0) {
    // past the row's last vector a thread loads that one again and leaves it out below
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i < SAFE) row[i] = R::load(z + i * THREADS * VEC + tid * VEC);
      else row[i] = R::load(z + min(i * THREADS + tid, full - 1) * VEC);
      // in the order of their use, and the entries' decoding behind them
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  float mass = 0.0f;
  if constexpr (LOSS == LOSS_DISTILL) {
    head[tid] = -1;
    float tt[KT];
    int tc[KT];
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const int j = k * THREADS + tid;
      const int64_t id = p.ids64 ? static_cast<int64_t>((static_cast<uint64_t>(id_hi[k]) << 32) | id_lo[k])
                                 : static_cast<int32_t>(id_lo[k]);
      const bool in = j < p.top && id >= 0 && id < V;
      tc[k] = in ? static_cast<int>(id) : -1;
      const float t = __uint_as_float(p.top_bf16 ? t_word[k] << 16 : t_word[k]);
      tt[k] = in ? t : -INFINITY;
    }
    // log2 p_j = (t_j - tm) c - log2 of the sum, p_j = exp2((t_j - tm) c) / sum; with the
    // normaliser L given the difference t_j / tau - L first, whose rounding is that of a small
    // number. (p_j from log2 p_j, or L scaled first, has 2 to 4 times the error.)
    float tm, tlog2, tinv, lse_t = 0.0f;
    if (p.top_lse) {
      tm = tlog2 = 0.0f;
      tinv = 1.0f;
      lse_t = p.top_lse[r];
    } else {
      Stat st{-INFINITY, 0.0f};
#pragma unroll
      for (int k = 0; k < KT; ++k) st = join(st, Stat{tt[k], tt[k] == -INFINITY ? 0.0f : 1.0f}, c);
      st = join_all<THREADS>(st, c, sh.teacher);
      tm = base_of(st.m);
      tlog2 = __builtin_amdgcn_logf(st.s);
      tinv = 1.0f / st.s;
      mass = st.s > 0.0f ? 1.0f : st.s;  // normalised among themselves; 0: no entries; NaN stays
    }
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const float e = p.top_lse ? fmaf(tt[k], p.inv_temperature, -lse_t) * kLog2e : (tt[k] - tm) * c;
      const float lp = e - tlog2;
      const float pk = tt[k] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(e) * tinv;
      if (p.top_lse) mass += pk;
      const int j = k * THREADS + tid;
      if (j < kMaxTop) {
        col[j] = tc[k];
        p_of[j] = pk;
        lp_of[j] = lp;
      }
    }
    if (p.top_lse) mass = sum_all<THREADS>(mass, sh.mass);
    else __syncthreads();
    // A column that occurs more than once: its first entry carries the sum, the others nothing.
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const int j = k * THREADS + tid;
      if (j >= p.top) continue;
      float fix = 0.0f;
      bool lead = tc[k] >= 0;
      for (int o = 0; lead && o < p.top; o += 4) {
        const int4 others = *reinterpret_cast<const int4*>(col + o);  // entries behind the last are -1
        const int oc[4] = {others.x, others.y, others.z, others.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (oc[e] == tc[k]) {
            if (o + e < j) lead = false;
            else fix += p_of[o + e];
          }
      }
      fix_of[j] = lead ? fix : -1.0f;  // sums are not negative (a NaN is kept)
      // into the list of the thread that writes this column (in any order: the list is only
      // walked for values of the entries' own)
      const int v = tc[k] / VEC;
      if (tc[k] >= 0 && v >= v0 && (last_part || v < v1)) {
        const int owner = v >= full ? tc[k] - full * VEC : (v - v0) % THREADS;
        next_of[j] = atomicExch(&head[owner], j);
      }
    }
  }

  // m and s: q_v = exp2((z_v - m) c) / s, log2 s. From a kept pair they are the values the
  // forward had, so that its backward computes what the pass over the row would have: one float
  // for both would lose log s beside a large m (a row of -1e9 has q = 1, not 1 / V, from it).
  float m, s, log2s;
  if (p.lse_given && p.lse_pairs) {
    m = p.lse[2 * r];
    s = p.lse[2 * r + 1];
    log2s = __builtin_amdgcn_logf(s);
  } else if (p.lse_given) {
    m = p.lse[r] * p.temperature;
    s = 1.0f;
    log2s = 0.0f;
  } else if constexpr (SPLIT) {
    // every wave joins the parts in the same order (at most 64, one a lane)
    const int lane = tid & 63;
    Stat st{-INFINITY, 0.0f};
    if (lane < p.splits) st = Stat{p.stats[(r * p.splits + lane) * 2], p.stats[(r * p.splits + lane) * 2 + 1]};
    m = max64(st.m);
    s = sum64(st.s * __builtin_amdgcn_exp2f((st.m - base_of(m)) * c));
    log2s = __builtin_amdgcn_logf(s);
  } else {
    Stat st{-INFINITY, 0.0f};
    // one rescale of the running sum per G vectors
    constexpr int G = NV == 0 ? 1 : 16 / VEC;
    auto take = [&](const u32x4* vec, auto n_tag, int at0) {
      constexpr int N = decltype(n_tag)::value;
      float v[N][VEC], mx = st.m;
#pragma unroll
      for (int g = 0; g < N; ++g) {
        R::unpack(vec[g], v[g]);
        const bool in = NV == 0 || at0 + g < SAFE || (at0 + g) * THREADS + tid < full;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          v[g][e] = in ? v[g][e] : -INFINITY;
          mx = fmaxf(mx, v[g][e]);
        }
      }
      const float at = base_of(mx);
      float s = st.s * __builtin_amdgcn_exp2f((st.m - at) * c);
#pragma unroll
      for (int g = 0; g < N; ++g)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += __builtin_amdgcn_exp2f((v[g][e] - at) * c);
      st = {mx, s};
    };
    if constexpr (NV > 0) {
#pragma unroll
      for (int i = 0; i + G <= NV; i += G) {
        take(row + i, std::integral_constant<int, G>{}, i);
        __builtin_amdgcn_sched_barrier(0);  // a group when it has arrived, not all of them behind the last
      }
      if constexpr (NV % G != 0) take(row + NV / G * G, std::integral_constant<int, NV % G>{}, NV / G * G);
    } else {
      for (int i = tid; i < full; i += THREADS) {
        const u32x4 v = R::load(z + static_cast<int64_t>(i) * VEC);
        take(&v, std::integral_constant<int, 1>{}, 0);
      }
    }
    if (tail < V) st = join(st, Stat{zl, zl == zl ? 1.0f : zl}, c);
    st = join_all<THREADS>(st, c, sh.row);
    m = st.m;
    s = st.s;
    log2s = __builtin_amdgcn_logf(s);
  }
  if (first && p.lse && !p.lse_given) {
    if (p.lse_pairs) {
      p.lse[2 * r] = m;
      p.lse[2 * r + 1] = s;
    } else {
      p.lse[r] = m * p.inv_temperature + log2s * kLn2;
    }
  }

  const float scale = w * up * p.inv_temperature;
  float coef;  // dlogits_v = coef q_v, less the kept entries' part
  if constexpr (LOSS == LOSS_POLICY) {
    const float lp = ((zt - m) * c - log2s) * kLn2;
    const float rho = __builtin_amdgcn_exp2f((lp - old_logp) * kLog2e);
    // 0 where the advantage is, also where rho has left fp32; a NaN stays
    const float kept = adv == 0.0f && rho == rho ? 0.0f : rho * adv;
    const float cut = fminf(fmaxf(rho, 1.0f - p.clip_low), 1.0f + p.clip_high) * adv;
    float loss = kept <= cut ? -kept : -cut;
    float slope = kept <= cut ? -kept : 0.0f;
    if (kept != kept) loss = slope = kept;
    if (p.ref_logp) {
      const float diff = ref_logp - lp, em1 = expm1_f(diff);
      loss += p.kl_coef * (em1 - diff);
      slope -= p.kl_coef * em1;
    }
    if (first) {
      if (p.loss) p.loss[r] = loss * w;
      if (p.logp) p.logp[r] = lp;
    }
    coef = -slope * scale;
  } else {
    coef = mass * scale;
  }
  if constexpr (LOSS == LOSS_DISTILL) {
    // The entries' logits and loss terms: each by the thread that will write its column, so
    // that in place no other thread can have overwritten it (SPLIT: from the workspace).
    __syncthreads();
    auto term = [&](int j, float zj) {
      const float pk = p_of[j];
      p_of[j] = pk != 0.0f ? pk * (lp_of[j] - ((zj - m) * c - log2s)) : 0.0f;
      lp_of[j] = zj;
    };
    if constexpr (SPLIT) {
      for (int j = tid; j < p.top; j += THREADS) term(j, p.own[r * p.top + j]);
      __syncthreads();
    } else {
      for (int j = head[tid]; j >= 0; j = next_of[j]) term(j, R::from(z[col[j]]));
    }
  }
  // The row's loss: the terms in the order of the entries.
  auto distill_row = [&] {
    __syncthreads();
    if (!p.loss || part != 0) return;
    float loss = 0.0f;
    for (int j = tid; j < p.top; j += THREADS) loss += p_of[j];
    loss = sum_all<THREADS>(loss, sh.loss);
    if (tid == 0) p.loss[r] = loss * kLn2 * w;
  };
  if (!d) {
    if constexpr (LOSS == LOSS_DISTILL) distill_row();
    return;
  }

  // In place: every thread has received the target's logit before any writes; a vector is
  // read, here or before, by the thread that writes it.
  if (LOSS == LOSS_POLICY && p.dlogits == p.logits) {
    wait_vmcnt<0>();
    __syncthreads();
  }
  const float cq = coef * (1.0f / s);
  auto give = [&](const u32x4& vec, int i) {
    const int64_t at = static_cast<int64_t>(i) * VEC;
    float v[VEC];
    R::unpack(vec, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = cq * __builtin_amdgcn_exp2f((v[e] - m) * c);
    R::store(d + at, v);
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
    {
      // unpacked anew: the first pass's 8 floats a vector do not stay beside the vector
      asm volatile("" : "+v"(row[i]));
      if (i < SAFE || i * THREADS + tid < full) give(row[i], i * THREADS + tid);
    }
  } else {
    for (int i = v0 + tid; i < v1; i += THREADS) give(R::load(z + static_cast<int64_t>(i) * VEC), i);
  }
  if (tail < V) {
    float v = cq * __builtin_amdgcn_exp2f((zl - m) * c);
    d[tail] = R::to(v);
  }
  if constexpr (LOSS == LOSS_POLICY) {
    // The target's column again, by the thread that wrote it above: its stores to one address
    // stay in order (a comparison per element instead took 2 of about 17 instructions).
    const int v = static_cast<int>(target) / VEC;
    const int owner = v >= full ? static_cast<int>(target) - full * VEC : (v - v0) % THREADS;
    if (v >= v0 && (last_part || v < v1) && tid == owner)
      d[target] = R::to(cq * __builtin_amdgcn_exp2f((zt - m) * c) - coef);
  }
  if constexpr (LOSS == LOSS_DISTILL) {
    // The kept columns again, with the teacher's part, by the thread that wrote them above:
    // its stores to one address stay in order. (Any other thread would have to wait for all
    // of the row's stores: 2048 rows of 152064 took 299 us that way.)
    for (int j = head[tid]; j >= 0; j = next_of[j])
      if (!(fix_of[j] < 0.0f))
        d[col[j]] = R::to(cq * __builtin_amdgcn_exp2f((lp_of[j] - m) * c) - fix_of[j] * scale);
    distill_row();
  }
}

template <typename E, int LOSS, int THREADS, int NV, int SAFE = 0>
hipError_t launch_as(const LossParams& p, hipStream_t st) {
  hipLaunchKernelGGL((loss_kernel<E, LOSS, THREADS, NV, SAFE>), dim3(static_cast<unsigned int>(p.rows)), dim3(THREADS), 0, st, p);
  return hipGetLastError();
}

// The smallest form that holds the row; a row past the largest is read twice. 19 vectors a thread are
// not the registers' limit (100 to 106 of 128; 24 would fit without spills): longer forms have not
// been measured.
template <typename E, int LOSS>
hipError_t launch(const LossParams& p, hipStream_t st) {
  if (p.splits > 1) {
    const dim3 grid(static_cast<unsigned int>(p.rows * p.splits));
    hipLaunchKernelGGL((loss_parts<E, LOSS, 256>), grid, dim3(256), 0, st, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((loss_kernel<E, LOSS, 256, 0, 0, true>), grid, dim3(256), 0, st, p);
    return hipGetLastError();
  }
  const int vectors = p.vocab / Row<E>::VEC;
  // without a gradient and with the normaliser given no row is read
  if (vectors < 1 || (!p.dlogits && p.lse_given)) return launch_as<E, LOSS, 256, 0>(p, st);
  if (vectors <= 256 * 4) return launch_as<E, LOSS, 256, 4>(p, st);
  if (vectors <= 256 * 8) return launch_as<E, LOSS, 256, 8, 4>(p, st);
  if (vectors <= 256 * 16) return launch_as<E, LOSS, 256, 16, 8>(p, st);
  if (vectors <= 512 * 16) return launch_as<E, LOSS, 512, 16, 8>(p, st);
  if (vectors <= 1024 * 12) return launch_as<E, LOSS, 1024, 12, 8>(p, st);
  if (vectors <= 1024 * 16) return launch_as<E, LOSS, 1024, 16, 12>(p, st);
  if (vectors <= 1024 * 19) return launch_as<E, LOSS, 1024, 19, 16>(p, st);
  return launch_as<E, LOSS, 1024, 0>(p, st);
}

}  // namespace

hipError_t launch_loss(int loss, bool bf16, const LossParams& p, hipStream_t st) {
  if (p.rows <= 0) return hipSuccess;
  if (loss == LOSS_POLICY)
    return bf16 ? launch<unsigned short, LOSS_POLICY>(p, st) : launch<float, LOSS_POLICY>(p, st);
  return bf16 ? launch<unsigned short, LOSS_DISTILL>(p, st) : launch<float, LOSS_DISTILL>(p, st);
}

}  // namespace muon
