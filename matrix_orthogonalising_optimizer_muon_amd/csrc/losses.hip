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
// exp((z - m)) over its columns (one rescale per 16-byte vector), joined in a fixed order;
// the second writes the gradient. All of it in fp32; exp((z - m) c) is formed from the
// difference, so that rows of the type's lowest values stay exact, and q = e / s.
#include <type_traits>

#include "internal.hpp"
#include "mfma_util.hpp"

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

// Joined over the workgroup, in a fixed order; every thread receives the result.
template <int THREADS>
__device__ __forceinline__ Stat join_all(Stat v, float c, Stat* lds) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = join(v, Stat{__shfl_xor(v.m, d), __shfl_xor(v.s, d)}, c);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) v = join(v, lds[w], c);
  __syncthreads();
  return v;
}
template <int THREADS>
__device__ __forceinline__ float sum_all(float v, float* lds) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) v += lds[w];
  __syncthreads();
  return v;
}

// exp(d) - 1 without cancellation: the series for small d (next term d^6 / 720 below
// 2^-24 of the result for |d| < 0.1), else the exponential.
__device__ __forceinline__ float expm1_f(float d) {
  if (fabsf(d) < 0.1f)
    return d * (1.0f + d * (0.5f + d * (0.16666667f + d * (0.041666668f + d * 0.0083333338f))));
  return __builtin_amdgcn_exp2f(d * kLog2e) - 1.0f;
}

struct Shared {
  Stat stat[16];
  float sum[16];
};

// NV > 0: the row stays in registers between the passes, NV 16-byte vectors a thread, and is
// read once. NV == 0: the second pass reads it again (rows too long to hold).
template <typename E, int LOSS, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void loss_kernel(const LossParams p) {
  using R = Row<E>;
  constexpr int VEC = R::VEC;
  constexpr int KT = LOSS == LOSS_DISTILL ? (kMaxTop + THREADS - 1) / THREADS : 1;  // kept entries a thread takes
  __shared__ Shared sh;
  __shared__ __attribute__((aligned(16))) int col[LOSS == LOSS_DISTILL ? kMaxTop : 4];   // the kept entries' columns, -1: absent
  __shared__ float mass_of[LOSS == LOSS_DISTILL ? kMaxTop : 1];                          // and teacher probabilities

  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  const int V = p.vocab;
  const E* z = static_cast<const E*>(p.logits) + r * p.ld;
  E* d = p.dlogits ? static_cast<E*>(p.dlogits) + r * p.ld_d : nullptr;
  const float c = p.inv_temperature * kLog2e;
  const float w = p.weights ? p.weights[r] : 1.0f;
  const int full = V / VEC;                 // whole vectors
  const int tail = full * VEC + tid;        // the column behind them that this thread takes
  int64_t target = 0;
  if constexpr (LOSS == LOSS_POLICY) target = p.targets[r];

  // A row that takes no part (weight 0, or no target) is not read.
  if (w == 0.0f || target < 0 || target >= V) {
    if (tid == 0) {
      if (p.loss) p.loss[r] = 0.0f;
      if (!p.lse_given && p.lse) p.lse[r] = 0.0f;
      if (LOSS == LOSS_POLICY && p.logp) p.logp[r] = 0.0f;
    }
    if (d) {
      float zero[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) zero[e] = 0.0f;
      for (int i = tid; i < full; i += THREADS) R::store(d + static_cast<int64_t>(i) * VEC, zero);
      if (tail < V) d[tail] = R::to(0.0f);
    }
    return;
  }

  // The teacher's entries first, then the row: loads return in order, so the columns are
  // known (and their logits requested) while the row is still on its way.
  float tt[KT], tz[KT];
  int tc[KT];
  if constexpr (LOSS == LOSS_DISTILL) {
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const int j = k * THREADS + tid;
      tc[k] = -1;
      tt[k] = -INFINITY;
      tz[k] = 0.0f;
      if (j < p.top) {
        const int64_t id = p.ids64 ? static_cast<const int64_t*>(p.ids)[r * p.ld_ids + j]
                                   : static_cast<const int32_t*>(p.ids)[r * p.ld_ids + j];
        const int64_t at = r * p.ld_top + j;
        const float t = p.top_bf16 ? Row<unsigned short>::from(static_cast<const unsigned short*>(p.top_logits)[at])
                                   : static_cast<const float*>(p.top_logits)[at];
        if (id >= 0 && id < V) {
          tc[k] = static_cast<int>(id);
          tt[k] = t;
        }
      }
    }
  }
  u32x4 row[NV > 0 ? NV : 1];
  if constexpr (NV > 0) {
    // past the row's last vector a thread loads that one again and leaves it out below
    if (d || !p.lse_given)
#pragma unroll
    for (int i = 0; i < NV; ++i) row[i] = R::load(z + static_cast<int64_t>(min(i * THREADS + tid, full - 1)) * VEC);
  }
  const float zl = tail < V ? R::from(z[tail]) : 0.0f;
  float zt = 0.0f;
  if constexpr (LOSS == LOSS_POLICY) {
    zt = R::from(z[target]);
  } else {
#pragma unroll
    for (int k = 0; k < KT; ++k)
      if (tc[k] >= 0) tz[k] = R::from(z[tc[k]]);
  }

  // m and s: q_v = exp2((z_v - m) c) / s, log2 of the normaliser (m c + log2 s).
  float m, inv_s, log2s;
  if (p.lse_given) {
    m = 0.0f;
    log2s = p.lse[r] * kLog2e;
    inv_s = 1.0f;
  } else {
    Stat st{-INFINITY, 0.0f};
    // one rescale of the running sum per G vectors
    constexpr int G = NV == 0 ? 1 : 16 / VEC;
    auto take = [&](const u32x4* vec, auto n_tag, int first) {
      constexpr int N = decltype(n_tag)::value;
      float v[N][VEC], mx = st.m;
#pragma unroll
      for (int g = 0; g < N; ++g) {
        R::unpack(vec[g], v[g]);
        const bool in = NV == 0 || (first + g) * THREADS + tid < full;
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
      for (int i = 0; i + G <= NV; i += G) take(row + i, std::integral_constant<int, G>{}, i);
      if constexpr (NV % G != 0) take(row + NV / G * G, std::integral_constant<int, NV % G>{}, NV / G * G);
    } else {
      for (int i = tid; i < full; i += THREADS) {
        const u32x4 v = R::load(z + static_cast<int64_t>(i) * VEC);
        take(&v, std::integral_constant<int, 1>{}, 0);
      }
    }
    if (tail < V) st = join(st, Stat{zl, zl == zl ? 1.0f : zl}, c);
    st = join_all<THREADS>(st, c, sh.stat);
    m = st.m;
    log2s = __builtin_amdgcn_logf(st.s);
    inv_s = 1.0f / st.s;
    if (tid == 0 && p.lse) p.lse[r] = m * p.inv_temperature + log2s * kLn2;
  }

  const float up = p.grad_rows ? p.grad_rows[r] : 1.0f;
  const float scale = w * up * p.inv_temperature;
  float coef;  // dlogits_v = coef q_v, less the kept entries' part
  float fix[KT];
  if constexpr (LOSS == LOSS_POLICY) {
    const float lp = ((zt - m) * c - log2s) * kLn2;
    const float adv = p.advantages[r];
    const float rho = __builtin_amdgcn_exp2f((lp - p.old_logp[r]) * kLog2e);
    const float kept = rho * adv;
    const float cut = fminf(fmaxf(rho, 1.0f - p.clip_low), 1.0f + p.clip_high) * adv;
    float loss = kept <= cut ? -kept : -cut;
    float slope = kept <= cut ? -kept : 0.0f;
    if (kept != kept) loss = slope = kept;
    if (p.ref_logp) {
      const float diff = p.ref_logp[r] - lp, em1 = expm1_f(diff);
      loss += p.kl_coef * (em1 - diff);
      slope -= p.kl_coef * em1;
    }
    if (tid == 0) {
      if (p.loss) p.loss[r] = loss * w;
      if (p.logp) p.logp[r] = lp;
    }
    coef = -slope * scale;
  } else {
    // Teacher: p_j = exp((t_j - tm) c - log2 of the normaliser)
    float tm, tlog2;
    if (p.top_lse) {
      tm = 0.0f;
      tlog2 = p.top_lse[r] * kLog2e;
    } else {
      Stat st{-INFINITY, 0.0f};
#pragma unroll
      for (int k = 0; k < KT; ++k) st = join(st, Stat{tt[k], tt[k] == -INFINITY ? 0.0f : 1.0f}, c);
      st = join_all<THREADS>(st, c, sh.stat);
      tm = base_of(st.m);
      tlog2 = __builtin_amdgcn_logf(st.s);
    }
    float mass = 0.0f, loss = 0.0f, pj[KT];
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const float lpj = (tt[k] - tm) * c - tlog2;        // log2 p_j
      pj[k] = tt[k] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(lpj);
      mass += pj[k];
      if (pj[k] != 0.0f) loss += pj[k] * (lpj - ((tz[k] - m) * c - log2s));
      const int j = k * THREADS + tid;
      if (j < kMaxTop) {
        col[j] = tc[k];
        mass_of[j] = pj[k];
      }
    }
    mass = sum_all<THREADS>(mass, sh.sum);
    loss = sum_all<THREADS>(loss, sh.sum);
    if (tid == 0 && p.loss) p.loss[r] = loss * kLn2 * w;
    coef = mass * scale;
    // A column that occurs more than once: its first entry carries the sum, the others nothing.
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      fix[k] = 0.0f;
      const int j = k * THREADS + tid;
      if (tc[k] < 0) continue;
      for (int o = 0; o < p.top; o += 4) {
        const int4 others = *reinterpret_cast<const int4*>(col + o);  // entries behind the last are -1
        const int oc[4] = {others.x, others.y, others.z, others.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (oc[e] == tc[k]) {
            if (o + e < j) tc[k] = -1;
            else fix[k] += mass_of[o + e];
          }
        if (tc[k] < 0) break;
      }
      fix[k] *= scale;
    }
  }
  if (!d) return;

  // In place: every thread has read the row's scalars by now (and, with the row in
  // registers, the row); with a second pass a thread reads a vector before it writes it.
  __syncthreads();
  const float cq = coef * inv_s;
  const float shift = p.lse_given ? log2s : 0.0f;
  auto give = [&](const u32x4& vec, int i) {
    const int64_t at = static_cast<int64_t>(i) * VEC;
    float v[VEC];
    R::unpack(vec, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = cq * __builtin_amdgcn_exp2f((v[e] - m) * c - shift);
    if constexpr (LOSS == LOSS_POLICY) {
      const int off = static_cast<int>(target) - i * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = off == e ? v[e] - coef : v[e];
    }
    R::store(d + at, v);
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * THREADS + tid < full) give(row[i], i * THREADS + tid);
  } else {
    for (int i = tid; i < full; i += THREADS) give(R::load(z + static_cast<int64_t>(i) * VEC), i);
  }
  if (tail < V) {
    float v = cq * __builtin_amdgcn_exp2f((zl - m) * c - shift);
    if (LOSS == LOSS_POLICY && tail == target) v -= coef;
    d[tail] = R::to(v);
  }
  if constexpr (LOSS == LOSS_DISTILL) {
    // The kept columns again, with the teacher's part. The row's stores have reached this
    // XCD's L2 before any of these is issued (a wait for them and a barrier; a device-wide
    // fence would write the L2 back: 1685 us against 339 us for 2048 rows of 152064).
    wait_vmcnt<0>();
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KT; ++k)
      if (tc[k] >= 0) d[tc[k]] = R::to(cq * __builtin_amdgcn_exp2f((tz[k] - m) * c - shift) - fix[k]);
  }
}

template <typename E, int LOSS, int THREADS, int NV>
hipError_t launch_as(const LossParams& p, hipStream_t st) {
  hipLaunchKernelGGL((loss_kernel<E, LOSS, THREADS, NV>), dim3(static_cast<unsigned int>(p.rows)), dim3(THREADS), 0, st, p);
  return hipGetLastError();
}

// The smallest form that holds the row; a row past the largest is read twice.
template <typename E, int LOSS>
hipError_t launch(const LossParams& p, hipStream_t st) {
  const int vectors = p.vocab / Row<E>::VEC;
  if (vectors < 1) return launch_as<E, LOSS, 256, 0>(p, st);
  if (vectors <= 256 * 4) return launch_as<E, LOSS, 256, 4>(p, st);
  if (vectors <= 256 * 8) return launch_as<E, LOSS, 256, 8>(p, st);
  if (vectors <= 256 * 16) return launch_as<E, LOSS, 256, 16>(p, st);
  if (vectors <= 512 * 16) return launch_as<E, LOSS, 512, 16>(p, st);
  if (vectors <= 1024 * 12) return launch_as<E, LOSS, 1024, 12>(p, st);
  if (vectors <= 1024 * 16) return launch_as<E, LOSS, 1024, 16>(p, st);
  if (vectors <= 1024 * 19) return launch_as<E, LOSS, 1024, 19>(p, st);
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
