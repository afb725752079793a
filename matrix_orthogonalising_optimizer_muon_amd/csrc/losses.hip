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

template <typename E, int LOSS, int THREADS>
__global__ __launch_bounds__(THREADS) void loss_kernel(const LossParams p) {
  using R = Row<E>;
  constexpr int VEC = R::VEC;
  __shared__ Shared sh;
  __shared__ float tz[LOSS == LOSS_DISTILL ? kMaxTop : 1];   // the kept entries' logits
  __shared__ float tp[LOSS == LOSS_DISTILL ? kMaxTop : 1];   // their teacher probabilities
  __shared__ int tid_of[LOSS == LOSS_DISTILL ? kMaxTop : 1]; // their columns, -1: absent

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

  // The scalars of the row that lie in the logits, before a gradient may overwrite them.
  float zt = 0.0f;
  if constexpr (LOSS == LOSS_POLICY) {
    zt = R::from(z[target]);
  } else {
    for (int j = tid; j < p.top; j += THREADS) {
      const int64_t id = p.ids64 ? static_cast<const int64_t*>(p.ids)[r * p.ld_ids + j]
                                 : static_cast<const int32_t*>(p.ids)[r * p.ld_ids + j];
      const bool in = id >= 0 && id < V;
      tid_of[j] = in ? static_cast<int>(id) : -1;
      tz[j] = in ? R::from(z[id]) : 0.0f;
      const int64_t at = r * p.ld_top + j;
      const float t = p.top_bf16 ? Row<unsigned short>::from(static_cast<const unsigned short*>(p.top_logits)[at])
                                 : static_cast<const float*>(p.top_logits)[at];
      tp[j] = in ? t : -INFINITY;
    }
  }

  // m and s: q_v = exp2((z_v - m) c) / s, log2 of the normaliser (m c + log2 s).
  float m, inv_s, log2s;
  if (p.lse_given) {
    m = 0.0f;
    log2s = p.lse[r] * kLog2e;
    inv_s = 1.0f;
  } else {
    Stat st{-INFINITY, 0.0f};
    for (int i = tid; i < full; i += THREADS) {
      float v[VEC];
      R::unpack(R::load(z + static_cast<int64_t>(i) * VEC), v);
      float mx = st.m;
#pragma unroll
      for (int e = 0; e < VEC; ++e) mx = fmaxf(mx, v[e]);
      const float at = base_of(mx);
      float s = st.s * __builtin_amdgcn_exp2f((st.m - at) * c);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += __builtin_amdgcn_exp2f((v[e] - at) * c);
      st = {mx, s};
    }
    if (tail < V) {
      const float v = R::from(z[tail]);
      st = join(st, Stat{v, v == v ? 1.0f : v}, c);
    }
    st = join_all<THREADS>(st, c, sh.stat);
    m = st.m;
    log2s = __builtin_amdgcn_logf(st.s);
    inv_s = 1.0f / st.s;
    if (tid == 0 && p.lse) p.lse[r] = m * p.inv_temperature + log2s * kLn2;
  }

  const float up = p.grad_rows ? p.grad_rows[r] : 1.0f;
  const float scale = w * up * p.inv_temperature;
  float coef;  // dlogits_v = coef q_v, less the kept entries' part
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
    __syncthreads();
    float tm, tlog2;
    if (p.top_lse) {
      tm = 0.0f;
      tlog2 = p.top_lse[r] * kLog2e;
    } else {
      Stat st{-INFINITY, 0.0f};
      for (int j = tid; j < p.top; j += THREADS) st = join(st, Stat{tp[j], tp[j] == -INFINITY ? 0.0f : 1.0f}, c);
      st = join_all<THREADS>(st, c, sh.stat);
      tm = base_of(st.m);
      tlog2 = __builtin_amdgcn_logf(st.s);
    }
    float mass = 0.0f, loss = 0.0f;
    for (int j = tid; j < p.top; j += THREADS) {
      const float lpj = (tp[j] - tm) * c - tlog2;        // log2 p_j
      const float pj = tp[j] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(lpj);
      mass += pj;
      if (pj != 0.0f) loss += pj * (lpj - ((tz[j] - m) * c - log2s));
      tp[j] = pj;
    }
    mass = sum_all<THREADS>(mass, sh.sum);
    loss = sum_all<THREADS>(loss, sh.sum);
    if (tid == 0 && p.loss) p.loss[r] = loss * kLn2 * w;
    coef = mass * scale;
  }
  if (!d) return;

  // In place: every thread's logits of the row's scalars are read by now.
  __syncthreads();
  const float cq = coef * inv_s;
  const float shift = p.lse_given ? log2s : 0.0f;
  for (int i = tid; i < full; i += THREADS) {
    const int64_t at = static_cast<int64_t>(i) * VEC;
    float v[VEC];
    R::unpack(R::load(z + at), v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = cq * __builtin_amdgcn_exp2f((v[e] - m) * c - shift);
    if constexpr (LOSS == LOSS_POLICY) {
      const int64_t off = target - at;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = off == e ? v[e] - coef : v[e];
    }
    R::store(d + at, v);
  }
  if (tail < V) {
    float v = cq * __builtin_amdgcn_exp2f((R::from(z[tail]) - m) * c - shift);
    if (LOSS == LOSS_POLICY && tail == target) v -= coef;
    d[tail] = R::to(v);
  }
  if constexpr (LOSS == LOSS_DISTILL) {
    // The kept columns again, with the teacher's part; the first entry of a column that
    // occurs more than once writes the sum. The row's stores have reached this XCD's L2
    // before any of these is issued (a wait for them and a barrier; a device-wide fence
    // would write the L2 back: 1685 us against 339 us for 2048 rows of 152064).
    wait_vmcnt<0>();
    __syncthreads();
    for (int j = tid; j < p.top; j += THREADS) {
      const int id = tid_of[j];
      if (id < 0) continue;
      float pj = 0.0f;
      bool first = true;
      for (int k = 0; k < p.top; ++k) {
        if (tid_of[k] != id) continue;
        if (k < j) { first = false; break; }
        pj += tp[k];
      }
      if (first)
        d[id] = R::to(cq * __builtin_amdgcn_exp2f((tz[j] - m) * c - shift) - pj * scale);
    }
  }
}

template <typename E, int LOSS>
hipError_t launch(const LossParams& p, hipStream_t st) {
  const dim3 grid(static_cast<unsigned int>(p.rows));
  if (p.vocab <= 16384)
    hipLaunchKernelGGL((loss_kernel<E, LOSS, 256>), grid, dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((loss_kernel<E, LOSS, 1024>), grid, dim3(1024), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_loss(int loss, bool bf16, const LossParams& p, hipStream_t st) {
  if (p.rows <= 0) return hipSuccess;
  if (loss == LOSS_POLICY)
    return bf16 ? launch<unsigned short, LOSS_POLICY>(p, st) : launch<float, LOSS_POLICY>(p, st);
  return bf16 ? launch<unsigned short, LOSS_DISTILL>(p, st) : launch<float, LOSS_DISTILL>(p, st);
}

}  // namespace muon
