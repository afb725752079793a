// Tokens sorted by expert and back.
//
// The plan: a stable counting sort of the choices (token t's j-th expert, f = t top + j) by
// expert. order[p] = f of the p-th row, slots[f] = p, offsets[e] = first row of expert e. A
// choice outside [0, experts) is dropped: slots -1; the places behind the last row have order -1.
//
// The rows: xs[slots[f]] = x[t]; y[t] = sum_j w[f] ys[slots[f]] and its gradients. All bound by
// HBM: each row is read or written once, the shared one of a token once for all its choices.
#include "layer.hpp"
#include "mfma_util.hpp"

namespace muon {
namespace {

typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

__device__ __forceinline__ unsigned short to_bf16(float f) {
  return __builtin_bit_cast(unsigned short, static_cast<__bf16>(f));
}

__device__ __forceinline__ int expert_of(const PlanParams& p, int64_t f) {
  if (p.ids64) {
    const int64_t e = static_cast<const int64_t*>(p.ids)[f];
    return e >= 0 && e < p.experts ? static_cast<int>(e) : p.experts;
  }
  const int e = static_cast<const int32_t*>(p.ids)[f];
  return e >= 0 && e < p.experts ? e : p.experts;
}

// The choices of a block, and of one of its four waves: contiguous runs of whole waves.
struct Run {
  int64_t begin, end;
};
__device__ __forceinline__ Run run_of(int64_t n, int blocks, int block, int wave) {
  const int64_t each = (n + 4 * 64 * static_cast<int64_t>(blocks) - 1) / (4 * 64 * static_cast<int64_t>(blocks)) * 64;
  const int64_t b = (static_cast<int64_t>(block) * 4 + wave) * each;
  return {min(b, n), min(b + each, n)};
}

__global__ __launch_bounds__(256) void plan_count(const PlanParams p) {
  __shared__ int count[kMaxExperts + 1];
  for (int e = threadIdx.x; e <= p.experts; e += 256) count[e] = 0;
  __syncthreads();
  const Run r = run_of(p.n, p.blocks, blockIdx.x, threadIdx.x >> 6);
  for (int64_t f = r.begin + (threadIdx.x & 63); f < r.end; f += 64) atomicAdd(&count[expert_of(p, f)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.experts; e += 256) p.counts[static_cast<int64_t>(blockIdx.x) * (p.experts + 1) + e] = count[e];
}

// Places. The counters are sums of integers: the order of the LDS atomics changes nothing.
__global__ __launch_bounds__(256) void plan_place(const PlanParams p) {
  constexpr int N = kMaxExperts + 1, PER = (N + 255) / 256;
  __shared__ int mine[4][N];      // a wave's choices by expert, then its next place
  __shared__ int before[N], total[N];
  __shared__ int wave_sum[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, buckets = p.experts + 1;
  for (int e = tid; e < buckets; e += 256) {
    before[e] = total[e] = 0;
    for (int w = 0; w < 4; ++w) mine[w][e] = 0;
  }
  __syncthreads();
  const Run r = run_of(p.n, p.blocks, blockIdx.x, wave);
  for (int64_t f = r.begin + lane; f < r.end; f += 64) atomicAdd(&mine[wave][expert_of(p, f)], 1);
  if (p.blocks > 1) {
    // the blocks' counts: threads side by side over experts, the rest over blocks
    int wide = 1;
    while (wide < buckets && wide < 256) wide *= 2;
    const int parts = 256 / wide, part = tid / wide;
    for (int e = tid % wide; e < buckets; e += wide) {
      int all = 0, less = 0;
#pragma unroll 16
      for (int b = part; b < p.blocks; b += parts) {
        const int c = p.counts[static_cast<int64_t>(b) * buckets + e];
        all += c;
        less += b < static_cast<int>(blockIdx.x) ? c : 0;
      }
      atomicAdd(&total[e], all);
      atomicAdd(&before[e], less);
    }
  }
  __syncthreads();
  if (p.blocks == 1) {
    for (int e = tid; e < buckets; e += 256) total[e] = mine[0][e] + mine[1][e] + mine[2][e] + mine[3][e];
    __syncthreads();
  }
  // exclusive sums over the buckets: PER neighbours a thread, threads by lane shifts, waves by LDS
  int own[PER], sum = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int e = tid * PER + k;
    own[k] = sum;
    sum += e < buckets ? total[e] : 0;
  }
  int upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int other = __shfl_up(upto, d);
    if (lane >= d) upto += other;
  }
  if (lane == 63) wave_sum[wave] = upto;
  __syncthreads();
  int start = upto - sum;
  for (int w = 0; w < wave; ++w) start += wave_sum[w];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int e = tid * PER + k;
    if (e < buckets) {
      const int first = start + own[k];
      if (blockIdx.x == 0) p.offsets[e] = first;
      int at = first + before[e];
      for (int w = 0; w < 4; ++w) {
        const int c = mine[w][e];
        mine[w][e] = at;
        at += c;
      }
    }
  }
  __syncthreads();
  // a wave's choices in order, 64 at a time: a lane's place is its expert's next one plus the
  // number of lanes below that chose the same
  volatile int* next = mine[wave];
  for (int64_t f0 = r.begin; f0 < r.end; f0 += 64) {
    const int64_t f = f0 + lane;
    const bool there = f < r.end;
    const int e = there ? expert_of(p, f) : N;
    unsigned long long same = ~0ull;
#pragma unroll
    for (int b = 0; b < 11; ++b) {
      const unsigned long long ones = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? ones : ~ones;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (there) {
      const int at = next[e] + rank;
      if (rank == __popcll(same) - 1) next[e] = at + 1;
      p.order[at] = e < p.experts ? static_cast<int>(f) : -1;
      p.slots[f] = e < p.experts ? at : -1;
    }
  }
}

template <bool F32>
struct Row {
  static constexpr int ES = F32 ? 4 : 2, VEC = 16 / ES;
  // elements c .. c + VEC - 1 of a row of `dim`, zeros behind it
  static __device__ __forceinline__ u32x4 load(const char* row, int c, int dim) {
    if (c + VEC <= dim) {
      if constexpr (F32) return *reinterpret_cast<const u32x4_a4*>(row + c * ES);
      else return *reinterpret_cast<const u32x4_a2*>(row + c * ES);
    }
    u32x4 v{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (c + e < dim) {
        if constexpr (F32) v[e] = *reinterpret_cast<const unsigned int*>(row + (c + e) * 4);
        else v[e / 2] |= static_cast<unsigned int>(*reinterpret_cast<const unsigned short*>(row + (c + e) * 2)) << (16 * (e & 1));
      }
    return v;
  }
  // Whole pieces of a row that is read once: past the caches, where they would push out what others read again.
  static __device__ __forceinline__ u32x4 load_once(const char* row, int c) {
    if constexpr (F32) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_a4*>(row + c * ES));
    else return __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(row + c * ES));
  }
  static __device__ __forceinline__ void store(char* row, int c, int dim, const u32x4& v) {
    if (c + VEC <= dim) {
      if constexpr (F32) *reinterpret_cast<u32x4_a4*>(row + c * ES) = v;
      else *reinterpret_cast<u32x4_a2*>(row + c * ES) = v;
      return;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (c + e < dim) {
        if constexpr (F32) *reinterpret_cast<unsigned int*>(row + (c + e) * 4) = v[e];
        else *reinterpret_cast<unsigned short*>(row + (c + e) * 2) = static_cast<unsigned short>(v[e / 2] >> (16 * (e & 1)));
      }
  }
  static __device__ __forceinline__ float get(const u32x4& v, int e) {
    if constexpr (F32) return __uint_as_float(v[e]);
    else return __uint_as_float(e & 1 ? v[e / 2] & 0xFFFF0000u : v[e / 2] << 16);
  }
  static __device__ __forceinline__ u32x4 put(const float (&f)[VEC]) {
    u32x4 v;
    if constexpr (F32) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(f[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = to_bf16(f[2 * e]) | (static_cast<unsigned int>(to_bf16(f[2 * e + 1])) << 16);
    }
    return v;
  }
};

// The number of threads that share a row: a power of two, one 16-byte piece each where 256 reach.
__device__ __forceinline__ int pieces_of(int dim, int vec, int most) {
  int w = 1;
  while (w < most && w * vec < dim) w *= 2;
  return w;
}

// xs[slots[f]] = x[t]: a token's row is read once and written for each choice; a row behind the
// last expert's is written as zeros by the choice of its number. The sizes below: 52 to 58 us, 5.2 to 5.8 TB/s.
template <bool F32>
__global__ __launch_bounds__(256) void rows_dispatch(const RowsParams p) {
  using R = Row<F32>;
  const int w = pieces_of(p.dim, R::VEC, 256);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (256 / w) + threadIdx.x / w;
  if (t >= p.tokens) return;
  const int64_t n = p.tokens * p.top;
  const int total = p.offsets[p.experts];
  const char* row = static_cast<const char*>(p.in) + t * p.ld_in * R::ES;
  char* out = static_cast<char*>(p.out);
  for (int c = threadIdx.x % w * R::VEC; c < p.dim; c += w * R::VEC) {
    const u32x4 v = R::load(row, c, p.dim);
    for (int j = 0; j < p.top; ++j) {
      const int64_t f = t * p.top + j;
      const int64_t s = p.slots[f];
      if (s >= 0 && s < n) R::store(out + s * p.ld_out * R::ES, c, p.dim, v);
      if (f >= total) R::store(out + f * p.ld_out * R::ES, c, p.dim, u32x4{0, 0, 0, 0});
    }
  }
}

// y[t] = sum_j w[f] ys[slots[f]] in the order of j, in fp32, rounded once. 8192 tokens x 8 choices of 2048 bf16
// columns: 59 us, 5.1 TB/s (86 us with loads through the caches, 65 us with eight of them in flight); 3001 x 3 of 413
// fp32, which the caches hold: 6.4 us (8.8 us past them).
template <bool F32>
__global__ __launch_bounds__(256) void rows_combine(const RowsParams p) {
  using R = Row<F32>;
  constexpr int U = 4;
  const int w = pieces_of(p.dim, R::VEC, 256);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (256 / w) + threadIdx.x / w;
  if (t >= p.tokens) return;
  const int64_t n = p.tokens * p.top;
  const char* in = static_cast<const char*>(p.in);
  for (int c = threadIdx.x % w * R::VEC; c < p.dim; c += w * R::VEC) {
    float sum[R::VEC] = {};
    auto add = [&](auto load) {
      for (int j0 = 0; j0 < p.top; j0 += U) {
        u32x4 v[U];
        float a[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          v[j] = u32x4{0, 0, 0, 0};
          a[j] = 0.0f;
          if (j0 + j < p.top) {
            const int64_t f = t * p.top + j0 + j;
            const int64_t s = p.slots[f];
            if (s >= 0 && s < n) {
              a[j] = p.weights ? p.weights[f] : 1.0f;
              v[j] = load(in + s * p.ld_in * R::ES);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
          for (int e = 0; e < R::VEC; ++e) sum[e] += a[j] * R::get(v[j], e);
      }
    };
    if (p.once && c + R::VEC <= p.dim) add([&](const char* row) { return R::load_once(row, c); });
    else add([&](const char* row) { return R::load(row, c, p.dim); });
    R::store(static_cast<char*>(p.out) + t * p.ld_out * R::ES, c, p.dim, R::put(sum));
  }
}

// A choice's gradients: dys[slots[f]] = w[f] dy[t], dw[f] = dy[t] . ys[slots[f]]. A quarter, half
// or whole wave a choice; the choices of a token are neighbours, so its dy comes from HBM once. The same sizes:
// 118 us, 4.8 TB/s.
template <bool F32>
__global__ __launch_bounds__(256) void rows_combine_grad(const RowsParams p) {
  using R = Row<F32>;
  const int w = pieces_of(p.dim, R::VEC, 64);
  const int64_t n = p.tokens * p.top;
  const int64_t f = static_cast<int64_t>(blockIdx.x) * (256 / w) + threadIdx.x / w;
  if (f >= n) return;
  const int total = p.offsets[p.experts];
  char* out = static_cast<char*>(p.out);
  const int c0 = threadIdx.x % w * R::VEC, step = w * R::VEC;
  if (out && f >= total)
    for (int c = c0; c < p.dim; c += step) R::store(out + f * p.ld_out * R::ES, c, p.dim, u32x4{0, 0, 0, 0});
  const int64_t s = p.slots[f];
  float dot = 0.0f;
  if (s >= 0 && s < n) {
    const char* dy = static_cast<const char*>(p.in) + f / p.top * p.ld_in * R::ES;
    const char* ys = static_cast<const char*>(p.in2) + s * p.ld_in2 * R::ES;
    const float a = p.weights ? p.weights[f] : 1.0f;
#pragma unroll 4
    for (int c = c0; c < p.dim; c += step) {
      const u32x4 g = R::load(dy, c, p.dim);
      if (p.dw) {
        const u32x4 y = p.once && c + R::VEC <= p.dim ? R::load_once(ys, c) : R::load(ys, c, p.dim);
#pragma unroll
        for (int e = 0; e < R::VEC; ++e) dot += R::get(g, e) * R::get(y, e);
      }
      if (out) {
        float v[R::VEC];
#pragma unroll
        for (int e = 0; e < R::VEC; ++e) v[e] = a * R::get(g, e);
        R::store(out + s * p.ld_out * R::ES, c, p.dim, R::put(v));
      }
    }
  }
  if (p.dw) {
    for (int d = w / 2; d > 0; d /= 2) dot += __shfl_xor(dot, d);
    if (threadIdx.x % w == 0) p.dw[f] = dot;
  }
}

int pieces(int dim, int vec, int most) {
  int w = 1;
  while (w < most && w * vec < dim) w *= 2;
  return w;
}

template <bool F32>
hipError_t rows(RowsOp op, const RowsParams& p, hipStream_t st) {
  const int each = 256 / pieces(p.dim, Row<F32>::VEC, op == ROWS_COMBINE_GRAD ? 64 : 256);
  const int64_t n = op == ROWS_COMBINE_GRAD ? p.tokens * p.top : p.tokens;
  const dim3 grid(static_cast<unsigned>((n + each - 1) / each));
  if (op == ROWS_DISPATCH) rows_dispatch<F32><<<grid, 256, 0, st>>>(p);
  else if (op == ROWS_COMBINE) rows_combine<F32><<<grid, 256, 0, st>>>(p);
  else rows_combine_grad<F32><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_plan(const PlanParams& p, hipStream_t st) {
  if (p.blocks > 1) {
    plan_count<<<p.blocks, 256, 0, st>>>(p);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  plan_place<<<p.blocks, 256, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_expert_rows(RowsOp op, bool f32, const RowsParams& p, hipStream_t st) {
  return f32 ? rows<true>(op, p, st) : rows<false>(op, p, st);
}

}  // namespace muon
