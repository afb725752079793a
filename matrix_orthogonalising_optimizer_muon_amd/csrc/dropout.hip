// Dropout from a counter: out = residual + keep x / (1 - p), the mask never stored.
//
// The random bits are Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011): counter (i / 8, offset), key seed, i the element's number in the
// rows x cols array. The four words are eight 16-bit numbers, one an element, low half first;
// an element is kept where its number is at least the threshold, p rounded to 1/65536. So the
// mask depends on the element's number alone, not on strides, launches or the machine, and
// the gradient is the same call on dy.
//
// Bound by HBM where ten rounds (twenty 32 x 32 bit products for eight elements) hide behind it.
#include "layer.hpp"
#include "mfma_util.hpp"

namespace muon {
namespace {

typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

__device__ __forceinline__ unsigned short to_bf16(float f) {
  return __builtin_bit_cast(unsigned short, static_cast<__bf16>(f));
}

__device__ __forceinline__ u32x4 philox(uint64_t counter, uint64_t offset, uint64_t seed) {
  uint32_t c0 = static_cast<uint32_t>(counter), c1 = static_cast<uint32_t>(counter >> 32);
  uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// Eight elements from element i of the array on, as 16- or 32-bit values in 16-byte pieces.
template <bool F32>
struct Eight {
  u32x4 v[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ float get(const Eight<F32>& x, int e) {
  if constexpr (F32) return __uint_as_float(x.v[e >> 2][e & 3]);
  else return __uint_as_float(e & 1 ? x.v[0][e >> 1] & 0xFFFF0000u : x.v[0][e >> 1] << 16);
}
template <bool F32>
__device__ __forceinline__ Eight<F32> load8(const void* p, int64_t at) {
  Eight<F32> x;
  if constexpr (F32) {
    const float* q = static_cast<const float*>(p) + at;
    x.v[0] = *reinterpret_cast<const u32x4_a4*>(q);
    x.v[1] = *reinterpret_cast<const u32x4_a4*>(q + 4);
  } else {
    x.v[0] = *reinterpret_cast<const u32x4_a2*>(static_cast<const unsigned short*>(p) + at);
  }
  return x;
}
template <bool F32>
__device__ __forceinline__ float load1(const void* p, int64_t at) {
  if constexpr (F32) return static_cast<const float*>(p)[at];
  else return __uint_as_float(static_cast<unsigned int>(static_cast<const unsigned short*>(p)[at]) << 16);
}

constexpr int kBlocks = 4;   // of eight elements a thread: that many loads in flight

template <bool F32, bool ADD>
__global__ __launch_bounds__(256) void drop(const DropParams p) {
  uint64_t seed = p.seed, offset = p.offset;
  if (p.counter) {
    seed = p.counter[0];
    offset = p.counter[1];
  }
  const int64_t n = p.rows * p.cols;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (256 * kBlocks) + threadIdx.x;
  Eight<F32> x[kBlocks], r[kBlocks];
  int64_t row[kBlocks], col[kBlocks];
  bool whole[kBlocks];
#pragma unroll
  for (int u = 0; u < kBlocks; ++u) {
    const int64_t i = (first + u * 256) * 8;
    row[u] = 0;
    col[u] = i;
    if (p.rows > 1 && i < n) {
      row[u] = i / p.cols;
      col[u] = i - row[u] * p.cols;
    }
    whole[u] = i < n && col[u] + 8 <= p.cols;
    if (whole[u]) {
      x[u] = load8<F32>(p.x, row[u] * p.ld_x + col[u]);
      if constexpr (ADD) r[u] = load8<F32>(p.residual, row[u] * p.ld_r + col[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < kBlocks; ++u) {
    const int64_t b = first + u * 256;
    if (b * 8 >= n) continue;
    const u32x4 bits = philox(static_cast<uint64_t>(b), offset, seed);
    if (whole[u]) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t number = e & 1 ? bits[e >> 1] >> 16 : bits[e >> 1] & 0xFFFFu;
        y[e] = number >= p.threshold ? get<F32>(x[u], e) * p.factor : 0.0f;
        if constexpr (ADD) y[e] += get<F32>(r[u], e);
      }
      const int64_t at = row[u] * p.ld_o + col[u];
      if constexpr (F32) {
        float* q = static_cast<float*>(p.out) + at;
        *reinterpret_cast<u32x4_a4*>(q) = u32x4{__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3])};
        *reinterpret_cast<u32x4_a4*>(q + 4) = u32x4{__float_as_uint(y[4]), __float_as_uint(y[5]), __float_as_uint(y[6]), __float_as_uint(y[7])};
      } else {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = to_bf16(y[2 * e]) | (static_cast<unsigned int>(to_bf16(y[2 * e + 1])) << 16);
        *reinterpret_cast<u32x4_a2*>(static_cast<unsigned short*>(p.out) + at) = w;
      }
    } else {
      // over a row's end, or the last elements
      int64_t rr = row[u], cc = col[u];
      for (int e = 0; e < 8 && b * 8 + e < n; ++e) {
        const uint32_t number = (bits[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
        float y = number >= p.threshold ? load1<F32>(p.x, rr * p.ld_x + cc) * p.factor : 0.0f;
        if constexpr (ADD) y += load1<F32>(p.residual, rr * p.ld_r + cc);
        if constexpr (F32) static_cast<float*>(p.out)[rr * p.ld_o + cc] = y;
        else static_cast<unsigned short*>(p.out)[rr * p.ld_o + cc] = to_bf16(y);
        if (++cc == p.cols) {
          cc = 0;
          ++rr;
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_dropout(bool f32, const DropParams& p, hipStream_t st) {
  const int64_t blocks = (p.rows * p.cols + 7) / 8;
  const dim3 grid(static_cast<unsigned>((blocks + 256 * kBlocks - 1) / (256 * kBlocks)));
  if (f32) {
    if (p.residual) drop<true, true><<<grid, 256, 0, st>>>(p);
    else drop<true, false><<<grid, 256, 0, st>>>(p);
  } else {
    if (p.residual) drop<false, true><<<grid, 256, 0, st>>>(p);
    else drop<false, false><<<grid, 256, 0, st>>>(p);
  }
  return hipGetLastError();
}

}  // namespace muon
