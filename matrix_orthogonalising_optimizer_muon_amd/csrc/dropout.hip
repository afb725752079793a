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
template <bool F32, bool ONCE>
__device__ __forceinline__ Eight<F32> load8(const void* p, int64_t at) {
  Eight<F32> x;
  if constexpr (F32) {
    const u32x4_a4* q = reinterpret_cast<const u32x4_a4*>(static_cast<const float*>(p) + at);
    x.v[0] = ONCE ? __builtin_nontemporal_load(q) : *q;
    x.v[1] = ONCE ? __builtin_nontemporal_load(q + 1) : q[1];
  } else {
    const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(static_cast<const unsigned short*>(p) + at);
    x.v[0] = ONCE ? __builtin_nontemporal_load(q) : *q;
  }
  return x;
}
template <bool F32>
__device__ __forceinline__ float load1(const void* p, int64_t at) {
  if constexpr (F32) return static_cast<const float*>(p)[at];
  else return __uint_as_float(static_cast<unsigned int>(static_cast<const unsigned short*>(p)[at]) << 16);
}

// Eight elements a thread. Two, four or eight such blocks a thread were slower: 16384 x 3584 bf16 with a residual 62.4 us
// with one (5.65 TB/s), 63.4, 66.0 and 69.1 us; without one 38.3 us (6.1 TB/s), 39.1, 43.7, 43.4 us; fp32 118 us (6.0
// TB/s) and 83 us (5.7 TB/s), 122 to 139 us and 85 to 96 us. ONCE: x and the residual are more than the caches keep and
// are read past them: 62.4 -> 54.1 us (6.5 TB/s); x alone 37.8 -> 39.8 us, so only with a residual.
template <bool F32, bool ADD, bool ONCE>
__global__ __launch_bounds__(256) void drop(const DropParams p) {
  const int64_t b = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, i = b * 8, n = p.rows * p.cols;
  if (i >= n) return;
  int64_t row = 0, col = i;
  if (p.rows > 1) {
    row = i / p.cols;
    col = i - row * p.cols;
  }
  const bool whole = col + 8 <= p.cols;
  Eight<F32> x, r;
  if (whole) {
    x = load8<F32, ONCE>(p.x, row * p.ld_x + col);
    if constexpr (ADD) r = load8<F32, ONCE>(p.residual, row * p.ld_r + col);
  }
  uint64_t seed = p.seed, offset = p.offset;
  if (p.counter) {
    seed = p.counter[0];
    offset = p.counter[1];
  }
  const u32x4 bits = philox(static_cast<uint64_t>(b), offset, seed);
  if (whole) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t number = e & 1 ? bits[e >> 1] >> 16 : bits[e >> 1] & 0xFFFFu;
      y[e] = number >= p.threshold ? get<F32>(x, e) * p.factor : 0.0f;
      if constexpr (ADD) y[e] += get<F32>(r, e);
    }
    const int64_t at = row * p.ld_o + col;
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
    return;
  }
  // over a row's end, or the last elements
  for (int e = 0; e < 8 && i + e < n; ++e) {
    const uint32_t number = (bits[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
    float y = number >= p.threshold ? load1<F32>(p.x, row * p.ld_x + col) * p.factor : 0.0f;
    if constexpr (ADD) y += load1<F32>(p.residual, row * p.ld_r + col);
    if constexpr (F32) static_cast<float*>(p.out)[row * p.ld_o + col] = y;
    else static_cast<unsigned short*>(p.out)[row * p.ld_o + col] = to_bf16(y);
    if (++col == p.cols) {
      col = 0;
      ++row;
    }
  }
}

}  // namespace

hipError_t launch_dropout(bool f32, const DropParams& p, hipStream_t st) {
  const int64_t blocks = (p.rows * p.cols + 7) / 8;
  const dim3 grid(static_cast<unsigned>((blocks + 255) / 256));
  const bool once = p.residual && p.rows * p.cols * (f32 ? 8 : 4) > (int64_t{128} << 20);  // half the 256 MB cache
  if (f32) {
    if (once) drop<true, true, true><<<grid, 256, 0, st>>>(p);
    else if (p.residual) drop<true, true, false><<<grid, 256, 0, st>>>(p);
    else drop<true, false, false><<<grid, 256, 0, st>>>(p);
  } else {
    if (once) drop<false, true, true><<<grid, 256, 0, st>>>(p);
    else if (p.residual) drop<false, true, false><<<grid, 256, 0, st>>>(p);
    else drop<false, false, false><<<grid, 256, 0, st>>>(p);
  }
  return hipGetLastError();
}

}  // namespace muon
